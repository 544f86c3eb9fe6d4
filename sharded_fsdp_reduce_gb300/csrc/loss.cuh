// loss.cuh -- internal arguments of the head loss: the three matrix products
// (logits, hidden gradient, weight gradient) and the row kernels between them.
#pragma once

#include <cuda.h>  // CUtensorMap

#include "chain.cuh"

namespace fsdp {
namespace loss {

// Tile of one CTA pair: 256 rows (128 per CTA) by 256 columns, 64 K at a time.
constexpr int kTileM = 256;
constexpr int kTileN = 256;
constexpr int kBlockK = 64;
// Columns whose exponentials share one reference (one epilogue warp's), their
// largest logit.
constexpr int kSpan = 64;
// What exponentials are stored times in fp16.
constexpr float kExpGain = 32768.0f;

// What a product's epilogue does with the accumulator.
enum Epilogue {
    kStats = 0,   // per row and span: largest logit and sum of exponentials (nothing stored)
    kExp = 1,     // kStats, and the exponentials stored (fp16, or fp32 for an fp32 head)
    kScale = 2,   // store scale * (accumulator + earlier bands)
};

// Operand orders of the three products: whether A and B are MN-major.
enum Orders { kLogits, kHiddenGrad, kWeightGrad };

struct GemmArgs {
    int64_t M, N;          // valid rows and columns
    int32_t kblocks;
    int32_t planes;        // 1, or 3 bf16 planes of an fp32 head's operands
    int32_t tiles_m, tiles_n, splits;
    int32_t k_each, k_more;  // K blocks of a split, and the splits that have one more
    int32_t group;         // tiles of the fast dimension visited together
    int32_t m_fast;        // 1: rows are the fast dimension
    int32_t operand_type;  // 0 fp16, 1 bf16
    // kStats, kExp
    const int64_t *targets;
    float *off, *sum;      // [spans][ld_rows]
    float *target_logit;   // [rows]
    int64_t ld_rows;
    // the same against a teacher's distribution (targets and target_logit are not used)
    const uint16_t *first;  // [rows][ld_first]: a row's entries before each span, and all of them
    int64_t ld_first;
    const int32_t *ids;     // [rows][top], in order
    float *at;              // [rows][top]: their logits
    int64_t top;
    float log2e;            // log2(e) / temperature
    // kScale
    const float *scale;    // device scalar, or NULL for 1
    float scale_const;     // and this constant factor
    const float *earlier;  // fp32 [M][ld_earlier] added to the accumulator, or NULL
    int64_t ld_earlier;
    void *out;
    int64_t ld_out, split_stride;
    int64_t store_cols;    // columns that may be written (the padding of workspace rows among them)
    int32_t store_bytes;   // 32, 16, or less: what out's base and stride are multiples of
    uint32_t *ticket;      // kStats, kExp: cleared for the row kernel that follows (or NULL)
    uint32_t *timeouts;
};


// One translation unit per output dtype of the gradients, and one for the logits.
// `exponentials`: where they go (used with kExp).
fsdp_status launch_logits(Epilogue ep, bool f32, const CUtensorMap &a, const CUtensorMap &b,
                          const CUtensorMap &exponentials, const GemmArgs &g, cudaStream_t s);
fsdp_status launch_soft_logits(Epilogue ep, bool f32, const CUtensorMap &a, const CUtensorMap &b,
                               const CUtensorMap &exponentials, const GemmArgs &g, cudaStream_t s);
fsdp_status launch_grad_bf16(Orders o, const CUtensorMap &a, const CUtensorMap &b, const GemmArgs &g, cudaStream_t s);
fsdp_status launch_grad_f16(Orders o, const CUtensorMap &a, const CUtensorMap &b, const GemmArgs &g, cudaStream_t s);
fsdp_status launch_grad_f32(Orders o, const CUtensorMap &a, const CUtensorMap &b, const GemmArgs &g, cudaStream_t s);

// Four warps wait, for at most `limit` cycles, for an arrival that comes after
// `arrive_after` cycles (never, if negative). outcomes[128]: 1 per thread
// whose wait saw it.
fsdp_status launch_wait_check(long long limit, long long arrive_after, int32_t *outcomes, uint32_t *timeouts,
                              cudaStream_t s);

// A few rows (loss_few.cu): the statistics per block instead of per span of
// columns. Up to about where the matrix products take over, dot products
// against those (us on the device, at 50257 x 768 / 32000 x 4096 / 128000 x
// 8192): bf16 losses of 4 rows 25 to 26 / 64 to 63 / 376 to 403, of 5 rows 55 to
// 26 / 123 to 69 / 716 to 382. An fp32 weight is packed first for the products:
// losses of 16 rows 108 to 134 / 269 to 416 / 2207 to 3037, of 24 rows 156 to
// 134 / 336 to 420 / 3171 to 3034, of 32 rows 200 to 134 / 445 to 421 / 3977 to
// 3044; gradients of 8 rows 207 to 242 / 608 to 732 / 4365 to 5286, of 12 rows
// 316 to 245 / 836 to 734 / 6363 to 5291.
inline int64_t few_rows(int dtype, bool grad) { return dtype == FSDP_F32 ? (grad ? 8 : 24) : (grad ? 0 : 4); }

// ---------------------------------------------------------------- a teacher's distribution

constexpr int64_t kIgnored = -100;        // target of a row without entries
constexpr int32_t kNoEntry = 0x7fffffff;  // id behind a row's last entry

// The teacher's entries, a row's in the order of their tokens: each one's
// probability over the entries and its logarithm.
struct SoftArgs {
    const void *teacher, *given;  // logits and tokens as the caller has them
    int64_t ld_teacher, ld_given;
    int32_t teacher_dtype, wide;  // wide: 64-bit tokens
    int64_t top, vocab;
    float temperature, inverse, log2e;  // 1 / temperature, log2(e) / temperature
    int32_t *ids;                 // [band][top]; NULL: the targets alone
    float2 *prob;                 // [band][top]: {p, log p}
    uint16_t *first;              // [band][ld_first], or NULL
    int64_t ld_first, spans;
    int64_t *targets;             // 0 for a row that counts, kIgnored, or vocab for one whose entries are wrong
};

// late: may run beside the kernel before it, whose predecessors have ended.
fsdp_status launch_prepare(const SoftArgs &a, int64_t row0, int64_t rows, bool late, cudaStream_t s);

// A few rows' logits to the gradients of them, in place.
struct FewSoftArgs {
    float *logits;
    const float2 *row_state;
    int64_t ld_logits, rows, vocab, top;
    const int64_t *targets;
    const int32_t *ids;
    const float2 *prob;
    float log2e;
};
fsdp_status launch_few_soft(const FewSoftArgs &a, cudaStream_t s);

// The distillation loss: args as the cross entropy's (its targets are not
// read), and the teacher's. In loss.cu.
fsdp_status soft_workspace(const fsdp_head_loss_args &args, int64_t top, int64_t *bytes_out);
fsdp_status soft_run(fsdp_head_loss_args args, SoftArgs soft, void *workspace, int64_t workspace_bytes, cudaStream_t s);
fsdp_status check_head(const fsdp_head_loss_args &args, const void *const *inputs, const size_t *input_bytes, int n_inputs);

struct FewArgs {
    const void *hidden, *weight;
    int64_t ld_hidden, ld_weight, rows, vocab, dim, blocks;
    const int64_t *targets;  // NULL: none
    float *off, *sum;  // [blocks][ld_rows]
    int64_t ld_rows;
    float *target_logit;
    float *logits;     // [rows][ld_logits], for the gradients, or NULL
    int64_t ld_logits;
    float log2e;       // log2(e), over the temperature
    uint32_t *ticket;  // cleared for the row kernel
};

struct FewGradArgs {
    const float *hidden, *weight, *logits;  // (soft: the gradients of the logits)
    int32_t soft;
    const float2 *row_state;  // {largest logit, sum of the exponentials against it}
    int64_t ld_hidden, ld_weight, ld_logits, rows, vocab, dim;
    const int64_t *targets;
    int64_t ignore;
    float *part;       // [parts][rows][ld_part]: the hidden gradient's sums
    int64_t ld_part, parts;
    float *d_weight;
    int64_t ld_d_weight;
    const float *scale;
};

int64_t few_blocks(int64_t vocab);
int64_t few_parts(int64_t vocab, int64_t dim);
fsdp_status launch_few(const FewArgs &a, int dtype, cudaStream_t s);
fsdp_status launch_few_dx(const FewGradArgs &a, cudaStream_t s);
fsdp_status launch_few_dw(const FewGradArgs &a, cudaStream_t s);

}  // namespace loss
}  // namespace fsdp
