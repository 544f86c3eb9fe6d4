// loss.cu -- softmax cross entropy of a linear head: fsdp_head_loss.
//
//   l[t,v] = sum_k X[t,k] W[v,k]        lse[t] = log sum_v exp l[t,v]
//   loss_t = lse[t] - l[t,y_t]          d[t,v] = exp(l[t,v] - lse[t]) - [v = y_t]
//   dX = g d W                          dW = g d^T X
//
// The logits in fp32 live in tensor memory only. The logits product's epilogue
// turns each span of 64 columns into exponentials against the span's own
// maximum, and keeps their fp32 sum and that maximum; a row kernel joins the
// spans into lse. Without gradients that is all: X and W are read, a few bytes
// per span are written. With gradients the exponentials of a band of tokens
// are also stored, in 16 bits, and turned in place into d; the two gradient
// products read d as it lies. That is three products of 2TVD operations
// instead of the four that forming the logits again would take, for one pass
// over the band (4 bytes an element): with D = 8192 a product's operations
// take 8 times that pass, with D = 768 about as long.
//
// What has fewer than 32 bits, for 16-bit heads: the stored exponentials (fp16)
// and d (the head's type, fp16 times 2^14), because the tensor cores take 16-bit
// operands and the pass is bound by its bytes. The gradients' error against 64
// bits is then 1.9e-3 for bf16 and 2.4e-4 for fp16 (1021 x 50257 x 768, 4096 x
// 50257 x 1280), where rounding nothing but the result leaves 1.7e-3 and 2.1e-4.
// Losses, sums, statistics and the target's p - 1 are fp32; fp32 heads keep
// fp32 exponentials and d in three parts.
#include <math.h>
#include <string.h>

#include "loss.cuh"

namespace fsdp {
namespace loss {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
// fp16 gradients of the logits are held times 2^14: d is at most 1 in
// magnitude, and a probability down to 2^-28 keeps all its bits.
constexpr float kHalfGain = 16384.0f;

// ---------------------------------------------------------------- rows

struct RowArgs {
    const float *off, *sum;  // [spans][ld_rows]
    int64_t ld_rows;
    int32_t spans;
    const float *target_logit;
    const int64_t *targets;
    int64_t rows, vocab, ignore;
    float2 *row_state;       // {largest logit, sum of the exponentials against it}
    float *token_loss;       // or NULL
    // the loss over all bands: block sums, joined by the last block
    double *part_sum;
    int64_t *part_count;
    int64_t first_block, all_blocks;
    uint32_t *ticket;
    float *loss, *scale;
    float grad_scale;
    int32_t mean;
};

__device__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
__device__ long long warp_sum(long long x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// e^x; e^0 is exactly 1.
__device__ __forceinline__ float exp_of(float x) { return exp2f(x * kLog2e); }

// (top, sum): sum * e^top. Joins another pair into it.
__device__ __forceinline__ void join(float &top, float &sum, float other_top, float other_sum) {
    const float most = fmaxf(top, other_top);
    if (most == -INFINITY) return;  // both empty
    sum = sum * exp_of(top - most) + other_sum * exp_of(other_top - most);
    top = most;
}

__device__ __forceinline__ void write_loss(const RowArgs &a, double sum, long long valid) {
    const double by = a.mean && valid > 0 ? static_cast<double>(valid) : 1.0;
    *a.loss = static_cast<float>(sum / by);
    *a.scale = static_cast<float>(a.grad_scale / by);
}

constexpr int kRows = 16;     // of a block
constexpr int kRowLoads = 8;  // spans a thread reads at once

// 16 rows per block of 1024 threads: a warp reads two spans of the 16 rows at
// a time (the statistics lie span by span), the 64 readers of a row share its
// spans. Latency-bound: 2 x 4 bytes per span and row, eight loads in flight
// per thread. The loss adds up per block, then over the blocks in one fixed
// order, in fp64.
__global__ void __launch_bounds__(1024) rows_kernel(const __grid_constant__ RowArgs a) {
    __shared__ float tops[32][kRows + 1], sums[32][kRows + 1];
    __shared__ double total[32];
    __shared__ long long count[32];
    __shared__ bool last;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    wait_previous();
    allow_next();
    {
        const int64_t row = int64_t(blockIdx.x) * kRows + lane % kRows;
        float top = -INFINITY, sum = 0.0f;
        if (row < a.rows) {
            const float *off = a.off + row, *part = a.sum + row;
            for (int s = threadIdx.x / kRows; s < a.spans; s += 1024 / kRows * kRowLoads) {
                float o[kRowLoads], x[kRowLoads];
#pragma unroll
                for (int i = 0; i < kRowLoads; ++i) {
                    const int at = s + 1024 / kRows * i;
                    o[i] = at < a.spans ? off[at * a.ld_rows] : -INFINITY;
                    x[i] = at < a.spans ? part[at * a.ld_rows] : 0.0f;
                }
                float most = top;
#pragma unroll
                for (int i = 0; i < kRowLoads; ++i) most = fmaxf(most, o[i]);
                sum *= exp_of(top - most);
#pragma unroll
                for (int i = 0; i < kRowLoads; ++i) sum += x[i] * exp_of(o[i] - most);
                top = most;
            }
        }
        join(top, sum, __shfl_xor_sync(0xffffffffu, top, kRows), __shfl_xor_sync(0xffffffffu, sum, kRows));
        if (lane < kRows) {
            tops[warp][lane] = top;
            sums[warp][lane] = sum;
        }
    }
    __syncthreads();
    if (warp < kRows) {  // a warp per row
        const int64_t row = int64_t(blockIdx.x) * kRows + warp;
        float top = tops[lane][warp], sum = sums[lane][warp];
#pragma unroll
        for (int o = 16; o; o >>= 1)
            join(top, sum, __shfl_xor_sync(0xffffffffu, top, o), __shfl_xor_sync(0xffffffffu, sum, o));
        if (lane == 0) {
            float t = 0.0f;
            long long valid = 0;
            if (row < a.rows) {
                a.row_state[row] = make_float2(top, sum);
                const int64_t y = a.targets[row];
                if (y != a.ignore) {
                    valid = 1;
                    // log sum + (top - target): the sum is at least 1, the
                    // target at most top, and both terms are small for a row
                    // that is sure of its target. A target outside the
                    // vocabulary has no loss: it shows as NaN.
                    t = y >= 0 && y < a.vocab ? logf(sum) + (top - a.target_logit[row]) : NAN;
                }
                if (a.token_loss != nullptr) a.token_loss[row] = t;
            }
            total[warp] = t;
            count[warp] = valid;
        }
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double loss = 0.0;
        long long valid = 0;
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            loss += total[r];
            valid += count[r];
        }
        last = false;
        if (a.all_blocks == 1) {
            write_loss(a, loss, valid);
        } else {
            a.part_sum[a.first_block + blockIdx.x] = loss;
            a.part_count[a.first_block + blockIdx.x] = valid;
            __threadfence();
            last = atomicAdd(a.ticket, 1u) + 1 == static_cast<uint32_t>(a.all_blocks);
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double x = 0.0;
    long long n = 0;
    for (int64_t i = threadIdx.x; i < a.all_blocks; i += 1024) {
        x += __ldcg(a.part_sum + i);
        n += __ldcg(reinterpret_cast<const long long *>(a.part_count) + i);
    }
    x = warp_sum(x);
    n = warp_sum(n);
    if (lane == 0) {
        total[warp] = x;
        count[warp] = n;
    }
    __syncthreads();
    if (warp == 0) {
        x = warp_sum(total[lane]);
        n = warp_sum(count[lane]);
        if (lane == 0) write_loss(a, x, n);
    }
}

// The gradients' common factor before the last band's loss is known: the
// valid rows of every band (only when there are several).
__global__ void __launch_bounds__(1024)
    count_kernel(const int64_t *targets, int64_t rows, int64_t ignore, float grad_scale, int mean, float *scale) {
    __shared__ long long count[32];
    wait_previous();
    allow_next();
    long long n = 0;
    for (int64_t i = threadIdx.x; i < rows; i += 1024) n += targets[i] != ignore;
    n = warp_sum(n);
    if (threadIdx.x % 32 == 0) count[threadIdx.x / 32] = n;
    __syncthreads();
    if (threadIdx.x < 32) {
        n = warp_sum(count[threadIdx.x]);
        if (threadIdx.x == 0) *scale = static_cast<float>(grad_scale / (mean && n > 0 ? static_cast<double>(n) : 1.0));
    }
}

// ---------------------------------------------------------------- d from the exponentials

struct GradArgs {
    void *e;                 // [rows][ld] exponentials; 16-bit types: d in place
    uint16_t *planes[3];     // an fp32 head: d as three bf16 planes
    int64_t ld, rows, vocab;
    const float *off;        // [spans][ld_rows]
    int64_t ld_rows;
    const float2 *row_state;
    const float *target_logit;
    const int64_t *targets;
    int64_t ignore;
    uint32_t row_blocks;
};

// x in three bf16 parts: each takes the next 8 bits. An infinite x is in the
// last part alone, which is multiplied with the other operand's first one and
// no other: the sums then see infinity times a number of that operand's sign
// (or times 0), as they would in fp32. In the first part it would also meet
// the other's lower parts, which may be 0 or of the other sign.
__device__ __forceinline__ void split3(float x, float &hi, float &mid, float &lo) {
    constexpr float kMost = 3.38953139e38f;  // bf16's largest: what rounds past it
    const bool infinite = isinf(x);
    const float y = infinite ? 0.0f : x;
    hi = __bfloat162float(__float2bfloat16_rn(y));
    if (hi > kMost) hi = kMost;
    if (hi < -kMost) hi = -kMost;
    const float r = y - hi;
    mid = __bfloat162float(__float2bfloat16_rn(r));
    lo = infinite ? x : r - mid;
}

constexpr int kGradCols = 512, kGradRows = 64;

// 64 rows x 512 columns per block, 8 columns per thread and row. Bound by HBM
// (or L2, where the band fits): 4 bytes moved per element in 16-bit types.
template <int DT> __global__ void __launch_bounds__(256) grad_kernel(const __grid_constant__ GradArgs a) {
    __shared__ float factor[kGradCols / kSpan][kGradRows];
    __shared__ int32_t hit[kGradRows];  // the target's column in this block, or -1; -2: no gradient
    __shared__ float at_target[kGradRows];
    // from the last columns to the first, as the logits product left them in L2
    const uint32_t block = gridDim.x - 1 - blockIdx.x;
    const int64_t row0 = int64_t(block % a.row_blocks) * kGradRows;
    const int64_t col0 = int64_t(block / a.row_blocks) * kGradCols;
    constexpr float kGain = DT == FSDP_F16 ? kHalfGain : 1.0f;
    constexpr float kFactor = DT == FSDP_F32 ? kGain : kGain / kExpGain;
    wait_previous();
    allow_next();
    for (int i = threadIdx.x; i < kGradRows * (kGradCols / kSpan); i += 256) {
        const int r = i % kGradRows, s = i / kGradRows;
        const int64_t row = row0 + r, span = col0 / kSpan + s;
        if (row < a.rows) {
            // e times e^(the span's largest - the row's) / sum is the
            // probability; a target outside the vocabulary makes the row's
            // gradient NaN, as its loss is
            const int64_t y = a.targets[row], at = y - col0;
            const bool bad = y != a.ignore && (y < 0 || y >= a.vocab);
            const float2 state = a.row_state[row];
            if (span * kSpan < a.vocab)
                factor[s][r] = bad ? NAN : kFactor * exp_of(a.off[span * a.ld_rows + row] - state.x) / state.y;
            if (s == 0) {
                hit[r] = y == a.ignore ? -2 : at >= 0 && at < kGradCols ? static_cast<int32_t>(at) : -1;
                // the target's own d from its fp32 logit: near 1 the stored
                // exponential's rounding would be all that is left of p - 1
                if (hit[r] >= 0 && at + col0 < a.vocab)
                    at_target[r] = kGain * (exp_of(a.target_logit[row] - state.x) / state.y - 1.0f);
            }
        }
    }
    __syncthreads();
    const int c = threadIdx.x % (kGradCols / 8) * 8;
    const int64_t col = col0 + c;
    if (col >= a.vocab) return;
    const int rows = static_cast<int>(min(int64_t(kGradRows), a.rows - row0));
#pragma unroll 4
    for (int r = threadIdx.x / (kGradCols / 8); r < rows; r += 256 / (kGradCols / 8)) {
        const int64_t at = (row0 + r) * a.ld + col;
        const float f = factor[c / kSpan][r];
        const int h = hit[r] - c;
        float v[8];
        if constexpr (DT == FSDP_F32) {
            const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.e) + at);
            const float4 y = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.e) + at + 4);
            v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
        } else {
            unpack8<FSDP_F16>(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.e) + at), v);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[j] = h == j ? at_target[r] : v[j] * f;
        }
        if (hit[r] == -2) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        }
        if constexpr (DT == FSDP_F32) {
            float p[3][8];
#pragma unroll
            for (int j = 0; j < 8; ++j) split3(v[j], p[0][j], p[1][j], p[2][j]);
#pragma unroll
            for (int z = 0; z < 3; ++z)
                *reinterpret_cast<uint4 *>(a.planes[z] + at) =
                    make_uint4(pack2<FSDP_BF16>(p[z][0], p[z][1]), pack2<FSDP_BF16>(p[z][2], p[z][3]),
                               pack2<FSDP_BF16>(p[z][4], p[z][5]), pack2<FSDP_BF16>(p[z][6], p[z][7]));
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.e) + at) =
                make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
        }
    }
}

// ---------------------------------------------------------------- operands TMA cannot address

// rows x cols at stride ld into 16-bit rows padded to ldp (a multiple of 8):
// a copy for 16-bit types, three bf16 planes for fp32. With targets (hidden
// states), rows that are ignored become zeros.
template <bool F32>
__global__ void __launch_bounds__(256) pack_kernel(const void *src, int64_t rows, int64_t cols, int64_t ld,
                                                   uint16_t *dst, int64_t ldp, int64_t plane,
                                                   const int64_t *targets, int64_t ignore, bool vec) {
    const int64_t words = ldp / 8, total = rows * words;
    wait_previous();
    allow_next();
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / words, c = (i - r * words) * 8;
        const bool zero = targets != nullptr && targets[r] == ignore;
        const int n = zero ? 0 : static_cast<int>(min(int64_t(8), cols - c));
        if constexpr (F32) {
            const float *s = static_cast<const float *>(src) + r * ld + c;
            float x[8], p[3][8];
            if (vec && n == 8) {
                const float4 lo = *reinterpret_cast<const float4 *>(s), hi = *reinterpret_cast<const float4 *>(s + 4);
                x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = j < n ? s[j] : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) split3(x[j], p[0][j], p[1][j], p[2][j]);
#pragma unroll
            for (int z = 0; z < 3; ++z)
                *reinterpret_cast<uint4 *>(dst + z * plane + r * ldp + c) =
                    make_uint4(pack2<FSDP_BF16>(p[z][0], p[z][1]), pack2<FSDP_BF16>(p[z][2], p[z][3]),
                               pack2<FSDP_BF16>(p[z][4], p[z][5]), pack2<FSDP_BF16>(p[z][6], p[z][7]));
        } else {
            const uint16_t *s = static_cast<const uint16_t *>(src) + r * ld + c;
            if (vec && n == 8) {
                *reinterpret_cast<uint4 *>(dst + r * ldp + c) = *reinterpret_cast<const uint4 *>(s);
                continue;
            }
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t lo = 2 * j < n ? s[2 * j] : 0u, hi = 2 * j + 1 < n ? s[2 * j + 1] : 0u;
                w[j] = lo | (hi << 16);
            }
            *reinterpret_cast<uint4 *>(dst + r * ldp + c) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---------------------------------------------------------------- split products

// out = scale * sum over the splits, in their order.
template <int DT>
__global__ void __launch_bounds__(256) join_kernel(const float *part, int splits, int64_t split_stride, int64_t rows,
                                                   int64_t cols, int64_t ldp, const float *scale, float scale_const,
                                                   void *out, int64_t ld) {
    wait_previous();
    allow_next();
    const float f = scale_const * *scale;
    const int64_t words = ldp / 4, total = rows * words;
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < total; i += int64_t(gridDim.x) * 256) {
        const int64_t r = i / words, c = (i - r * words) * 4;
        float4 x = *reinterpret_cast<const float4 *>(part + r * ldp + c);
        for (int s = 1; s < splits; ++s) {
            const float4 y = *reinterpret_cast<const float4 *>(part + s * split_stride + r * ldp + c);
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        const float v[4] = {x.x * f, x.y * f, x.z * f, x.w * f};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c + j < cols) Dtype<DT>::store(out, r * ld + c + j, v[j]);
    }
}

// ---------------------------------------------------------------- host: the plan

constexpr int64_t kDefaultBandBytes = int64_t(4) << 30;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

struct Plan {
    bool f32, grad, few, pack_x, pack_w;
    int64_t band, bands, spans, ldv, ldd, blocks;
    int splits_x, splits_w;
    // byte offsets into the workspace
    int64_t scale, ticket, part_sum, part_count, row_state, target_logit, off, sum, x, w, e, d, part, sum_w, bytes;
};

constexpr int kMostSplits = 32;

// How many pieces a product's K is cut into: with few tiles most pairs would
// idle, and with little more than a multiple of the pairs the last round is
// nearly empty. Takes the least of rounds of K blocks (about 0.3 us for each
// of its plane products) plus the fp32 partial results written and read (about
// 6 TB/s).
int choose_splits(int64_t tiles, int64_t kblocks, int products, int64_t m, int64_t n) {
    const int64_t pairs = sm_count() / 2 > 0 ? sm_count() / 2 : 1;
    int best = 1;
    double least = 0.0;
    for (int s = 1; s <= kMostSplits && (s == 1 || kblocks * products / s >= 8); ++s) {
        const double rounds = static_cast<double>(ceil_div(tiles * s, pairs));
        double us = rounds * (static_cast<double>(ceil_div(kblocks, s)) * products * 0.3 + 2.0);
        if (s > 1) us += 4.0 + static_cast<double>(m) * n * 8.0 * s / 6.0e6;
        if (s == 1 || us < least) {
            least = us;
            best = s;
        }
    }
    return best;
}

// The power of two, at most 32, that an address and a stride in bytes are multiples of.
int32_t alignment(const void *p, int64_t stride) {
    const uintptr_t both = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(stride) | 32;
    return static_cast<int32_t>(both & -both);
}

bool direct(const void *p, int64_t ld) { return aligned(p, 16) && ld % 8 == 0; }

// Rows that the default budget allows a band.
int64_t budget_band(int64_t bytes_per_row) {
    const int64_t band = kDefaultBandBytes / bytes_per_row / kTileM * kTileM;
    return band < kTileM ? kTileM : band;
}

int hidden_splits(const fsdp_head_loss_args &a, int64_t rows) {
    return choose_splits(ceil_div(rows, kTileM) * ceil_div(a.dim, kTileN), ceil_div(a.vocab, kBlockK),
                         a.dtype == FSDP_F32 ? 6 : 1, rows, round_up(a.dim, 64));
}
int weight_splits(const fsdp_head_loss_args &a, int64_t rows) {
    return choose_splits(ceil_div(a.vocab, kTileM) * ceil_div(a.dim, kTileN), ceil_div(rows, kBlockK),
                         a.dtype == FSDP_F32 ? 6 : 1, a.vocab, round_up(a.dim, 64));
}

// How a call runs.
Plan choose(const fsdp_head_loss_args &a) {
    Plan p;
    memset(&p, 0, sizeof(p));
    p.f32 = a.dtype == FSDP_F32;
    p.grad = a.d_hidden != nullptr || a.d_weight != nullptr;
    // (the few rows' gradient kernels take up to 2^16 column tiles)
    p.few = a.tokens <= few_rows(a.dtype, p.grad) && a.dim <= (1 << 22);
    // the weight gradient multiplies every row's hidden values: the packed copy
    // has zeros in ignored rows, so that what lies there (padding that was never
    // written) does not matter
    p.pack_x = !p.few && (p.f32 || a.d_weight != nullptr || !direct(a.hidden, a.ld_hidden));
    p.pack_w = !p.few && (p.f32 || !direct(a.weight, a.ld_weight));
    p.ldv = round_up(a.vocab, 64);
    p.ldd = round_up(a.dim, 64);
    p.spans = p.few ? few_blocks(a.vocab) : ceil_div(a.vocab, kSpan);
    int64_t band = p.few ? a.tokens : a.band;  // (a few rows are one band whatever was asked for)
    if (band == 0) {
        // gradients: what fits the default budget (exponentials, and the planes
        // of an fp32 head); losses alone: the statistics (8 bytes a span and
        // row) stay below it for any band this size
        band = budget_band(p.grad ? p.ldv * (p.f32 ? 10 : 2) : 8 * p.spans);
        // as many bands as that takes, of nearly equal length
        const int64_t each = ceil_div(a.tokens, ceil_div(a.tokens, band));
        band = round_up(each, kTileM) < band ? round_up(each, kTileM) : band;
    }
    p.band = band < a.tokens ? band : a.tokens;
    p.bands = ceil_div(a.tokens, p.band);
    p.blocks = 0;
    for (int64_t b = 0; b < p.bands; ++b) {
        const int64_t rows = a.tokens - b * p.band < p.band ? a.tokens - b * p.band : p.band;
        p.blocks += ceil_div(rows, kRows);
    }
    p.splits_x = p.splits_w = 1;
    if (a.d_hidden) p.splits_x = p.few ? static_cast<int>(few_parts(a.vocab, a.dim)) : hidden_splits(a, p.band);
    if (a.d_weight && p.bands == 1 && !p.few) p.splits_w = weight_splits(a, p.band);
    return p;
}

// What the workspace's parts hold.
struct Room {
    int64_t blocks, band, stats, x, w, e, d, part, sum_w;  // counts of the first three, then bytes
};

int64_t larger(int64_t a, int64_t b) { return a > b ? a : b; }

Room room_of(const fsdp_head_loss_args &a, const Plan &p) {
    Room r;
    memset(&r, 0, sizeof(r));
    const int64_t planes = p.f32 ? 3 : 1;
    r.blocks = p.blocks;
    r.band = p.band;
    r.stats = p.spans * p.band;
    if (p.pack_x) r.x = 2 * planes * a.tokens * p.ldd;
    if (p.pack_w) r.w = 2 * planes * a.vocab * p.ldd;
    if (p.grad) {
        r.e = p.band * p.ldv * (p.f32 ? 4 : 2);
        if (p.f32 && !p.few) r.d = p.band * p.ldv * 6;
        if (p.splits_x > 1 || p.few) r.part = 4 * p.splits_x * p.band * p.ldd;
        if (p.splits_w > 1) r.part = larger(r.part, 4 * p.splits_w * a.vocab * p.ldd);
        if (a.d_weight && p.bands > 1) r.sum_w = 4 * a.vocab * p.ldd;
    }
    return r;
}

// Every part as large as any call of at most this one's tokens needs it. A
// shorter call can need more of some than a longer one: it may cut a product
// into more pieces, work in one band where the longer one takes two halves,
// or run as a few rows.
Room room_up_to(const fsdp_head_loss_args &a) {
    const Plan p = choose(a);
    Room r = room_of(a, p);
    if (p.few) return r;  // (grows with the rows)
    fsdp_head_loss_args few = a;
    few.tokens = few_rows(a.dtype, p.grad);
    if (few.tokens > 0 && a.dim <= (1 << 22)) {
        const Plan q = choose(few);
        const Room f = room_of(few, q);
        r.band = larger(r.band, f.band);
        r.stats = larger(r.stats, f.stats);
        r.e = larger(r.e, f.e);
        r.part = larger(r.part, f.part);
    }
    // the longest band of these calls: they are as long as their tokens up to
    // what was asked for or what the budget allows
    int64_t band = a.band > 0 ? a.band : budget_band(p.grad ? p.ldv * (p.f32 ? 10 : 2) : 8 * p.spans);
    band = band < a.tokens ? band : a.tokens;
    r.band = larger(r.band, band);
    r.stats = larger(r.stats, p.spans * band);
    if (p.grad) {
        r.e = larger(r.e, band * p.ldv * (p.f32 ? 4 : 2));
        if (p.f32) r.d = band * p.ldv * 6;
        if (a.d_hidden) {
            // the more rows of a tile, the fewer pieces: the tile's first row
            // has the most, its last the longest
            for (int64_t rows = 1; rows <= band; rows += kTileM) {
                const int s = hidden_splits(a, rows);
                const int64_t end = rows + kTileM - 1 < band ? rows + kTileM - 1 : band;
                if (s > 1) r.part = larger(r.part, 4 * s * end * p.ldd);
            }
        }
        if (a.d_weight) {
            int most = 1;
            for (int64_t rows = 1; rows <= band && most < kMostSplits; rows += kBlockK)
                if (const int s = weight_splits(a, rows); s > most) most = s;
            if (most > 1) r.part = larger(r.part, 4 * most * a.vocab * p.ldd);
        }
    }
    return r;
}

// The parts one after another, at multiples of a kilobyte.
void place(Plan &p, const Room &r) {
    int64_t at = 0;
    auto take = [&at](int64_t bytes) {
        const int64_t here = at;
        at = round_up(at + bytes, 1024);
        return here;
    };
    p.scale = take(8);
    p.ticket = p.scale + 4;
    p.part_sum = take(8 * r.blocks);
    p.part_count = take(8 * r.blocks);
    p.row_state = take(8 * r.band);
    p.target_logit = take(4 * r.band);
    p.off = take(4 * r.stats);
    p.sum = take(4 * r.stats);
    p.x = take(r.x);
    p.w = take(r.w);
    p.e = take(r.e);
    p.d = r.d > 0 ? take(r.d) : p.e;
    p.part = take(r.part);
    p.sum_w = take(r.sum_w);
    p.bytes = at;
}

Plan make_plan(const fsdp_head_loss_args &a) {
    Plan p = choose(a);
    place(p, room_of(a, p));
    return p;
}

// The bytes that are enough for this call and for every shorter one.
int64_t bytes_up_to(const fsdp_head_loss_args &a) {
    Plan p = choose(a);
    place(p, room_up_to(a));
    return p.bytes;
}

// ---------------------------------------------------------------- host: tensor maps

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime's lookup (the library links no
// driver library of its own); null if the driver has none.
EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess || !f) {
            (void)cudaGetLastError();
            return static_cast<EncodeFn>(nullptr);
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// Rows of `cols` elements at stride ld, `planes` of them; boxes of box_bytes
// (128, or 64) by box_rows by all planes, swizzled over as many bytes, zeros
// outside.
fsdp_status make_map(CUtensorMap *map, CUtensorMapDataType type, const void *base, int64_t cols, int64_t rows,
                     int64_t planes, int64_t ld, int64_t plane, int box_rows, int box_bytes = 128) {
    const EncodeFn fn = encode_fn();
    if (!fn) return cuda_status(cudaErrorNotSupported);
    const int size = type == CU_TENSOR_MAP_DATA_TYPE_FLOAT32 ? 4 : 2;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(planes)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * size), static_cast<cuuint64_t>(plane * size)};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_bytes / size), static_cast<cuuint32_t>(box_rows),
                               static_cast<cuuint32_t>(planes)};
    const cuuint32_t unit[3] = {1, 1, 1};
    const CUresult r = fn(map, type, 3, const_cast<void *>(base), dims, strides, box, unit,
                          CU_TENSOR_MAP_INTERLEAVE_NONE,
                          box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? FSDP_OK : cuda_status(cudaErrorInvalidValue);
}

int grid_of(int64_t items) {
    const int64_t want = ceil_div(items, 256), most = static_cast<int64_t>(sm_count()) * 16;
    return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

// ---------------------------------------------------------------- host: one call

// A 16-bit operand as its products see it.
struct Operand {
    const uint8_t *base;
    int64_t ld, plane;
    int planes;
};

fsdp_status pack(const void *src, bool f32, int64_t rows, int64_t cols, int64_t ld, uint8_t *dst, int64_t ldp,
                 const int64_t *targets, int64_t ignore, cudaStream_t s) {
    const int grid = grid_of(rows * ldp / 8);
    uint16_t *d = reinterpret_cast<uint16_t *>(dst);
    return launch_chained(f32 ? pack_kernel<true> : pack_kernel<false>, static_cast<unsigned>(grid), 256, 0, s, src,
                          rows, cols, ld, d, ldp, rows * ldp, targets, ignore,
                          aligned(src, 16) && ld * (f32 ? 4 : 2) % 16 == 0);
}

fsdp_status launch_grad(int dtype, Orders o, const CUtensorMap &a, const CUtensorMap &b, const GemmArgs &g,
                        cudaStream_t s) {
    switch (dtype) {
        case FSDP_BF16: return launch_grad_bf16(o, a, b, g, s);
        case FSDP_F16: return launch_grad_f16(o, a, b, g, s);
        default: return launch_grad_f32(o, a, b, g, s);
    }
}

// One gradient product: out [M,N] of dtype at stride ld = scale * (A B + earlier), K split as planned.
struct Product {
    Orders orders;
    int64_t M, N, K;
    int splits;
    const float *earlier;
    int64_t ld_earlier;
    void *out;
    int64_t ld_out;
    int out_dtype;
    bool scaled;  // false: a band's fp32 sum, scaled with the last band
};

fsdp_status run_product(const Product &q, const Plan &p, const fsdp_head_loss_args &a, uint8_t *ws,
                        const CUtensorMap &ma, const CUtensorMap &mb, cudaStream_t s) {
    GemmArgs g;
    memset(&g, 0, sizeof(g));
    g.M = q.M;
    g.N = q.N;
    g.kblocks = static_cast<int32_t>(ceil_div(q.K, kBlockK));
    g.planes = p.f32 ? 3 : 1;
    g.tiles_m = static_cast<int32_t>(ceil_div(q.M, kTileM));
    g.tiles_n = static_cast<int32_t>(ceil_div(q.N, kTileN));
    g.splits = q.splits;
    // dW: all column tiles of a row tile together (d is read once, X stays in
    // L2); dX: squares of tiles, both operands being long in K
    g.m_fast = q.orders == kHiddenGrad;
    g.group = q.orders == kHiddenGrad ? 8 : 32;
    g.operand_type = a.dtype == FSDP_F16 ? 0 : 1;
    const float *scale = reinterpret_cast<const float *>(ws + p.scale);
    const float gain = a.dtype == FSDP_F16 ? 1.0f / kHalfGain : 1.0f;
    g.timeouts = a.wait_timeouts;
    if (q.splits > 1) {
        g.scale_const = 1.0f;
        float *part = reinterpret_cast<float *>(ws + p.part);
        g.out = part;
        g.ld_out = g.store_cols = p.ldd;
        g.split_stride = q.M * p.ldd;
        g.store_bytes = 32;
        const fsdp_status st = launch_grad_f32(q.orders, ma, mb, g, s);
        if (st != FSDP_OK) return st;
        auto join = q.out_dtype == FSDP_BF16  ? join_kernel<FSDP_BF16>
                    : q.out_dtype == FSDP_F16 ? join_kernel<FSDP_F16>
                                              : join_kernel<FSDP_F32>;
        return launch_chained(join, static_cast<unsigned>(grid_of(q.M * p.ldd / 4)), 256, 0, s,
                              static_cast<const float *>(part), q.splits, q.M * p.ldd, q.M, q.N, p.ldd, scale, gain,
                              q.out, q.ld_out);
    }
    g.scale = q.scaled ? scale : nullptr;
    g.scale_const = q.scaled ? gain : 1.0f;
    g.earlier = q.earlier;
    g.ld_earlier = q.ld_earlier;
    g.out = q.out;
    g.ld_out = q.ld_out;
    g.store_cols = q.N;
    g.store_bytes = alignment(q.out, q.ld_out * dtype_size(q.out_dtype));
    return launch_grad(q.out_dtype, q.orders, ma, mb, g, s);
}

fsdp_status run_few(const fsdp_head_loss_args &a, const Plan &p, uint8_t *ws, cudaStream_t s) {
    FewArgs f;
    f.hidden = a.hidden;
    f.weight = a.weight;
    f.ld_hidden = a.ld_hidden;
    f.ld_weight = a.ld_weight;
    f.rows = a.tokens;
    f.vocab = a.vocab;
    f.dim = a.dim;
    f.blocks = p.spans;
    f.targets = a.targets;
    f.off = reinterpret_cast<float *>(ws + p.off);
    f.sum = reinterpret_cast<float *>(ws + p.sum);
    f.ld_rows = p.band;
    f.target_logit = reinterpret_cast<float *>(ws + p.target_logit);
    f.ticket = reinterpret_cast<uint32_t *>(ws + p.ticket);
    f.logits = p.grad ? reinterpret_cast<float *>(ws + p.e) : nullptr;
    f.ld_logits = p.ldv;
    return launch_few(f, a.dtype, s);
}

// The gradients of a few fp32 rows, from their logits and lse.
fsdp_status run_few_grad(const fsdp_head_loss_args &a, const Plan &p, uint8_t *ws, cudaStream_t s) {
    FewGradArgs f;
    f.hidden = static_cast<const float *>(a.hidden);
    f.weight = static_cast<const float *>(a.weight);
    f.logits = reinterpret_cast<const float *>(ws + p.e);
    f.row_state = reinterpret_cast<const float2 *>(ws + p.row_state);
    f.ld_hidden = a.ld_hidden;
    f.ld_weight = a.ld_weight;
    f.ld_logits = p.ldv;
    f.rows = a.tokens;
    f.vocab = a.vocab;
    f.dim = a.dim;
    f.targets = a.targets;
    f.ignore = a.ignore_index;
    f.part = reinterpret_cast<float *>(ws + p.part);
    f.ld_part = p.ldd;
    f.parts = p.splits_x;
    f.d_weight = static_cast<float *>(a.d_weight);
    f.ld_d_weight = a.ld_d_weight;
    f.scale = reinterpret_cast<const float *>(ws + p.scale);
    if (a.d_hidden) {
        fsdp_status st = launch_few_dx(f, s);
        if (st == FSDP_OK)
            st = launch_chained(join_kernel<FSDP_F32>, static_cast<unsigned>(grid_of(a.tokens * p.ldd / 4)), 256, 0, s,
                                static_cast<const float *>(f.part), p.splits_x, a.tokens * p.ldd, a.tokens, a.dim,
                                p.ldd, f.scale, 1.0f, a.d_hidden, a.ld_d_hidden);
        if (st != FSDP_OK) return st;
    }
    return a.d_weight ? launch_few_dw(f, s) : FSDP_OK;
}

// The rows' sums and losses, of one band.
fsdp_status run_rows(const fsdp_head_loss_args &a, const Plan &p, uint8_t *ws, int64_t row0, int64_t rows,
                     int64_t &block, cudaStream_t s) {
    RowArgs r;
    r.off = reinterpret_cast<const float *>(ws + p.off);
    r.sum = reinterpret_cast<const float *>(ws + p.sum);
    r.ld_rows = p.band;
    r.spans = static_cast<int32_t>(p.spans);
    r.target_logit = reinterpret_cast<const float *>(ws + p.target_logit);
    r.targets = a.targets + row0;
    r.rows = rows;
    r.vocab = a.vocab;
    r.ignore = a.ignore_index;
    r.row_state = reinterpret_cast<float2 *>(ws + p.row_state);
    r.token_loss = a.token_loss ? a.token_loss + row0 : nullptr;
    r.part_sum = reinterpret_cast<double *>(ws + p.part_sum);
    r.part_count = reinterpret_cast<int64_t *>(ws + p.part_count);
    r.first_block = block;
    r.all_blocks = p.blocks;
    r.ticket = reinterpret_cast<uint32_t *>(ws + p.ticket);
    r.loss = a.loss;
    r.scale = reinterpret_cast<float *>(ws + p.scale);
    r.grad_scale = a.grad_scale;
    r.mean = a.reduction == FSDP_LOSS_MEAN;
    const unsigned blocks = static_cast<unsigned>(ceil_div(rows, kRows));
    block += blocks;
    return launch_chained(rows_kernel, blocks, 1024, 0, s, r);
}

fsdp_status run(const fsdp_head_loss_args &a, const Plan &p, uint8_t *ws, cudaStream_t s) {
    int64_t block = 0;
    if (p.few) {
        fsdp_status few = run_few(a, p, ws, s);
        if (few == FSDP_OK) few = run_rows(a, p, ws, 0, a.tokens, block, s);
        return few == FSDP_OK && p.grad ? run_few_grad(a, p, ws, s) : few;
    }
    const int64_t D = a.dim, V = a.vocab;
    const int size = dtype_size(a.dtype);
    const int planes = p.f32 ? 3 : 1;
    Operand x{static_cast<const uint8_t *>(a.hidden), a.ld_hidden, a.tokens * a.ld_hidden, 1};
    Operand w{static_cast<const uint8_t *>(a.weight), a.ld_weight, V * a.ld_weight, 1};
    fsdp_status st = FSDP_OK;
    if (p.pack_x) {
        st = pack(a.hidden, p.f32, a.tokens, D, a.ld_hidden, ws + p.x, p.ldd, a.targets, a.ignore_index, s);
        x = Operand{ws + p.x, p.ldd, a.tokens * p.ldd, planes};
    }
    if (st == FSDP_OK && p.pack_w) {
        st = pack(a.weight, p.f32, V, D, a.ld_weight, ws + p.w, p.ldd, nullptr, 0, s);
        w = Operand{ws + p.w, p.ldd, V * p.ldd, planes};
    }
    if (st != FSDP_OK) return st;
    float *scale = reinterpret_cast<float *>(ws + p.scale);
    if (p.grad && p.bands > 1) {
        st = launch_chained(count_kernel, 1, 1024, 0, s, a.targets, a.tokens, a.ignore_index, a.grad_scale,
                            static_cast<int>(a.reduction == FSDP_LOSS_MEAN), scale);
        if (st != FSDP_OK) return st;
    }
    const CUtensorMapDataType t16 =
        a.dtype == FSDP_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap w_k, w_n;
    st = make_map(&w_k, t16, w.base, D, V, w.planes, w.ld, w.plane, 128);
    if (st == FSDP_OK) st = make_map(&w_n, t16, w.base, D, V, w.planes, w.ld, w.plane, 64);
    if (st != FSDP_OK) return st;
    for (int64_t b = 0; b < p.bands; ++b) {
        const int64_t row0 = b * p.band;
        const int64_t rows = a.tokens - row0 < p.band ? a.tokens - row0 : p.band;
        const uint8_t *xb = x.base + 2 * row0 * x.ld;
        CUtensorMap x_k, x_n, e_out;
        st = make_map(&x_k, t16, xb, D, rows, x.planes, x.ld, x.plane, 128);
        if (st != FSDP_OK) return st;
        // the logits, as statistics and exponentials
        GemmArgs g;
        memset(&g, 0, sizeof(g));
        g.M = rows;
        g.N = V;
        g.kblocks = static_cast<int32_t>(ceil_div(D, kBlockK));
        g.planes = p.f32 ? 3 : 1;
        g.tiles_m = static_cast<int32_t>(ceil_div(rows, kTileM));
        g.tiles_n = static_cast<int32_t>(ceil_div(V, kTileN));
        g.splits = 1;
        g.m_fast = 1;  // W is the long operand: read once, X stays in L2
        g.group = 16;
        g.operand_type = a.dtype == FSDP_F16 ? 0 : 1;
        g.targets = a.targets + row0;
        g.off = reinterpret_cast<float *>(ws + p.off);
        g.sum = reinterpret_cast<float *>(ws + p.sum);
        g.target_logit = reinterpret_cast<float *>(ws + p.target_logit);
        g.ld_rows = p.band;
        g.ticket = b == 0 ? reinterpret_cast<uint32_t *>(ws + p.ticket) : nullptr;
        g.timeouts = a.wait_timeouts;
        e_out = x_k;
        if (p.grad) {
            st = make_map(&e_out, p.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, ws + p.e,
                          p.ldv, rows, 1, p.ldv, rows * p.ldv, 32, 64);
            if (st != FSDP_OK) return st;
        }
        st = launch_logits(p.grad ? kExp : kStats, p.f32, x_k, w_k, e_out, g, s);
        if (st != FSDP_OK) return st;
        if ((st = run_rows(a, p, ws, row0, rows, block, s)) != FSDP_OK) return st;
        if (!p.grad) continue;
        // d, then the two products
        GradArgs d;
        memset(&d, 0, sizeof(d));
        d.e = ws + p.e;
        const int64_t plane = rows * p.ldv;
        if (p.f32)
            for (int z = 0; z < 3; ++z) d.planes[z] = reinterpret_cast<uint16_t *>(ws + p.d) + z * plane;
        d.ld = p.ldv;
        d.rows = rows;
        d.vocab = V;
        d.off = g.off;
        d.ld_rows = p.band;
        d.row_state = reinterpret_cast<const float2 *>(ws + p.row_state);
        d.target_logit = g.target_logit;
        d.targets = g.targets;
        d.ignore = a.ignore_index;
        d.row_blocks = static_cast<uint32_t>(ceil_div(rows, kGradRows));
        const int64_t all = ceil_div(V, kGradCols) * d.row_blocks;
        if (all > 0x7fffffff) return FSDP_ERR_INVALID_ARG;
        const unsigned dgrid = static_cast<unsigned>(all);
        auto grad = a.dtype == FSDP_BF16  ? grad_kernel<FSDP_BF16>
                    : a.dtype == FSDP_F16 ? grad_kernel<FSDP_F16>
                                          : grad_kernel<FSDP_F32>;
        if ((st = launch_chained(grad, dgrid, 256, 0, s, d)) != FSDP_OK) return st;
        if (a.d_hidden) {
            CUtensorMap d_k;
            st = make_map(&d_k, t16, ws + p.d, V, rows, planes, p.ldv, plane, 128);
            if (st != FSDP_OK) return st;
            const Product q{kHiddenGrad, rows, D, V, p.splits_x, nullptr, 0,
                            static_cast<uint8_t *>(a.d_hidden) + row0 * a.ld_d_hidden * size, a.ld_d_hidden,
                            static_cast<int>(a.dtype), true};
            if ((st = run_product(q, p, a, ws, d_k, w_n, s)) != FSDP_OK) return st;
        }
        if (a.d_weight) {
            CUtensorMap d_m;
            st = make_map(&d_m, t16, ws + p.d, V, rows, planes, p.ldv, plane, 64);
            if (st == FSDP_OK) st = make_map(&x_n, t16, xb, D, rows, x.planes, x.ld, x.plane, 64);
            if (st != FSDP_OK) return st;
            float *sum_w = reinterpret_cast<float *>(ws + p.sum_w);
            const bool last = b + 1 == p.bands;
            const Product q{kWeightGrad, V, D, rows, p.splits_w, b > 0 ? sum_w : nullptr, p.ldd,
                            last ? a.d_weight : sum_w, last ? a.ld_d_weight : p.ldd,
                            last ? static_cast<int>(a.dtype) : static_cast<int>(FSDP_F32), last};
            if ((st = run_product(q, p, a, ws, d_m, x_n, s)) != FSDP_OK) return st;
        }
    }
    return FSDP_OK;
}

// ---------------------------------------------------------------- host: checks

size_t span_bytes(int64_t rows, int64_t cols, int64_t ld, int size) {
    return rows > 0 ? static_cast<size_t>(((rows - 1) * ld + cols) * size) : 0;
}

fsdp_status check(const fsdp_head_loss_args *a) {
    if (!a) return FSDP_ERR_INVALID_ARG;
    if (!dtype_valid(a->dtype)) return FSDP_ERR_UNSUPPORTED_DTYPE;
    constexpr int64_t kMost = int64_t(1) << 30;  // tile coordinates are 32-bit
    if (a->tokens < 0 || a->tokens > kMost || a->vocab < 1 || a->vocab > kMost || a->dim < 1 || a->dim > kMost)
        return FSDP_ERR_INVALID_ARG;
    if (a->reserved != 0 || a->band < 0 || (a->reduction != FSDP_LOSS_MEAN && a->reduction != FSDP_LOSS_SUM) || !isfinite(a->grad_scale))
        return FSDP_ERR_INVALID_ARG;
    // products of sizes stay far inside 64 bits
    constexpr int64_t kMostLd = int64_t(1) << 34, kMostArea = int64_t(1) << 50;
    if (a->tokens > kMostArea / a->vocab) return FSDP_ERR_INVALID_ARG;
    const int size = dtype_size(a->dtype);
    struct Matrix {
        const void *p;
        int64_t rows, ld;
        bool needed;
    } m[4] = {{a->hidden, a->tokens, a->ld_hidden, a->tokens > 0},
              {a->weight, a->vocab, a->ld_weight, true},
              {a->d_hidden, a->tokens, a->ld_d_hidden, false},
              {a->d_weight, a->vocab, a->ld_d_weight, false}};
    for (const Matrix &x : m) {
        if (!x.p) {
            if (x.needed) return FSDP_ERR_INVALID_ARG;
            continue;
        }
        if (x.ld < a->dim || x.ld > kMostLd || x.rows > kMostArea / x.ld) return FSDP_ERR_INVALID_ARG;
        if (!aligned(x.p, size)) return FSDP_ERR_ALIGNMENT;
    }
    if (!a->loss || (a->tokens > 0 && !a->targets)) return FSDP_ERR_INVALID_ARG;
    if (!aligned(a->loss, 4) || !aligned(a->token_loss, 4) || !aligned(a->targets, 8) || !aligned(a->wait_timeouts, 4))
        return FSDP_ERR_ALIGNMENT;
    // no output overlaps an input or another output
    const void *in[3] = {a->hidden, a->weight, a->targets};
    const size_t nin[3] = {span_bytes(a->tokens, a->dim, a->ld_hidden, size),
                           span_bytes(a->vocab, a->dim, a->ld_weight, size), static_cast<size_t>(a->tokens) * 8};
    const void *out[4] = {a->loss, a->token_loss, a->d_hidden, a->d_weight};
    const size_t nout[4] = {4, a->token_loss ? static_cast<size_t>(a->tokens) * 4 : 0,
                            a->d_hidden ? span_bytes(a->tokens, a->dim, a->ld_d_hidden, size) : 0,
                            a->d_weight ? span_bytes(a->vocab, a->dim, a->ld_d_weight, size) : 0};
    for (int i = 0; i < 4; ++i) {
        for (int k = 0; k < 3; ++k)
            if (overlaps(out[i], nout[i], in[k], nin[k])) return FSDP_ERR_INVALID_ARG;
        for (int k = i + 1; k < 4; ++k)
            if (overlaps(out[i], nout[i], out[k], nout[k])) return FSDP_ERR_INVALID_ARG;
    }
    return FSDP_OK;
}

}  // namespace
}  // namespace loss
}  // namespace fsdp

using namespace fsdp;

extern "C" {

FSDP_API fsdp_status fsdp_head_loss_workspace(const fsdp_head_loss_args *args, int64_t *bytes_out) {
    const fsdp_status st = loss::check(args);
    if (st != FSDP_OK) return st;
    if (!bytes_out) return FSDP_ERR_INVALID_ARG;
    *bytes_out = args->tokens == 0 ? 0 : loss::bytes_up_to(*args);
    return FSDP_OK;
}

FSDP_API fsdp_status fsdp_head_loss(const fsdp_head_loss_args *args, void *workspace, int64_t workspace_bytes,
                                    void *stream) {
    const fsdp_status st = loss::check(args);
    if (st != FSDP_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const fsdp_head_loss_args &a = *args;
    if (a.tokens == 0) {
        // no rows: a loss of 0 and a zero weight gradient
        cudaError_t e = cudaMemsetAsync(a.loss, 0, 4, s);
        if (e == cudaSuccess && a.d_weight) {
            const size_t size = static_cast<size_t>(dtype_size(a.dtype));
            e = cudaMemset2DAsync(a.d_weight, a.ld_d_weight * size, 0, a.dim * size, a.vocab, s);
        }
        return cuda_status(e);
    }
    const loss::Plan p = loss::make_plan(a);
    if (!workspace || workspace_bytes < p.bytes) return FSDP_ERR_INVALID_ARG;
    if (!aligned(workspace, 1024)) return FSDP_ERR_ALIGNMENT;
    const void *used[7] = {a.hidden, a.weight, a.targets, a.loss, a.token_loss, a.d_hidden, a.d_weight};
    const size_t size = static_cast<size_t>(dtype_size(a.dtype));
    const size_t bytes[7] = {((a.tokens - 1) * a.ld_hidden + a.dim) * size,
                             ((a.vocab - 1) * a.ld_weight + a.dim) * size,
                             static_cast<size_t>(a.tokens) * 8,
                             4,
                             a.token_loss ? static_cast<size_t>(a.tokens) * 4 : 0,
                             a.d_hidden ? ((a.tokens - 1) * a.ld_d_hidden + a.dim) * size : 0,
                             a.d_weight ? ((a.vocab - 1) * a.ld_d_weight + a.dim) * size : 0};
    for (int i = 0; i < 7; ++i)
        if (overlaps(used[i], bytes[i], workspace, static_cast<size_t>(p.bytes))) return FSDP_ERR_INVALID_ARG;
    // the operands' tiles are bulk copies between device buffers
    if (host_resident(a.hidden) || host_resident(a.weight)) return FSDP_ERR_INVALID_ARG;
    return loss::run(a, p, static_cast<uint8_t *>(workspace), s);
}

FSDP_API fsdp_status fsdp_check_head_loss_wait(int64_t limit_cycles, int64_t arrive_after_cycles, int32_t *outcomes,
                                               uint32_t *wait_timeouts, void *stream) {
    constexpr int64_t kMost = int64_t(1) << 31;
    if (limit_cycles < 1 || limit_cycles > kMost || arrive_after_cycles > kMost || !outcomes)
        return FSDP_ERR_INVALID_ARG;
    if (!aligned(outcomes, 4) || !aligned(wait_timeouts, 4)) return FSDP_ERR_ALIGNMENT;
    return loss::launch_wait_check(limit_cycles, arrive_after_cycles, outcomes, wait_timeouts,
                                   static_cast<cudaStream_t>(stream));
}

}  // extern "C"
