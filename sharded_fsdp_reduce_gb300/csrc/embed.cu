// embed.cu -- the token embedding: fsdp_embed (out[t] = scale W[token_t]), and
// the host side of its gradient, fsdp_embed_grad (the kernels: embed_grad.cu).
//
// The lookup reads the rows in use and writes every output row once: bound by
// HBM for long batches (rows of frequent tokens come from L2), by latency for a
// few tokens: one load of the token, one of its row. A warp copies 2 KB of a
// row, four 16-byte words a lane, all of them in flight at once.
#include <math.h>

#include "embed.cuh"

namespace fsdp {
namespace embed {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

template <int DT, bool VEC> __global__ void __launch_bounds__(kThreads) lookup_kernel(const LookupArgs a) {
    using S = Slice<DT, VEC>;
    wait_previous();
    allow_next();
    const int64_t at = int64_t(blockIdx.x) * kWarps + threadIdx.x / 32;
    const int64_t t = at / a.slices;
    if (t >= a.n) return;
    const int64_t col0 = (at - t * a.slices) * S::kCols + threadIdx.x % 32 * S::kElems;
    const int64_t token = a.tokens[t];
    uint8_t *out = a.out + t * a.out_bytes;
    float f[S::kElems];
    if (token < 0 || token >= a.vocab) {
        // padding has a row of zeros; a token outside the vocabulary shows as NaN
        const float v = token == a.ignore ? 0.0f : NAN;
#pragma unroll
        for (int e = 0; e < S::kElems; ++e) f[e] = v;
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            const int64_t col = col0 + j * 32 * S::kElems;
            if (col < a.dim) Word<DT, VEC>::store(out, col, f);
        }
        return;
    }
    const uint8_t *row = a.weight + token * a.weight_bytes;
    Word<DT, VEC> w[S::kWords];
#pragma unroll
    for (int j = 0; j < S::kWords; ++j) {
        const int64_t col = col0 + j * 32 * S::kElems;
        if (col < a.dim) w[j].load_cached(row, col);
    }
    const bool ignored = token == a.ignore;  // (an ignored token may be one of the vocabulary)
    const float scale = a.scale;
#pragma unroll
    for (int j = 0; j < S::kWords; ++j) {
        const int64_t col = col0 + j * 32 * S::kElems;
        if (col >= a.dim) continue;
        w[j].widen(f);
#pragma unroll
        for (int e = 0; e < S::kElems; ++e) f[e] = ignored ? 0.0f : f[e] * scale;
        Word<DT, VEC>::store(out, col, f);
    }
}

template <int DT> fsdp_status launch_type(LookupArgs a, cudaStream_t s) {
    // whole words: both sides aligned, and rows of whole words
    const bool vec = aligned(a.weight, 16) && aligned(a.out, 16) && a.weight_bytes % 16 == 0 && a.out_bytes % 16 == 0 &&
                     a.dim * Dtype<DT>::kSize % 16 == 0;
    const int64_t cols = vec ? Slice<DT, true>::kCols : Slice<DT, false>::kCols;
    a.slices = (a.dim + cols - 1) / cols;
    const int64_t blocks = (a.n * a.slices + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffff) return FSDP_ERR_INVALID_ARG;
    return launch_chained(vec ? lookup_kernel<DT, true> : lookup_kernel<DT, false>, static_cast<unsigned>(blocks),
                          kThreads, 0, s, a);
}

// ---------------------------------------------------------------- host: checks and plan

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

size_t span_bytes(int64_t rows, int64_t cols, int64_t ld, int size) {
    return rows > 0 ? static_cast<size_t>(((rows - 1) * ld + cols) * size) : 0;
}

// What both calls have: sizes, and a [tokens][dim] and a [vocab][dim] matrix.
fsdp_status check(int dtype, int64_t n, int64_t vocab, int64_t dim, const void *tokens, const void *rows,
                  int64_t ld_rows, const void *table, int64_t ld_table, float scale) {
    if (!dtype_valid(dtype)) return FSDP_ERR_UNSUPPORTED_DTYPE;
    constexpr int64_t kMost = int64_t(1) << 30, kMostLd = int64_t(1) << 34, kMostArea = int64_t(1) << 50;
    if (n < 0 || n > kMost || vocab < 1 || vocab > kMost || dim < 1 || dim > kMost || !isfinite(scale))
        return FSDP_ERR_INVALID_ARG;
    if ((n > 0 && (!tokens || !rows)) || !table) return FSDP_ERR_INVALID_ARG;
    if (ld_rows < dim || ld_rows > kMostLd || n > kMostArea / ld_rows || ld_table < dim || ld_table > kMostLd ||
        vocab > kMostArea / ld_table)
        return FSDP_ERR_INVALID_ARG;
    const int size = dtype_size(dtype);
    if (!aligned(tokens, 8) || !aligned(rows, size) || !aligned(table, size)) return FSDP_ERR_ALIGNMENT;
    const size_t n_rows = span_bytes(n, dim, ld_rows, size), n_table = span_bytes(vocab, dim, ld_table, size);
    const size_t n_tokens = static_cast<size_t>(n) * 8;
    if (overlaps(rows, n_rows, table, n_table) || overlaps(rows, n_rows, tokens, n_tokens) ||
        overlaps(table, n_table, tokens, n_tokens))
        return FSDP_ERR_INVALID_ARG;
    return FSDP_OK;
}

struct Plan {
    bool vec;
    int32_t passes, bits;
    int32_t block, words;
    int64_t blocks, slices, ld_part;
    // byte offsets into the workspace
    int64_t key[2], pos[2], tickets, part, bytes;
};

bool vectors(const fsdp_embed_grad_args &a) {
    const int size = dtype_size(a.dtype);
    return aligned(a.d_out, 16) && aligned(a.d_weight, 16) && a.ld_d_out * size % 16 == 0 &&
           a.ld_d_weight * size % 16 == 0 && a.dim * size % 16 == 0;
}

// p.bytes is enough for every call of no more tokens, however aligned.
Plan make_plan(const fsdp_embed_grad_args &a) {
    const int64_t n = a.count;
    Plan p;
    p.vec = vectors(a);
    int32_t bits = 1;  // of the largest key, which stands for no token
    while ((a.vocab >> bits) != 0) ++bits;
    p.passes = (bits + kMostBits - 1) / kMostBits;
    p.bits = (bits + p.passes - 1) / p.passes;
    // the slices as even as whole words of the lanes make them
    p.slices = ceil_div(a.dim * dtype_size(a.dtype), kSliceBytes);
    const int64_t lane_words = ceil_div(ceil_div(a.dim, p.vec ? 16 / dtype_size(a.dtype) : 1), 32);
    p.words = static_cast<int32_t>(ceil_div(lane_words, p.slices));
    // long blocks where there are enough of them for the four places on an SM
    const int64_t ctas = int64_t(sm_count() > 0 ? sm_count() : 1) * 4;
    p.block = kMostBlock;
    while (p.block > kLeastBlock && ceil_div(n, p.block) * p.slices < ctas) p.block /= 2;
    p.blocks = ceil_div(n, p.block);
    const int64_t most_blocks = ceil_div(n, kLeastBlock);
    p.ld_part = round_up(a.dim, 8);
    int64_t at = 0;
    auto take = [&at](int64_t bytes) {
        const int64_t here = at;
        at = round_up(at + bytes, 256);
        return here;
    };
    for (int i = 0; i < 2; ++i) {
        p.key[i] = take(4 * n);
        p.pos[i] = take(4 * n);
    }
    p.tickets = take(12 * most_blocks * p.slices);
    p.part = take(8 * most_blocks * p.ld_part);
    p.bytes = at;
    return p;
}

fsdp_status run_grad(const fsdp_embed_grad_args &a, const Plan &p, uint8_t *ws, cudaStream_t s) {
    const int size = dtype_size(a.dtype);
    fsdp_status st = FSDP_OK;
    SortArgs o;
    o.tokens = a.tokens;
    o.ignore = a.ignore_index;
    o.n = static_cast<uint32_t>(a.count);
    o.vocab = static_cast<uint32_t>(a.vocab);
    o.passes = p.passes;
    o.bits = p.bits;
    for (int i = 0; i < 2; ++i) {
        o.key[i] = reinterpret_cast<uint32_t *>(ws + p.key[i]);
        o.pos[i] = reinterpret_cast<uint32_t *>(ws + p.pos[i]);
    }
    o.tickets = reinterpret_cast<uint32_t *>(ws + p.tickets);
    o.n_tickets = static_cast<uint32_t>(3 * p.blocks * p.slices);
    const bool place = can_place(a.count, a.vocab);
    if (a.count > 0) st = place ? launch_place(o, s) : launch_sort(o, s);
    if (st != FSDP_OK || (a.count == 0 && a.accumulate)) return st;
    SumArgs r;
    const int last = place ? 0 : (p.passes - 1) % 2;
    r.key = o.key[last];
    r.pos = o.pos[last];
    r.n = o.n;
    r.vocab = o.vocab;
    r.dim = a.dim;
    r.d_out = static_cast<const uint8_t *>(a.d_out);
    r.d_weight = static_cast<uint8_t *>(a.d_weight);
    r.out_bytes = a.ld_d_out * size;
    r.weight_bytes = a.ld_d_weight * size;
    r.part = reinterpret_cast<float *>(ws + p.part);
    r.ld_part = p.ld_part;
    r.tickets = o.tickets;
    r.blocks = static_cast<uint32_t>(p.blocks);
    r.block = p.block;
    r.words = p.words;
    // three on an SM leave a place for the sums (32768 tokens, 128000 x 8192 bf16:
    // one 426 us, two 401, three 394, four 391; 1021, 50257 x 768: 29, 17.7, 15.9, 17.1)
    const int64_t fill = int64_t(sm_count() > 0 ? sm_count() : 1) * 3, most = (a.vocab + 31) / 32;
    r.fill_ctas = a.accumulate ? 0 : static_cast<uint32_t>(fill < most ? fill : most);
    r.tokens = a.tokens;
    r.ignore = a.ignore_index;
    r.size = size;
    r.slices = static_cast<uint32_t>(p.slices);
    r.scale = a.scale;
    return launch_sums(r, a.dtype, p.vec, a.accumulate != 0, s);
}

fsdp_status check_grad(const fsdp_embed_grad_args *a) {
    if (!a || (a->accumulate != 0 && a->accumulate != 1)) return FSDP_ERR_INVALID_ARG;
    return check(a->dtype, a->count, a->vocab, a->dim, a->tokens, a->d_out, a->ld_d_out, a->d_weight, a->ld_d_weight,
                 a->scale);
}

}  // namespace

fsdp_status launch_lookup(const LookupArgs &a, int dtype, cudaStream_t s) {
    switch (dtype) {
        case FSDP_BF16: return launch_type<FSDP_BF16>(a, s);
        case FSDP_F16: return launch_type<FSDP_F16>(a, s);
        default: return launch_type<FSDP_F32>(a, s);
    }
}

}  // namespace embed
}  // namespace fsdp

using namespace fsdp;

extern "C" {

FSDP_API fsdp_status fsdp_embed(const fsdp_embed_args *args, void *stream) {
    if (!args || args->reserved != 0) return FSDP_ERR_INVALID_ARG;
    const fsdp_embed_args &a = *args;
    const fsdp_status st = embed::check(a.dtype, a.count, a.vocab, a.dim, a.tokens, a.out, a.ld_out, a.weight,
                                        a.ld_weight, a.scale);
    if (st != FSDP_OK) return st;
    if (a.count == 0) return FSDP_OK;
    const int size = dtype_size(a.dtype);
    embed::LookupArgs l{a.tokens, a.count, a.vocab, a.dim, a.ignore_index, static_cast<const uint8_t *>(a.weight),
                        static_cast<uint8_t *>(a.out), a.ld_weight * size, a.ld_out * size, 0, a.scale};
    return embed::launch_lookup(l, a.dtype, static_cast<cudaStream_t>(stream));
}

FSDP_API fsdp_status fsdp_embed_grad_workspace(const fsdp_embed_grad_args *args, int64_t *bytes_out) {
    const fsdp_status st = embed::check_grad(args);
    if (st != FSDP_OK) return st;
    if (!bytes_out) return FSDP_ERR_INVALID_ARG;
    *bytes_out = args->count == 0 ? 0 : embed::make_plan(*args).bytes;
    return FSDP_OK;
}

FSDP_API fsdp_status fsdp_embed_grad(const fsdp_embed_grad_args *args, void *workspace, int64_t workspace_bytes,
                                     void *stream) {
    const fsdp_status st = embed::check_grad(args);
    if (st != FSDP_OK) return st;
    const fsdp_embed_grad_args &a = *args;
    const embed::Plan p = embed::make_plan(a);
    if (a.count > 0) {
        if (p.blocks * p.slices > 0x3fffffff) return FSDP_ERR_INVALID_ARG;
        if (!workspace || workspace_bytes < p.bytes) return FSDP_ERR_INVALID_ARG;
        if (!aligned(workspace, 256)) return FSDP_ERR_ALIGNMENT;
        const int size = dtype_size(a.dtype);
        const size_t n = static_cast<size_t>(p.bytes);
        if (overlaps(workspace, n, a.tokens, static_cast<size_t>(a.count) * 8) ||
            overlaps(workspace, n, a.d_out, embed::span_bytes(a.count, a.dim, a.ld_d_out, size)) ||
            overlaps(workspace, n, a.d_weight, embed::span_bytes(a.vocab, a.dim, a.ld_d_weight, size)))
            return FSDP_ERR_INVALID_ARG;
    }
    return embed::run_grad(a, p, static_cast<uint8_t *>(workspace), static_cast<cudaStream_t>(stream));
}

}  // extern "C"
