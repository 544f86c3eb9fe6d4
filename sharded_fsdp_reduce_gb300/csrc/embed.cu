// embed.cu -- the token embedding: fsdp_embed (out[t] = scale W[token_t]), and
// the host side of its gradient, fsdp_embed_grad (the kernels: embed_grad.cu).
//
// The lookup reads the rows in use and writes every output row once: bound by
// HBM for long batches (rows of frequent tokens come from L2), by latency for a
// few tokens: one load of the token, one of its row. A warp copies 2 KB of a
// row, four 16-byte words a lane, all of them in flight at once; of short rows
// it copies several, as many as its lanes hold and four after one another.
// 16384 tokens of a 128000 x 8192 bf16 table 59 us, 6.4 TB/s; of 768 columns
// 5.2; 65536 of 64 columns 3.5 (9.8 with a warp for each row). Rows of 16-bit
// elements that are not aligned go in pairs, bound by instructions: 65536 of
// 771 columns 50 us.
#include <math.h>

#include "embed.cuh"

namespace fsdp {
namespace embed {
namespace {

constexpr int kThreads = 256;

// A lane's rows, words of a row, and the elements of a word: 16 bytes where both
// rows are aligned to them, else two 16-bit elements (of which a row's first or
// last word may have one) or one fp32.
template <int DT, bool VEC, int ROWS> struct Lookup {
    static constexpr int kSize = Dtype<DT>::kSize;
    static constexpr int kElems = (VEC ? 16 : 4) / kSize;
    static constexpr int kWords = (VEC ? 4 : 8) / ROWS;
};

// Two 16-bit elements at a 2-byte boundary: one aligned word, or each by itself.
// (Both aligned words around them would reach two bytes before and behind: past
// the end of a table that ends there.)
__device__ __forceinline__ uint32_t load_pair(const uint8_t *p) {
    if ((reinterpret_cast<uintptr_t>(p) & 2) == 0) return __ldg(reinterpret_cast<const uint32_t *>(p));
    const uint16_t *half = reinterpret_cast<const uint16_t *>(p);
    return __ldg(half) | static_cast<uint32_t>(__ldg(half + 1)) << 16;
}

// The word at p, of the elements first .. of a row of dim; one that the row has
// not is not read.
template <int DT, bool VEC> __device__ __forceinline__ void load_word(const uint8_t *p, int first, int dim, uint4 &x) {
    if constexpr (VEC) {
        x = __ldg(reinterpret_cast<const uint4 *>(p));
    } else if constexpr (DT == FSDP_F32) {
        x.x = __ldg(reinterpret_cast<const uint32_t *>(p));
    } else if (first >= 0 && first + 1 < dim) {
        x.x = load_pair(p);
    } else {
        const uint32_t one = *reinterpret_cast<const uint16_t *>(first < 0 ? p + 2 : p);
        x.x = first < 0 ? one << 16 : one;
    }
}

// A word of the output: the values times scale, or `other` in their place.
template <int DT, bool VEC>
__device__ __forceinline__ void store_scaled(uint8_t *p, int first, int dim, const uint4 &x, float scale, bool instead,
                                             float other) {
    constexpr int kElems = (VEC ? 16 : 4) / Dtype<DT>::kSize;
    float f[kElems];
    if constexpr (DT == FSDP_F32) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < kElems; ++e) f[e] = __uint_as_float(w[e]);
    } else if constexpr (VEC) {
        unpack8<DT>(x, f);
    } else {
        f[0] = Dtype<DT>::load(&x.x, 0);
        f[1] = Dtype<DT>::load(&x.x, 1);
    }
#pragma unroll
    for (int e = 0; e < kElems; ++e) f[e] = instead ? other : f[e] * scale;
    if constexpr (VEC && DT == FSDP_F32) {
        st_state(reinterpret_cast<float *>(p), make_float4(f[0], f[1], f[2], f[3]));
    } else if constexpr (VEC) {
        st_stream(p, make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7])));
    } else if constexpr (DT == FSDP_F32) {
        *reinterpret_cast<float *>(p) = f[0];
    } else if (first >= 0 && first + 1 < dim) {
        *reinterpret_cast<uint32_t *>(p) = pack2<DT>(f[0], f[1]);
    } else {
        Dtype<DT>::store(p, first < 0 ? 1 : 0, first < 0 ? f[1] : f[0]);
    }
}

template <int DT, bool VEC, int ROWS> __global__ void __launch_bounds__(kThreads) lookup_kernel(const LookupArgs a) {
    using L = Lookup<DT, VEC, ROWS>;
    const int lanes = ROWS == 1 ? 32 : 1 << a.lanes_log;  // of a row
    const int lane = threadIdx.x % 32, dim = static_cast<int>(a.dim);
    const int64_t warp = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32;
    int64_t row0;
    int word0 = lane & (lanes - 1);
    if constexpr (ROWS == 1) {
        row0 = warp / a.slices;
        word0 += static_cast<int>(warp - row0 * a.slices) * (32 * L::kWords);
    } else {
        row0 = warp * (ROWS * 32 >> a.lanes_log) + (lane >> a.lanes_log);
    }
    wait_previous();
    allow_next();
    int64_t token[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t row = row0 + r * (32 / lanes);
        token[r] = row < a.n ? a.tokens[row] : -1;
    }
    uint4 x[ROWS][L::kWords];
    // a row's first element here (a pair begins at a 4-byte boundary of the output)
    auto first_of = [&](int64_t row) {
        const int first = word0 * L::kElems;
        if constexpr (VEC || L::kElems == 1) return first;
        return first - static_cast<int>((reinterpret_cast<uintptr_t>(a.out) + row * a.out_bytes) >> 1 & 1);
    };
    const int step = lanes * L::kElems;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t row = row0 + r * (32 / lanes);
        if (row >= a.n || token[r] < 0 || token[r] >= a.vocab) continue;
        const int first = first_of(row);
        const uint8_t *p = a.weight + token[r] * a.weight_bytes + int64_t(first) * L::kSize;
#pragma unroll
        for (int j = 0; j < L::kWords; ++j)
            if (first + j * step < dim) load_word<DT, VEC>(p + j * step * L::kSize, first + j * step, dim, x[r][j]);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t row = row0 + r * (32 / lanes);
        if (row >= a.n) continue;
        // padding has a row of zeros (it may be a token of the vocabulary); any
        // other token outside of it shows as NaN
        const bool none = token[r] == a.ignore, instead = none || token[r] < 0 || token[r] >= a.vocab;
        const int first = first_of(row);
        uint8_t *p = a.out + row * a.out_bytes + int64_t(first) * L::kSize;
#pragma unroll
        for (int j = 0; j < L::kWords; ++j)
            if (first + j * step < dim)
                store_scaled<DT, VEC>(p + j * step * L::kSize, first + j * step, dim, x[r][j], a.scale, instead,
                                      none ? 0.0f : NAN);
    }
}

template <int DT, bool VEC> fsdp_status launch_rows(LookupArgs a, cudaStream_t s) {
    // words of a row (unaligned pairs: one more at most than there are)
    const int64_t words = VEC ? a.dim * Dtype<DT>::kSize / 16 : DT == FSDP_F32 ? a.dim : a.dim / 2 + 1;
    constexpr int kRows = 4, kShort = 32 * Lookup<DT, VEC, kRows>::kWords;
    int64_t warps;
    if (words > kShort || a.n <= 32) {  // (few tokens: a warp each)
        a.slices = (words + 32 * Lookup<DT, VEC, 1>::kWords - 1) / (32 * Lookup<DT, VEC, 1>::kWords);
        warps = a.n * a.slices;
    } else {
        a.lanes_log = 0;
        while ((int64_t(Lookup<DT, VEC, kRows>::kWords) << a.lanes_log) < words) ++a.lanes_log;
        const int64_t each = kRows * 32 >> a.lanes_log;
        warps = (a.n + each - 1) / each;
    }
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffff) return FSDP_ERR_INVALID_ARG;
    return launch_chained(words > kShort || a.n <= 32 ? lookup_kernel<DT, VEC, 1> : lookup_kernel<DT, VEC, kRows>,
                          static_cast<unsigned>(blocks), kThreads, 0, s, a);
}

template <int DT> fsdp_status launch_type(const LookupArgs &a, cudaStream_t s) {
    // whole words: both sides aligned, and rows of whole words
    const bool vec = aligned(a.weight, 16) && aligned(a.out, 16) && a.weight_bytes % 16 == 0 && a.out_bytes % 16 == 0 &&
                     a.dim * Dtype<DT>::kSize % 16 == 0;
    return vec ? launch_rows<DT, true>(a, s) : launch_rows<DT, false>(a, s);
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
    // one 402 us, two 396, three 389, four 387; 1021, 50257 x 768: 31, 17.6, 15.8, 17.4)
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
                        static_cast<uint8_t *>(a.out), a.ld_weight * size, a.ld_out * size, 1, 5, a.scale};
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
