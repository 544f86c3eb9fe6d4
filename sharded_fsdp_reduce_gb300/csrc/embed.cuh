// embed.cuh -- internal arguments of the token embedding: its lookup, and its
// gradient (a sort of the tokens, the rows of each added up, zeros elsewhere).
#pragma once

#include "chain.cuh"

namespace fsdp {
namespace embed {

// What the lookup's warp copies of a row: 32 lanes times this many words of 16
// bytes, or of one element where rows are not 16-byte aligned.
template <int DT, bool VEC> struct Slice {
    static constexpr int kSize = Dtype<DT>::kSize;
    static constexpr int kElems = VEC ? 16 / kSize : 1;  // of a word
    static constexpr int kWords = VEC ? 4 : 16;          // of a lane
    static constexpr int kCols = 32 * kWords * kElems;
};

// kElems consecutive values as fp32, and back (rounded once).
template <int DT, bool VEC> struct Word;
template <int DT> struct Word<DT, true> {
    uint4 raw;
    __device__ __forceinline__ void load(const uint8_t *row, int64_t col) {
        raw = ld_stream(row + col * Dtype<DT>::kSize);
    }
    __device__ __forceinline__ void load_cached(const uint8_t *row, int64_t col) {
        raw = __ldg(reinterpret_cast<const uint4 *>(row + col * Dtype<DT>::kSize));
    }
    __device__ __forceinline__ void load_coherent(const uint8_t *row, int64_t col) {
        raw = *reinterpret_cast<const uint4 *>(row + col * Dtype<DT>::kSize);
    }
    __device__ __forceinline__ void widen(float *f) const {
        if constexpr (DT == FSDP_F32) {
            f[0] = __uint_as_float(raw.x), f[1] = __uint_as_float(raw.y);
            f[2] = __uint_as_float(raw.z), f[3] = __uint_as_float(raw.w);
        } else {
            unpack8<DT>(raw, f);
        }
    }
    __device__ __forceinline__ static void store(uint8_t *row, int64_t col, const float *f) {
        uint4 w;
        if constexpr (DT == FSDP_F32)
            w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        else
            w = make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]), pack2<DT>(f[6], f[7]));
        st_stream(row + col * Dtype<DT>::kSize, w);
    }
};
template <int DT> struct Word<DT, false> {
    float x;
    __device__ __forceinline__ void load(const uint8_t *row, int64_t col) { x = Dtype<DT>::load(row, col); }
    __device__ __forceinline__ void load_cached(const uint8_t *row, int64_t col) { load(row, col); }
    __device__ __forceinline__ void load_coherent(const uint8_t *row, int64_t col) { load(row, col); }
    __device__ __forceinline__ void widen(float *f) const { f[0] = x; }
    __device__ __forceinline__ static void store(uint8_t *row, int64_t col, const float *f) {
        Dtype<DT>::store(row, col, f[0]);
    }
};

struct LookupArgs {
    const int64_t *tokens;
    int64_t n, vocab, dim, ignore;
    const uint8_t *weight;
    uint8_t *out;
    int64_t weight_bytes, out_bytes;  // from one row to the next
    int64_t slices;                   // warps of a row
    float scale;
};

fsdp_status launch_lookup(const LookupArgs &a, int dtype, cudaStream_t s);

// Largest digit of a sorting pass, and the most passes (30-bit tokens).
constexpr int kMostBits = 10;

struct SortArgs {
    const int64_t *tokens;
    int64_t ignore;
    uint32_t n, vocab;
    int32_t passes, bits;
    uint32_t *key[2], *pos[2];  // a pass writes the p % 2-th (few entries: the last pass alone)
    uint32_t *tickets;          // cleared for the sums
    uint32_t n_tickets;
};

constexpr int kSliceBytes = 1024;  // of a row, for a CTA
constexpr int kSumWarps = 8, kLeastBlock = 4 * kSumWarps, kMostBlock = 16 * kSumWarps;

struct SumArgs {
    const uint32_t *key, *pos;  // tokens in order, and where they stood; key >= vocab: not a token
    uint32_t n, vocab;
    int64_t dim;
    const uint8_t *d_out;
    uint8_t *d_weight;
    int64_t out_bytes, weight_bytes;
    float *part;        // [blocks][2][ld_part]: sums of runs that cross a block's first or last entry
    int64_t ld_part;
    // [3][blocks][slices]: the parts that are there of the first group of a run
    // that begins in the block, its groups, the parts of a group that begins there
    uint32_t *tickets;
    uint32_t blocks, slices;
    int32_t block;      // entries of one
    int32_t words;      // of a lane in a slice
    // zeros for the rows that no token uses, by this many CTAs more
    uint32_t fill_ctas;
    const int64_t *tokens;
    int64_t ignore;
    int32_t size;       // of an element
    float scale;
};

// Few tokens: their order in key[0] and pos[0].
bool can_place(int64_t n, int64_t vocab);
fsdp_status launch_place(const SortArgs &a, cudaStream_t s);
fsdp_status launch_sort(const SortArgs &a, cudaStream_t s);
fsdp_status launch_sums(const SumArgs &a, int dtype, bool vec, bool add, cudaStream_t s);

}  // namespace embed
}  // namespace fsdp
