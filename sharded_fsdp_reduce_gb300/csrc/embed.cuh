// embed.cuh -- internal arguments of the token embedding: its lookup, and its
// gradient (a sort of the tokens, the rows of each added up, zeros elsewhere).
#pragma once

#include "chain.cuh"

namespace fsdp {
namespace embed {

struct LookupArgs {
    const int64_t *tokens;
    int64_t n, vocab, dim, ignore;
    const uint8_t *weight;
    uint8_t *out;
    int64_t weight_bytes, out_bytes;  // from one row to the next
    int64_t slices;                   // warps of a row
    int32_t lanes_log;                // or lanes of a short one, a power of two
    float scale;
};

fsdp_status launch_lookup(const LookupArgs &a, int dtype, cudaStream_t s);

// Bits of a sorting pass's digit, at most.
constexpr int kMostBits = 10;

struct SortArgs {
    const int64_t *tokens;
    int64_t ignore;
    uint32_t n, vocab;
    int32_t passes, bits;
    uint32_t *key[2], *pos[2];  // pass p writes the p % 2-th (up to 65536 entries: the last pass alone)
    uint32_t *tickets;          // cleared for the sums
    uint32_t n_tickets;
};

constexpr int kSliceBytes = 1024;  // of a row, for a CTA
// Sorted entries whose sums a CTA forms: 4, 8 or 16 for each of its warps.
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
