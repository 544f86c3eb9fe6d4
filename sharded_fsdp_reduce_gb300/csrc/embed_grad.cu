// embed_grad.cu -- the gradient of the token embedding:
//
//   dW[v] = scale * (sum of dY[t] over the tokens t that are v, in their order)
//
// written to the whole table, or added to the rows in use.
//
// The tokens are put in order first, in one launch (few by counting, more by a
// stable radix sort in a cluster), so that a row's summands lie side by side and
// add up in one fixed order: the same bits every time, whatever order the warps
// run in. A second launch has the sums, 32 to 128 sorted entries and 1 KB of
// their rows to a CTA: what begins and ends within them is written at once, a
// run that crosses to other CTAs' entries leaves fp32 parts, which the last of
// them adds in order. The first CTAs of that launch fill the rows that no token
// uses with zeros; they run beside the sort as well.
//
// Bound by HBM for large tables and long batches: dY is read once, the table
// written once. 32768 tokens of a 128000 x 8192 bf16 table: 388 us, 6.7 TB/s.
// Bound by the two launches' latency for a few tokens added to a table (1021 of
// 50257 x 768: 8 us; 8192: 20).
#include "embed.cuh"
#include "tcgen.cuh"

namespace fsdp {
namespace embed {
namespace {

// ---------------------------------------------------------------- sort

// 512 threads of at most 64 registers: an SM has room for CTAs of the zeros
// beside one of these.
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32, kItems = 8;
constexpr uint32_t kTile = kSortThreads * kItems;  // entries of a CTA in one go
constexpr int kMostCtas = 16;                      // of the cluster (eight are portable)
constexpr uint32_t kDigits = 1u << kMostBits;
static_assert(kDigits <= 2 * kSortThreads && kTile < 65536, "a thread has two digits; counts of a tile fit 16 bits");

struct SortShared {
    uint32_t count[kSortWarps][kDigits / 2];  // of two digits: entries of a warp; then those of the warps before it
    uint2 total[kDigits / 2];                 // of two digits over the CTA (its peers read them)
    uint32_t base[kDigits];                   // where its next entry with a digit goes
    uint32_t sums[kSortWarps];
    uint32_t local[kDigits];                  // where the tile's entries with a digit are in `staged`
    uint2 staged[kTile];                      // the tile's entries {key, position} by digit
    uint2 entry[kTile];                       // the CTA's entries between passes, of few entries
};

__device__ __forceinline__ uint2 load_peer(const uint2 *p, uint32_t rank) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
                 : "=r"(v.x), "=r"(v.y)
                 : "r"(tc::peer_addr(tma::smem_addr(p), rank))
                 : "memory");
    return v;
}
__device__ __forceinline__ void store_peer(uint2 *p, uint32_t rank, uint2 v) {
    asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(tc::peer_addr(tma::smem_addr(p), rank)), "r"(v.x),
                 "r"(v.y)
                 : "memory");
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}

// Exclusive sum over the block's threads.
__device__ __forceinline__ uint32_t before_all(uint32_t x, uint32_t *sums) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint32_t sum = x;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    uint32_t all = lane < kSortWarps ? sums[lane] : 0u;
#pragma unroll
    for (int o = 1; o < kSortWarps; o *= 2) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, all, o);
        if (lane >= o) all += y;
    }
    const uint32_t warps_before = __shfl_sync(0xffffffffu, all, max(warp - 1, 0));
    __syncthreads();
    return sum - x + (warp > 0 ? warps_before : 0u);
}

// One tile's entries in registers: a warp holds 32 * items consecutive ones.
struct SortTile {
    uint32_t key[kItems], pos[kItems];
    uint32_t spot[kItems];  // digit << 16 | place among the warp's entries with that digit
    int items;
    uint32_t first;  // this lane's first entry (the next ones are 32 apart)
    uint32_t end;
};

// LARGE: between passes the entries are in memory, else in the CTAs' shared memory.
template <bool LARGE>
__device__ __forceinline__ void load_tile(const SortArgs &a, const SortShared &s, int pass, uint32_t begin, uint32_t end,
                                          SortTile &t) {
    t.items = static_cast<int>((end - begin + kSortThreads - 1) / kSortThreads);
    const uint32_t local = threadIdx.x / 32 * 32 * t.items + threadIdx.x % 32;
    t.first = begin + local;
    t.end = end;
    const uint32_t *key = a.key[(pass + 1) % 2], *pos = a.pos[(pass + 1) % 2];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t at = t.first + 32 * i;
        t.key[i] = 0;
        if (i >= t.items || at >= end) continue;
        if (pass == 0) {
            const int64_t token = a.tokens[at];
            const bool none = token == a.ignore || token < 0 || token >= a.vocab;
            t.key[i] = none ? a.vocab : static_cast<uint32_t>(token);
            t.pos[i] = at;
        } else if constexpr (LARGE) {
            t.key[i] = __ldcg(key + at);
            t.pos[i] = __ldcg(pos + at);
        } else {
            const uint2 e = s.entry[local + 32 * i];
            t.key[i] = e.x;
            t.pos[i] = e.y;
        }
    }
}

// Every entry's digit and its place among the warp's; then, per digit, the
// warps' counts become what comes before them. Returns the counts of this
// thread's two digits over the tile.
__device__ __forceinline__ uint2 rank_tile(SortShared &s, SortTile &t, int shift, int bits) {
    const uint32_t digits = 1u << bits;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint16_t *count = reinterpret_cast<uint16_t *>(s.count[warp]);
    for (uint32_t d = lane; d < (digits + 1) / 2; d += 32) s.count[warp][d] = 0;
    __syncwarp();
    // the lanes with the same digit, of every entry
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (i >= t.items) break;  // (the same for all)
        uint32_t peers = __ballot_sync(0xffffffffu, t.first + 32 * i < t.end);
#pragma unroll
        for (int b = 0; b < kMostBits; ++b) {
            if (b >= bits) break;
            const bool one = t.key[i] >> (shift + b) & 1u;
            const uint32_t ones = __ballot_sync(0xffffffffu, one);
            peers &= one ? ones : ~ones;
        }
        t.spot[i] = peers;
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (i >= t.items) break;
        const bool live = t.first + 32 * i < t.end;
        const uint32_t digit = (t.key[i] >> shift) & (digits - 1), peers = t.spot[i];
        uint32_t before = 0;
        if (live) before = count[digit];
        __syncwarp();
        if (live && lane == __ffs(peers) - 1) count[digit] = static_cast<uint16_t>(before + __popc(peers));
        __syncwarp();
        t.spot[i] = digit << 16 | (before + __popc(peers & ((1u << lane) - 1)));
    }
    __syncthreads();
    uint32_t sum = 0;  // two counts in one word: neither passes 16 bits
    if (2 * threadIdx.x < digits) {
        uint32_t x[kSortWarps];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) x[w] = s.count[w][threadIdx.x];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            s.count[w][threadIdx.x] = sum;
            sum += x[w];
        }
    }
    return make_uint2(sum & 0xffffu, sum >> 16);
}

// A stable radix sort by digits of up to 10 bits. Each CTA has a stretch of the
// entries; the CTAs' counts of every digit tell where its entries go, which it
// puts in that order first, so that neighbours go out together. Entries
// that are no token have the key `vocab` and come last. Up to sixteen tiles of
// entries stay in the cluster's shared memory until the last pass (LARGE: more,
// through memory). Bound by latency: two passes over 8192 entries take 9 us,
// over 32768 16, over 65536 18; through memory over 131072 45, over a million 308.
template <bool LARGE>
__global__ void __launch_bounds__(kSortThreads, 2) sort_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    SortShared &s = *reinterpret_cast<SortShared *>(raw);
    const uint32_t rank = tc::cluster_rank(), ctas = cluster_size();
    uint32_t each = (a.n + ctas - 1) / ctas;
    const int each_log = 32 - __clz(max(each, 2u) - 1);
    if constexpr (!LARGE) each = 1u << each_log;  // (at most a tile)
    const uint32_t begin = min(rank * each, a.n), end = min(begin + each, a.n);
    const uint32_t digits = 1u << a.bits;
    wait_previous();
    allow_next();
    for (uint32_t i = rank * kSortThreads + threadIdx.x; i < a.n_tickets; i += ctas * kSortThreads) a.tickets[i] = 0;
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.bits;
        const bool last = pass + 1 == a.passes;
        SortTile t;
        uint2 total = make_uint2(0, 0);
        for (uint32_t at = begin; at < end; at += kTile) {
            load_tile<LARGE>(a, s, pass, at, min(at + kTile, end), t);
            const uint2 x = rank_tile(s, t, shift, a.bits);
            total.x += x.x;
            total.y += x.y;
            if constexpr (LARGE) __syncthreads();
        }
        if (2 * threadIdx.x < digits) s.total[threadIdx.x] = total;
        tc::cluster_sync();  // (and everyone has its entries in registers)
        uint2 all = make_uint2(0, 0), before = make_uint2(0, 0);
        if (2 * threadIdx.x < digits) {
            for (uint32_t c0 = 0; c0 < ctas; c0 += 4) {
                uint2 x[4];  // (together: a peer's memory is far)
#pragma unroll
                for (uint32_t u = 0; u < 4; ++u) x[u] = load_peer(&s.total[threadIdx.x], min(c0 + u, ctas - 1));
#pragma unroll
                for (uint32_t u = 0; u < 4; ++u) {
                    const uint32_t c = c0 + u;
                    all.x += c < ctas ? x[u].x : 0u;
                    all.y += c < ctas ? x[u].y : 0u;
                    before.x += c < rank ? x[u].x : 0u;
                    before.y += c < rank ? x[u].y : 0u;
                }
            }
        }
        const uint32_t start = before_all(all.x + all.y, s.sums);
        if (2 * threadIdx.x < digits) {
            s.base[2 * threadIdx.x] = start + before.x;
            s.base[2 * threadIdx.x + 1] = start + all.x + before.y;
        }
        for (uint32_t at = begin; at < end; at += kTile) {
            uint2 here = total;
            if constexpr (LARGE) {
                load_tile<LARGE>(a, s, pass, at, min(at + kTile, end), t);
                here = rank_tile(s, t, shift, a.bits);
            }
            const uint32_t local = before_all(here.x + here.y, s.sums);
            if (2 * threadIdx.x < digits) {
                s.local[2 * threadIdx.x] = local;
                s.local[2 * threadIdx.x + 1] = local + here.x;
            }
            __syncthreads();
            const uint16_t *count = reinterpret_cast<const uint16_t *>(s.count[threadIdx.x / 32]);
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                if (i >= t.items || t.first + 32 * i >= t.end) continue;
                const uint32_t digit = t.spot[i] >> 16;
                s.staged[s.local[digit] + count[digit] + (t.spot[i] & 0xffffu)] = make_uint2(t.key[i], t.pos[i]);
            }
            __syncthreads();
            const uint32_t entries = min(kTile, end - at);
#pragma unroll 2
            for (uint32_t i = threadIdx.x; i < entries; i += kSortThreads) {
                const uint2 e = s.staged[i];
                const uint32_t digit = (e.x >> shift) & (digits - 1), to = s.base[digit] + i - s.local[digit];
                if (LARGE || last) {
                    a.key[pass % 2][to] = e.x;
                    a.pos[pass % 2][to] = e.y;
                } else {
                    store_peer(&s.entry[to & (each - 1)], to >> each_log, e);
                }
            }
            if constexpr (LARGE) {
                __syncthreads();
                if (2 * threadIdx.x < digits) {
                    s.base[2 * threadIdx.x] += here.x;
                    s.base[2 * threadIdx.x + 1] += here.y;
                }
            }
        }
        // the next pass reads what the cluster has written, and overwrites the totals
        if constexpr (LARGE) __threadfence();
        tc::cluster_sync();
    }
}

// ---------------------------------------------------------------- few tokens: their order by counting

// Up to 4096 tokens below 2^20 (or none: key `vocab`) are sorted by all CTAs at
// once: an entry's place is the number of smaller ones, a token and its position
// in one 32-bit word, which a warp counts in shared memory. In a graph of such
// launches 1021 entries take 1.8 us (the radix sort with its waits 7.8), 4096 3.6
// (8.4).
constexpr uint32_t kPlaceBits = 12, kPlaceMost = 1u << kPlaceBits;
static_assert(kPlaceMost * sizeof(uint32_t) <= 116 << 10, "the entries fit");
constexpr int64_t kPlaceVocab = int64_t(1) << (32 - kPlaceBits);
constexpr int kPlaceThreads = 1024;
// More than half of an SM's shared memory, so that no SM gets two CTAs while the
// kernel before is still on others (4096 tokens added: 11.5 us in all, else 13.6).
constexpr int kPlaceShared = 116 << 10;

__global__ void __launch_bounds__(kPlaceThreads, 1) place_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ __align__(16) uint32_t entry[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t padded = (a.n + 127) / 128 * 128;
    wait_previous();
    allow_next();
    for (uint32_t i = blockIdx.x * kPlaceThreads + threadIdx.x; i < a.n_tickets; i += gridDim.x * kPlaceThreads)
        a.tickets[i] = 0;
    for (uint32_t i = threadIdx.x; i < padded; i += kPlaceThreads) {
        uint32_t e = 0xffffffffu;
        if (i < a.n) {
            const int64_t token = a.tokens[i];
            const bool none = token == a.ignore || token < 0 || token >= a.vocab;
            e = (none ? a.vocab : static_cast<uint32_t>(token)) << kPlaceBits | i;
        }
        entry[i] = e;
    }
    __syncthreads();
    for (uint32_t i = blockIdx.x + gridDim.x * warp; i < a.n; i += kPlaceThreads / 32 * gridDim.x) {
        const uint32_t x = entry[i];
        uint32_t below = 0;
        for (uint32_t j = 4 * lane; j < padded; j += 128) {
            const uint4 e = *reinterpret_cast<const uint4 *>(entry + j);
            below += (e.x < x) + (e.y < x) + (e.z < x) + (e.w < x);
        }
        below = __reduce_add_sync(0xffffffffu, below);
        if (lane == 0) {
            a.key[0][below] = x >> kPlaceBits;
            a.pos[0][below] = i;
        }
    }
}

// ---------------------------------------------------------------- rows that no token uses

constexpr int kThreads = 256, kWarps = kThreads / 32;
static_assert(kWarps == kSumWarps, "the host cuts the entries for as many warps");
constexpr uint32_t kAll = 0xffffffffu;
constexpr int64_t kWindow = 65536;  // rows whose use is known at a time, a bit each

__device__ __forceinline__ void zero_row(uint8_t *row, int64_t bytes, int size, int lane) {
    // up to 16-byte alignment element by element, as at the end
    int64_t head = -reinterpret_cast<intptr_t>(row) & 15;
    if (head > bytes) head = bytes;
    const int64_t words = (bytes - head) / 16, tail = head + 16 * words;
    for (int64_t b = lane * size; b < head; b += 32 * size) {
        if (size == 2)
            *reinterpret_cast<uint16_t *>(row + b) = 0;
        else
            *reinterpret_cast<uint32_t *>(row + b) = 0;
    }
    for (int64_t w = lane; w < words; w += 32) st_stream(row + head + 16 * w, make_uint4(0, 0, 0, 0));
    for (int64_t b = tail + lane * size; b < bytes; b += 32 * size) {
        if (size == 2)
            *reinterpret_cast<uint16_t *>(row + b) = 0;
        else
            *reinterpret_cast<uint32_t *>(row + b) = 0;
    }
}

// The first CTAs of the sums' grid have a stretch of the table each: they mark
// the rows that the tokens use and write zeros to the others. They need nothing
// of the sort before them on the stream and wait for it last, so they run
// beside it, and the sums beside them as soon as it has ended: zeros, then sums
// took 31 us more for 32768 tokens of 128000 x 8192 bf16.
__device__ __forceinline__ void fill_rows(const SumArgs &a, uint32_t *used) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t vocab = a.vocab, each = (vocab + a.fill_ctas - 1) / a.fill_ctas;
    const int64_t begin = min(blockIdx.x * each, vocab), end = min(begin + each, vocab);
    if (a.n == 0) wait_previous();  // (no sort: the kernel before is the caller's)
    for (int64_t row0 = begin; row0 < end; row0 += kWindow) {
        const int64_t rows = min(kWindow, end - row0);
        for (int i = threadIdx.x; i < (rows + 31) / 32; i += kThreads) used[i] = 0;
        __syncthreads();
#pragma unroll 8
        for (int64_t i = threadIdx.x; i < a.n; i += kThreads) {
            const int64_t token = a.tokens[i], at = token - row0;
            if (at < 0 || at >= rows || token == a.ignore) continue;
            const uint32_t bit = 1u << (at % 32);
            if (!(*static_cast<volatile uint32_t *>(used + at / 32) & bit)) atomicOr(used + at / 32, bit);
        }
        __syncthreads();
        for (int64_t r = warp; r < rows; r += kWarps)
            if (!(used[r / 32] >> (r % 32) & 1u))
                zero_row(a.d_weight + (row0 + r) * a.weight_bytes, a.dim * a.size, a.size, lane);
        __syncthreads();
    }
    wait_previous();
    allow_next();
}

// ---------------------------------------------------------------- sums

// Rows of a warp on their way, and rows that sums are added to: three CTAs of an
// SM have room for them.
constexpr int kSlots = 4, kThere = 3;

// A warp's slice of a row: 1 KB, in words of a lane of 16 bytes, or of one
// element where rows are not 16-byte aligned (then with up to 16 bytes more, as
// whole 16-byte granules are copied).
template <int DT, bool VEC> struct SumSlice {
    static constexpr int kSize = Dtype<DT>::kSize;
    static constexpr int kElems = VEC ? 16 / kSize : 1;           // of a word
    static constexpr int kWords = kSliceBytes / 32 / kSize / kElems;  // of a lane, at most
    static constexpr int kBytes = kSliceBytes + (VEC ? 0 : 16);
    using Sum = float[kWords][kElems];
};

// What a warp keeps in shared memory: the rows on their way, what their runs'
// sums are added to, and the sum of a run that began before its entries. The
// sum of a run that goes on after them takes the place of the rows, which have
// come by then.
template <int DT, bool VEC, bool ADD> struct WarpShared {
    using S = SumSlice<DT, VEC>;
    union {
        uint4 rows[kSlots][S::kBytes / 16];
        float tail[S::kWords][S::kElems][32];
    };
    uint4 there[ADD ? kThere : 1][S::kBytes / 16];
    float head[S::kWords][S::kElems][32];
    __device__ WarpShared() {}
};

// Copy up to 16 bytes to shared memory (zeros behind them).
__device__ __forceinline__ void copy_async(void *dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tma::smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A warp's copy of `bytes` of a row. Aligned rows: a lane copies what it will
// read. Others: the granules that hold them, from the last 16-byte boundary (the
// bytes before the first element are of the same allocation) to the last byte.
template <int DT, bool VEC> __device__ __forceinline__ void copy_row(uint4 *dst, const uint8_t *src, int bytes) {
    const int lane = threadIdx.x % 32;
    if constexpr (VEC) {
#pragma unroll
        for (int j = 0; j < SumSlice<DT, VEC>::kWords; ++j) {
            const int at = (j * 32 + lane) * 16;
            if (at < bytes) copy_async(dst + j * 32 + lane, src + at, 16);
        }
    } else {
        const int shift = reinterpret_cast<uintptr_t>(src) & 15;
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            const int at = (j * 32 + lane) * 16, left = shift + bytes - at;
            if (left > 0) copy_async(dst + j * 32 + lane, src - shift + at, left < 16 ? left : 16);
        }
    }
}

// A lane's j-th word of a copied row.
template <int DT, bool VEC> __device__ __forceinline__ void read_word(const uint4 *row, int shift, int j, float *f) {
    const int lane = threadIdx.x % 32;
    if constexpr (!VEC) {
        f[0] = Dtype<DT>::load(reinterpret_cast<const uint8_t *>(row) + shift, j * 32 + lane);
    } else if constexpr (DT == FSDP_F32) {
        const float4 x = *reinterpret_cast<const float4 *>(row + j * 32 + lane);
        f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w;
    } else {
        unpack8<DT>(row[j * 32 + lane], f);
    }
}

// A word of a row, rounded.
template <int DT, bool VEC> __device__ __forceinline__ void store_word(uint8_t *row, int col, const float *f) {
    if constexpr (!VEC)
        Dtype<DT>::store(row, col, f[0]);
    else if constexpr (DT == FSDP_F32)
        st_state(reinterpret_cast<float *>(row) + col, make_float4(f[0], f[1], f[2], f[3]));
    else
        st_stream(row + col * 2, make_uint4(pack2<DT>(f[0], f[1]), pack2<DT>(f[2], f[3]), pack2<DT>(f[4], f[5]),
                                            pack2<DT>(f[6], f[7])));
}

template <int N> __device__ __forceinline__ void store_floats(float *p, const float *f) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 4)
            *reinterpret_cast<float4 *>(p + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) p[e] = f[e];
    }
}
template <int N> __device__ __forceinline__ void add_floats(const float *p, float *f) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(p + e));
            f[e] += x.x, f[e + 1] += x.y, f[e + 2] += x.z, f[e + 3] += x.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] += __ldcg(p + e);
    }
}

// How many blocks the run of block b's first entry goes back over (its last
// one: on after), beside the next one. A warp looks at 32 blocks at a time.
__device__ __forceinline__ uint32_t more_blocks(const SumArgs &a, uint32_t b, uint32_t key, bool back) {
    const int lane = threadIdx.x % 32;
    uint32_t more = 0;
    for (;;) {
        // the last entry of the block before, the first one of the block after
        const int64_t at = back ? (int64_t(b) - 1 - more - lane) * a.block - 1 : (int64_t(b) + 2 + more + lane) * a.block;
        const uint32_t same = __ballot_sync(kAll, at >= 0 && at < a.n && a.key[at] == key);
        if (same != kAll) return more + __ffs(~same) - 1;
        more += 32;
    }
}

// The columns of a CTA's slice.
struct Columns {
    int64_t first;
    int count, words;  // words of a lane (the same for all slices)
};

// Sum of the parts of a run in the blocks first, first + step, ... before
// `end`. A run's part is the second one in the block it begins in, else the
// first.
template <int DT, bool VEC>
__device__ __forceinline__ void add_parts(const SumArgs &a, const Columns &c, uint32_t from, uint32_t first, uint32_t end,
                                          uint32_t step, typename SumSlice<DT, VEC>::Sum &sum) {
    using S = SumSlice<DT, VEC>;
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int j = 0; j < S::kWords; ++j)
#pragma unroll
        for (int e = 0; e < S::kElems; ++e) sum[j][e] = 0.0f;
#pragma unroll 4
    for (uint32_t i = first; i < end; i += step) {
        const float *part = a.part + (int64_t(i) * 2 + (i == from ? 1 : 0)) * a.ld_part + c.first;
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            const int col = (j * 32 + lane) * S::kElems;
            if (col < c.count) add_floats<S::kElems>(part + col, sum[j]);
        }
    }
}

// This run's part of block b, of its blocks from .. to, to memory; true, with
// the whole run's sum, for the warp that brings the last one. A run over many
// blocks is added up in two steps, by the last warps of a few groups and then
// by the last of those: one warp took 20 us for the parts of 102 blocks.
template <int DT, bool VEC>
__device__ __forceinline__ bool join_parts(const SumArgs &a, uint32_t b, uint32_t slice, const Columns &c, uint32_t from,
                                           uint32_t to, typename SumSlice<DT, VEC>::Sum &sum) {
    using S = SumSlice<DT, VEC>;
    const int lane = threadIdx.x % 32;
    const uint32_t blocks = to - from + 1;
    uint32_t group = 16;
    while (group * group < blocks) group *= 2;
    uint32_t first = b - (b - from) % group, end = min(first + group, to + 1), step = 1, at = b;
    // (a block may have a run's later group and another run's first one)
    uint32_t *ticket = a.tickets + ((first == from ? 0 : 2 * uint64_t(a.blocks)) + first) * a.slices + slice;
#pragma unroll 1
    for (;;) {
        float *mine = a.part + (int64_t(at) * 2 + (at == from ? 1 : 0)) * a.ld_part + c.first;
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            const int col = (j * 32 + lane) * S::kElems;
            if (col < c.count) store_floats<S::kElems>(mine + col, sum[j]);
        }
        __threadfence();
        __syncwarp();
        uint32_t there = 0;
        if (lane == 0) there = atomicAdd(ticket, 1u) + 1;
        if (__shfl_sync(kAll, there, 0) != (end - first + step - 1) / step) return false;
        __threadfence();
        add_parts<DT, VEC>(a, c, from, first, end, step, sum);
        if (step > 1 || blocks <= group) return true;
        // the group's sum, in its first part's place
        at = first;
        first = from;
        end = to + 1;
        step = group;
        ticket = a.tickets + (uint64_t(a.blocks) + from) * a.slices + slice;
    }
}

// A block of sorted entries, for one slice of the columns; each warp has 4 to 16
// of the entries. It adds up their rows as they come (four are on their way, in
// shared memory: 32 warps of an SM have 128 KB in flight) and writes the runs
// that lie within its entries. The parts of a run that warps share meet in
// shared memory, where the warp that the run begins in (the first one, for a
// run from before the block) adds them up in order. A run that crosses the
// block's first or last entry leaves its part in memory; the warp that brings
// the last part of it adds them up, again in order.
template <int DT, bool VEC, bool ADD>
__global__ void __launch_bounds__(kThreads, ADD ? 3 : 4) sum_kernel(const __grid_constant__ SumArgs a) {
    using S = SumSlice<DT, VEC>;
    using Shared = WarpShared<DT, VEC, ADD>;
    extern __shared__ __align__(16) uint8_t raw[];
    Shared *shared = reinterpret_cast<Shared *>(raw);
    __shared__ bool through[kWarps];    // a run from before the warp's entries goes on after them
    __shared__ uint32_t back, ahead;    // blocks that runs from before and after the block go over, beside the next one
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, each = a.block / kWarps;
    if constexpr (!ADD) {
        static_assert(kWarps * sizeof(Shared) >= kWindow / 8, "a bit for each row of a window");
        if (blockIdx.x < a.fill_ctas) {
            fill_rows(a, reinterpret_cast<uint32_t *>(raw));
            return;
        }
    }
    const uint32_t cta = blockIdx.x - a.fill_ctas, slice = cta % a.slices, b = cta / a.slices;
    Columns c;
    c.words = a.words;
    c.first = int64_t(slice) * 32 * c.words * S::kElems;
    c.count = static_cast<int>(min(int64_t(32 * c.words * S::kElems), a.dim - c.first));
    const int64_t first_byte = c.first * S::kSize;
    Shared &mine = shared[warp];
    wait_previous();
    allow_next();
    // the warp's entries in its lanes, and the ones before and after them
    const uint32_t lo = b * a.block + warp * each;  // (below 2^30 + 128)
    const uint32_t key = lane <= each && lo + lane < a.n ? a.key[lo + lane] : a.vocab;
    const uint32_t pos = lane < each && lo + lane < a.n ? a.pos[lo + lane] : 0u;
    const uint32_t before = lo > 0 && lo <= a.n ? a.key[lo - 1] : a.vocab;
    const int count = __popc(__ballot_sync(kAll, lane < each && key < a.vocab));  // (what is no token comes last)
    const uint32_t next = __shfl_down_sync(kAll, key, 1);
    const uint32_t ends = __ballot_sync(kAll, lane < count && next != key);  // an entry that is its run's last
    const bool open = count > 0 && before == __shfl_sync(kAll, key, 0);
    const bool goes_on = count > 0 && !(ends >> (count - 1) & 1u);  // (then count == each)
    if (lane == 0) through[warp] = open && ends == 0;
    auto row_of = [&](int i) { return a.d_out + int64_t(__shfl_sync(kAll, pos, i)) * a.out_bytes + first_byte; };
    auto to_of = [&](int i) { return a.d_weight + int64_t(__shfl_sync(kAll, key, i)) * a.weight_bytes + first_byte; };
    auto shift_of = [](const uint8_t *p) { return VEC ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15); };
    // row i to its slot, and the row that the run's sum of the entry before is added to
    auto issue = [&](int i) {
        if (i < count) copy_row<DT, VEC>(mine.rows[i % kSlots], row_of(i), c.count * S::kSize);
        if constexpr (ADD) {
            if (i > 0 && i <= count && (ends >> (i - 1) & 1u))
                copy_row<DT, VEC>(mine.there[(i - 1) % kThere], to_of(i - 1), c.count * S::kSize);
        }
        copy_commit();
    };
#pragma unroll
    for (int i = 0; i < kSlots; ++i) issue(i);
    // (while the rows are on their way)
    if (warp == 0 && open) {
        const uint32_t n = more_blocks(a, b, __shfl_sync(kAll, key, 0), true);
        if (lane == 0) back = n;
    }
    if (warp == kWarps - 1 && goes_on) {
        const uint32_t n = more_blocks(a, b, __shfl_sync(kAll, key, each), false);
        if (lane == 0) ahead = n;
    }
    typename S::Sum sum;
    auto clear = [&] {
#pragma unroll
        for (int j = 0; j < S::kWords; ++j)
#pragma unroll
            for (int e = 0; e < S::kElems; ++e) sum[j][e] = 0.0f;
    };
    // a lane's columns of a row's sum to the gradient: times scale, and (ADD) added
    // to what is there
    auto write_row = [&](uint8_t *to, const uint4 *there) {
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            const int col = (j * 32 + lane) * S::kElems;
            if (col >= c.count) continue;
            float f[S::kElems];
            if constexpr (ADD) read_word<DT, VEC>(there, shift_of(to), j, f);
#pragma unroll
            for (int e = 0; e < S::kElems; ++e) f[e] = ADD ? fmaf(sum[j][e], a.scale, f[e]) : sum[j][e] * a.scale;
            store_word<DT, VEC>(to, col, f);
        }
    };
    auto add_there = [&](const uint8_t *to) {  // (a row that nothing has been copied of)
        if constexpr (ADD) {
            __syncwarp();
            copy_row<DT, VEC>(mine.there[0], to, c.count * S::kSize);
            copy_commit();
            copy_wait<0>();
            __syncwarp();
        }
    };
    clear();
    bool first = true;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        if (ADD && (ends >> i & 1u))
            copy_wait<kSlots - 2>();
        else
            copy_wait<kSlots - 1>();
        if constexpr (!VEC) __syncwarp();  // (other lanes' granules)
        const int shift = VEC ? 0 : shift_of(row_of(i));
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            if (j >= c.words) break;
            float f[S::kElems];
            read_word<DT, VEC>(mine.rows[i % kSlots], shift, j, f);
#pragma unroll
            for (int e = 0; e < S::kElems; ++e) sum[j][e] += f[e];
        }
        if (ends >> i & 1u) {
            if (first && open) {
#pragma unroll
                for (int j = 0; j < S::kWords; ++j)
#pragma unroll
                    for (int e = 0; e < S::kElems; ++e) mine.head[j][e][lane] = sum[j][e];
            } else {
                write_row(to_of(i), mine.there[ADD ? i % kThere : 0]);
            }
            first = false;
            clear();
        }
        if constexpr (!VEC) __syncwarp();
        issue(i + kSlots);
    }
    __syncwarp();  // (all lanes' rows have come and been read)
    if (goes_on) {
#pragma unroll
        for (int j = 0; j < S::kWords; ++j)
#pragma unroll
            for (int e = 0; e < S::kElems; ++e) {
                if (first && open)
                    mine.head[j][e][lane] = sum[j][e];
                else
                    mine.tail[j][e][lane] = sum[j][e];
            }
    }
    __syncthreads();
    // the runs that the warps share, or that cross the block's ends: those this
    // warp has the first part of
    const bool from_before = warp == 0 && open, begins = goes_on && !(first && open);
#pragma unroll 1
    for (int which = from_before ? 0 : 1; which < (begins ? 2 : 1); ++which) {
#pragma unroll
        for (int j = 0; j < S::kWords; ++j)
#pragma unroll
            for (int e = 0; e < S::kElems; ++e) sum[j][e] = which == 0 ? mine.head[j][e][lane] : mine.tail[j][e][lane];
        bool goes = which == 1 || through[0];
#pragma unroll 1
        for (int other = warp + 1; goes && other < kWarps; ++other) {
#pragma unroll
            for (int j = 0; j < S::kWords; ++j)
#pragma unroll
                for (int e = 0; e < S::kElems; ++e) sum[j][e] += shared[other].head[j][e][lane];
            goes = through[other];
        }
        const int entry = which == 0 ? 0 : each - 1;
        if (which == 0 || goes) {
            const uint32_t from = which == 0 ? b - 1 - back : b, to = goes ? b + 1 + ahead : b;
            if (!join_parts<DT, VEC>(a, b, slice, c, from, to, sum)) continue;
        }
        add_there(to_of(entry));
        write_row(to_of(entry), mine.there[0]);
    }
}

template <int DT, bool VEC, bool ADD> fsdp_status launch_type(const SumArgs &a, cudaStream_t s) {
    constexpr size_t kShared = kWarps * sizeof(WarpShared<DT, VEC, ADD>);
    static PerDeviceOnce once;
    const int dev = current_device();
    if (!once.is_done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(sum_kernel<DT, VEC, ADD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kShared));
        if (e != cudaSuccess) return cuda_status(e);
        once.mark(dev);
    }
    // (the blocks times the slices are below 2^31: a workspace of that many tickets)
    return launch_chained(sum_kernel<DT, VEC, ADD>, a.fill_ctas + a.blocks * a.slices, kThreads, kShared, s, a);
}

template <int DT> fsdp_status launch_form(const SumArgs &a, bool vec, bool add, cudaStream_t s) {
    if (vec) return add ? launch_type<DT, true, true>(a, s) : launch_type<DT, true, false>(a, s);
    return add ? launch_type<DT, false, true>(a, s) : launch_type<DT, false, false>(a, s);
}

template <bool LARGE> fsdp_status launch_sort_kernel(const SortArgs &a, unsigned ctas, cudaStream_t s) {
    static PerDeviceOnce once;
    const int dev = current_device();
    if (!once.is_done(dev)) {
        cudaError_t e = cudaFuncSetAttribute(sort_kernel<LARGE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(sizeof(SortShared)));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(sort_kernel<LARGE>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_status(e);
        once.mark(dev);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(ctas);
    config.blockDim = dim3(kSortThreads);
    config.dynamicSmemBytes = sizeof(SortShared);
    config.stream = s;
    config.attrs = attr;
    config.numAttrs = 2;
    return cuda_status(cudaLaunchKernelEx(&config, sort_kernel<LARGE>, a));
}

}  // namespace

fsdp_status launch_sort(const SortArgs &a, cudaStream_t s) {
    // two entries a thread up to eight CTAs; sixteen where those do not hold them
    unsigned ctas = 1;
    while (ctas < 8 && ctas * 2 * kSortThreads < a.n) ctas *= 2;
    if (a.n > ctas * kTile) ctas = kMostCtas;
    return a.n > kMostCtas * kTile ? launch_sort_kernel<true>(a, ctas, s) : launch_sort_kernel<false>(a, ctas, s);
}

bool can_place(int64_t n, int64_t vocab) { return n > 0 && n <= kPlaceMost && vocab < kPlaceVocab; }

fsdp_status launch_place(const SortArgs &a, cudaStream_t s) {
    static PerDeviceOnce once;
    const int dev = current_device();
    if (!once.is_done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlaceShared);
        if (e != cudaSuccess) return cuda_status(e);
        once.mark(dev);
    }
    const uint32_t sms = sm_count() > 0 ? sm_count() : 1;
    return launch_chained(place_kernel, a.n < sms ? a.n : sms, kPlaceThreads, kPlaceShared, s, a);
}

fsdp_status launch_sums(const SumArgs &a, int dtype, bool vec, bool add, cudaStream_t s) {
    switch (dtype) {
        case FSDP_BF16: return launch_form<FSDP_BF16>(a, vec, add, s);
        case FSDP_F16: return launch_form<FSDP_F16>(a, vec, add, s);
        default: return launch_form<FSDP_F32>(a, vec, add, s);
    }
}

}  // namespace embed
}  // namespace fsdp
