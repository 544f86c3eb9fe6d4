// embed_grad.cu -- the gradient of the token embedding:
//
//   dW[v] = scale * (sum of dY[t] over the tokens t that are v, in their order)
//
// written to the whole table, or added to the rows in use.
//
// The tokens are sorted first (one launch: a cluster of up to eight CTAs, a
// stable radix sort), so that a row's summands lie side by side and add up in
// one fixed order: the same bits every time, whatever order the warps run in.
// Rows that no token uses are filled with zeros beside the sort, which keeps
// only a few SMs busy. Then a CTA adds up 32 to 128 sorted entries for a slice
// of the columns; what begins and ends within them is written at once, a run
// that crosses to other CTAs' entries leaves fp32 parts, which the last of
// them adds in order.
//
// Bound by HBM: dY is read once, the table written once. 32768 tokens of a
// 128000 x 8192 bf16 table: 439 us, 5.9 TB/s (zeros 300, sums 131).
#include "embed.cuh"
#include "tcgen.cuh"

namespace fsdp {
namespace embed {
namespace {

// ---------------------------------------------------------------- sort

// 512 threads of at most 64 registers: beside a CTA of the fill kernel, an SM
// holds one of these.
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32, kItems = 8;
constexpr uint32_t kTile = kSortThreads * kItems;  // entries of a CTA in one go
constexpr int kMostCtas = 8;                       // of the cluster (the portable limit)
constexpr uint32_t kDigits = 1u << kMostBits;
static_assert(kDigits <= 2 * kSortThreads && kTile < 65536, "a thread has two digits; counts of a tile fit 16 bits");

struct SortShared {
    uint32_t count[kSortWarps][kDigits / 2];  // of two digits: entries of a warp; then those of the warps before it
    uint2 total[kDigits / 2];                 // of two digits over the CTA (its peers read them)
    uint32_t base[kDigits];                   // where its next entry with a digit goes
    uint32_t sums[kSortWarps];
    uint2 entry[kTile];                       // {key, position} between passes, of few entries
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
__device__ __forceinline__ uint2 rank_tile(SortShared &s, SortTile &t, int shift, uint32_t digits) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint16_t *count = reinterpret_cast<uint16_t *>(s.count[warp]);
    for (uint32_t d = lane; d < (digits + 1) / 2; d += 32) s.count[warp][d] = 0;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (i >= t.items) break;  // (the same for all)
        const bool live = t.first + 32 * i < t.end;
        const uint32_t digit = live ? (t.key[i] >> shift) & (digits - 1) : 0xffffu;
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
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
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t x = s.count[w][threadIdx.x];
            s.count[w][threadIdx.x] = sum;
            sum += x;
        }
    }
    return make_uint2(sum & 0xffffu, sum >> 16);
}

// A stable radix sort by digits of up to 10 bits. Each CTA has a stretch of the
// entries; the CTAs' counts of every digit tell where its entries go. Entries
// that are no token have the key `vocab` and come last. Up to eight tiles of
// entries stay in the cluster's shared memory until the last pass. Bound by
// latency (two passes: 1021 tokens 8 us, 8192 11, 32768 22; through memory and
// with 1024 threads 14, 16 and 28).
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
            const uint2 x = rank_tile(s, t, shift, digits);
            total.x += x.x;
            total.y += x.y;
            if constexpr (LARGE) __syncthreads();
        }
        if (2 * threadIdx.x < digits) s.total[threadIdx.x] = total;
        tc::cluster_sync();  // (and everyone has its entries in registers)
        uint2 all = make_uint2(0, 0), before = make_uint2(0, 0);
        if (2 * threadIdx.x < digits) {
#pragma unroll
            for (uint32_t c = 0; c < kMostCtas; ++c) {
                if (c >= ctas) break;
                const uint2 x = load_peer(&s.total[threadIdx.x], c);
                all.x += x.x;
                all.y += x.y;
                before.x += c < rank ? x.x : 0u;
                before.y += c < rank ? x.y : 0u;
            }
        }
        const uint32_t start = before_all(all.x + all.y, s.sums);
        if (2 * threadIdx.x < digits) {
            s.base[2 * threadIdx.x] = start + before.x;
            s.base[2 * threadIdx.x + 1] = start + all.x + before.y;
        }
        __syncthreads();
        for (uint32_t at = begin; at < end; at += kTile) {
            uint2 here = make_uint2(0, 0);
            if constexpr (LARGE) {
                load_tile<LARGE>(a, s, pass, at, min(at + kTile, end), t);
                here = rank_tile(s, t, shift, digits);
                __syncthreads();
            }
            const uint16_t *count = reinterpret_cast<const uint16_t *>(s.count[threadIdx.x / 32]);
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                if (i >= t.items || t.first + 32 * i >= t.end) continue;
                const uint32_t digit = t.spot[i] >> 16;
                const uint32_t to = s.base[digit] + count[digit] + (t.spot[i] & 0xffffu);
                if (LARGE || last) {
                    a.key[pass % 2][to] = t.key[i];
                    a.pos[pass % 2][to] = t.pos[i];
                } else {
                    store_peer(&s.entry[to & (each - 1)], to >> each_log, make_uint2(t.key[i], t.pos[i]));
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

// ---------------------------------------------------------------- rows that no token uses

constexpr int kFillThreads = 1024;
constexpr int64_t kWindow = 16384;  // rows whose use is known at a time
// More than half of an SM's shared memory, and less than the sort leaves: an SM
// has room for one CTA of this kernel, beside the sort's or not. (Two on one
// took twice as long: 32768 tokens, 128000 x 8192 bf16, 600 us in all against 490.)
constexpr int kFillShared = 120 << 10;

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

// A CTA per SM, each with a stretch of the table: it marks the rows that the
// tokens use and writes zeros to the others. Follows the sort on the stream but
// needs nothing of it, so it waits for it last: when this kernel has ended, the
// sort has too.
__global__ void __launch_bounds__(kFillThreads, 2) fill_kernel(const __grid_constant__ FillArgs a) {
    __shared__ uint32_t used[kWindow / 32];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t each = (a.vocab + gridDim.x - 1) / gridDim.x;
    const int64_t begin = blockIdx.x * each, end = min(begin + each, a.vocab);
    if (a.n == 0) wait_previous();  // (no sort: the kernel before is the caller's)
    for (int64_t row0 = begin; row0 < end; row0 += kWindow) {
        const int64_t rows = min(kWindow, end - row0);
        for (int i = threadIdx.x; i < kWindow / 32; i += kFillThreads) used[i] = 0;
        __syncthreads();
#pragma unroll 8
        for (int64_t i = threadIdx.x; i < a.n; i += kFillThreads) {
            const int64_t token = a.tokens[i], at = token - row0;
            if (at < 0 || at >= rows || token == a.ignore) continue;
            const uint32_t bit = 1u << (at % 32);
            if (!(*static_cast<volatile uint32_t *>(&used[at / 32]) & bit)) atomicOr(&used[at / 32], bit);
        }
        __syncthreads();
        for (int64_t r = warp; r < rows; r += kFillThreads / 32)
            if (!(used[r / 32] >> (r % 32) & 1u))
                zero_row(a.d_weight + (row0 + r) * a.row_bytes, a.dim * a.size, a.size, lane);
        __syncthreads();
    }
    wait_previous();
    allow_next();
}

// ---------------------------------------------------------------- sums

constexpr int kThreads = 256, kWarps = kThreads / 32;
static_assert(kWarps == kSumWarps, "the host cuts the entries for as many warps");
constexpr int kSlots = 4;  // rows of a warp on their way
constexpr uint32_t kAll = 0xffffffffu;

// What a warp keeps in shared memory: the rows on their way, and the sum of a
// run that began before its entries. The sum of a run that goes on after them
// takes the place of the rows, which have come by then.
template <int DT, bool VEC> struct WarpShared {
    using S = Slice<DT, VEC, kSumWords>;
    union {
        Word<DT, VEC> rows[kSlots][S::kWords][32];
        float tail[S::kWords][S::kElems][32];
    };
    float head[S::kWords][S::kElems][32];
    __device__ WarpShared() {}
};

// A lane's columns of one row's sum to the gradient: times scale, and added to
// what is there.
template <int DT, bool VEC>
__device__ __forceinline__ void write_row(const SumArgs &a, uint32_t key, int64_t col0,
                                          float (&sum)[Slice<DT, VEC, kSumWords>::kWords]
                                                      [Slice<DT, VEC, kSumWords>::kElems]) {
    using S = Slice<DT, VEC, kSumWords>;
    uint8_t *row = a.d_weight + int64_t(key) * a.weight_bytes;
    if (a.accumulate) {
        Word<DT, VEC> there[S::kWords];
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            const int64_t col = col0 + j * 32 * S::kElems;
            if (col < a.dim) there[j].load_coherent(row, col);
        }
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            const int64_t col = col0 + j * 32 * S::kElems;
            if (col >= a.dim) continue;
            float f[S::kElems];
            there[j].widen(f);
#pragma unroll
            for (int e = 0; e < S::kElems; ++e) f[e] = fmaf(sum[j][e], a.scale, f[e]);
            Word<DT, VEC>::store(row, col, f);
        }
    } else {
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            const int64_t col = col0 + j * 32 * S::kElems;
            if (col >= a.dim) continue;
            float f[S::kElems];
#pragma unroll
            for (int e = 0; e < S::kElems; ++e) f[e] = sum[j][e] * a.scale;
            Word<DT, VEC>::store(row, col, f);
        }
    }
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

__device__ __forceinline__ uint32_t key_at(const SumArgs &a, int64_t at) { return a.key[at]; }

// The block that a run which block b's first entry continues begins in.
__device__ __forceinline__ uint32_t first_block(const SumArgs &a, uint32_t b, uint32_t key) {
    uint32_t hi = b - 1;  // (its last entry is of the run)
    if (hi == 0 || key_at(a, int64_t(hi) * a.block - 1) != key) return hi;
    uint32_t lo = 0;
    --hi;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (key_at(a, (int64_t(mid) + 1) * a.block - 1) == key)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// The last block that begins with a run which goes on after block b.
__device__ __forceinline__ uint32_t last_block(const SumArgs &a, uint32_t b, uint32_t key) {
    uint32_t lo = b + 1, hi = a.blocks - 1;
    if (lo == hi || key_at(a, (int64_t(lo) + 1) * a.block) != key) return lo;
    ++lo;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo + 1) / 2;
        if (key_at(a, int64_t(mid) * a.block) == key)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// This run's part of block b to memory; true, with the whole run's sum, for
// the warp that brings its last part.
template <int DT, bool VEC>
__device__ __forceinline__ bool join_parts(const SumArgs &a, uint32_t b, uint32_t slice, int64_t col0, uint32_t key, bool head,
                                           bool tail,
                                           float (&sum)[Slice<DT, VEC, kSumWords>::kWords]
                                                       [Slice<DT, VEC, kSumWords>::kElems]) {
    using S = Slice<DT, VEC, kSumWords>;
    float *mine = a.part + (int64_t(b) * 2 + (head ? 0 : 1)) * a.ld_part;
#pragma unroll
    for (int j = 0; j < S::kWords; ++j) {
        const int64_t col = col0 + j * 32 * S::kElems;
        if (col < a.dim) store_floats<S::kElems>(mine + col, sum[j]);
    }
    const uint32_t from = head ? first_block(a, b, key) : b, to = tail ? last_block(a, b, key) : b;
    __threadfence();
    __syncwarp();
    uint32_t there = 0;
    if (threadIdx.x % 32 == 0) there = atomicAdd(a.tickets + uint64_t(from) * a.slices + slice, 1u);
    if (__shfl_sync(kAll, there, 0) != to - from) return false;
    __threadfence();
#pragma unroll
    for (int j = 0; j < S::kWords; ++j)
#pragma unroll
        for (int e = 0; e < S::kElems; ++e) sum[j][e] = 0.0f;
#pragma unroll 4
    for (uint32_t i = from; i <= to; ++i) {
        const float *part = a.part + (int64_t(i) * 2 + (i == from ? 1 : 0)) * a.ld_part;
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            const int64_t col = col0 + j * 32 * S::kElems;
            if (col < a.dim) add_floats<S::kElems>(part + col, sum[j]);
        }
    }
    return true;
}

// Copy 16 bytes of a row to shared memory, for the thread that asks alone.
__device__ __forceinline__ void copy_async(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tma::smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A block of sorted entries, for one slice of the columns; each warp has 4 to 16
// of the entries. It adds up their rows as they come (four are on their way, in
// shared memory: 32 warps of an SM have 128 KB in flight) and writes the runs
// that lie within its entries. The parts of a run that warps share meet in
// shared memory, where the warp that the run begins in (the first one, for a
// run from before the block) adds them up in order. A run that crosses the
// block's first or last entry leaves its part in memory; the warp that brings
// the last part of it adds them up, again in order.
template <int DT, bool VEC> __global__ void __launch_bounds__(kThreads, VEC ? 4 : 3) sum_kernel(const __grid_constant__ SumArgs a) {
    using S = Slice<DT, VEC, kSumWords>;
    extern __shared__ __align__(16) uint8_t raw[];
    WarpShared<DT, VEC> *shared = reinterpret_cast<WarpShared<DT, VEC> *>(raw);
    __shared__ bool opens[kWarps], through[kWarps];  // began before the warp's entries; and goes on after them
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, each = a.block / kWarps;
    const uint32_t slice = blockIdx.x % a.slices, b = blockIdx.x / a.slices;
    const int64_t col0 = int64_t(slice) * S::kCols + lane * S::kElems;
    WarpShared<DT, VEC> &mine = shared[warp];
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
    if (lane == 0) {
        opens[warp] = open;
        through[warp] = open && ends == 0;
    }
    auto issue = [&](int i) {  // row i to its slot
        if (i < count) {
            const uint8_t *row = a.d_out + int64_t(__shfl_sync(kAll, pos, i)) * a.out_bytes;
#pragma unroll
            for (int j = 0; j < S::kWords; ++j) {
                const int64_t col = col0 + j * 32 * S::kElems;
                if (col < a.dim) copy_async(&mine.rows[i % kSlots][j][lane], row + col * S::kSize);
            }
        }
        copy_commit();
    };
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < kSlots; ++i) issue(i);
    }
    float sum[S::kWords][S::kElems];
    bool fresh = true, first = true;
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
        if constexpr (VEC) {
            copy_wait<kSlots - 1>();
        } else if (i % kSlots == 0) {  // elements of any alignment: four rows at once
            Word<DT, VEC> w[kSlots][S::kWords];
#pragma unroll
            for (int u = 0; u < kSlots; ++u) {
                const uint8_t *row = a.d_out + int64_t(__shfl_sync(kAll, pos, min(i + u, count - 1))) * a.out_bytes;
#pragma unroll
                for (int j = 0; j < S::kWords; ++j) {
                    const int64_t col = col0 + j * 32 * S::kElems;
                    if (col < a.dim) w[u][j].load(row, col);
                }
            }
#pragma unroll
            for (int u = 0; u < kSlots; ++u)
#pragma unroll
                for (int j = 0; j < S::kWords; ++j) mine.rows[u][j][lane] = w[u][j];
        }
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            float f[S::kElems];
            mine.rows[i % kSlots][j][lane].widen(f);
#pragma unroll
            for (int e = 0; e < S::kElems; ++e) sum[j][e] = fresh ? f[e] : sum[j][e] + f[e];
        }
        if constexpr (VEC) issue(i + kSlots);
        fresh = ends >> i & 1u;
        if (!fresh) continue;
        if (first && open) {
#pragma unroll
            for (int j = 0; j < S::kWords; ++j)
#pragma unroll
                for (int e = 0; e < S::kElems; ++e) mine.head[j][e][lane] = sum[j][e];
        } else {
            write_row<DT, VEC>(a, __shfl_sync(kAll, key, i), col0, sum);
        }
        first = false;
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
        const uint32_t k = __shfl_sync(kAll, key, which == 0 ? 0 : each - 1);
        if ((which == 0 || goes) && !join_parts<DT, VEC>(a, b, slice, col0, k, which == 0, goes, sum)) continue;
        write_row<DT, VEC>(a, k, col0, sum);
    }
}

template <int DT, bool VEC> fsdp_status launch_type(const SumArgs &a, cudaStream_t s) {
    constexpr size_t kShared = kWarps * sizeof(WarpShared<DT, VEC>);
    static PerDeviceOnce once;
    const int dev = current_device();
    if (!once.is_done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(sum_kernel<DT, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kShared));
        if (e != cudaSuccess) return cuda_status(e);
        once.mark(dev);
    }
    // (the blocks times the slices are below 2^31: a workspace of that many tickets)
    return launch_chained(sum_kernel<DT, VEC>, a.blocks * a.slices, kThreads, kShared, s, a);
}

template <bool LARGE> fsdp_status launch_sort_kernel(const SortArgs &a, unsigned ctas, cudaStream_t s) {
    static PerDeviceOnce once;
    const int dev = current_device();
    if (!once.is_done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(sort_kernel<LARGE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(sizeof(SortShared)));
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
    // two entries a thread up to eight CTAs
    unsigned ctas = 1;
    while (ctas < kMostCtas && ctas * 2 * kSortThreads < a.n) ctas *= 2;
    return a.n > kMostCtas * kTile ? launch_sort_kernel<true>(a, ctas, s) : launch_sort_kernel<false>(a, ctas, s);
}

fsdp_status launch_fill(const FillArgs &a, cudaStream_t s) {
    const int64_t sms = sm_count() > 0 ? sm_count() : 1, most = (a.vocab + 31) / 32;
    static PerDeviceOnce once;
    const int dev = current_device();
    if (!once.is_done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(fill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFillShared);
        if (e != cudaSuccess) return cuda_status(e);
        once.mark(dev);
    }
    return launch_chained(fill_kernel, static_cast<unsigned>(sms < most ? sms : most), kFillThreads, kFillShared, s, a);
}

fsdp_status launch_sums(const SumArgs &a, int dtype, bool vec, cudaStream_t s) {
    switch (dtype) {
        case FSDP_BF16: return vec ? launch_type<FSDP_BF16, true>(a, s) : launch_type<FSDP_BF16, false>(a, s);
        case FSDP_F16: return vec ? launch_type<FSDP_F16, true>(a, s) : launch_type<FSDP_F16, false>(a, s);
        default: return vec ? launch_type<FSDP_F32, true>(a, s) : launch_type<FSDP_F32, false>(a, s);
    }
}

}  // namespace embed
}  // namespace fsdp
