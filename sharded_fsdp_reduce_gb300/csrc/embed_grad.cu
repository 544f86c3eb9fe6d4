// embed_grad.cu -- the gradient of the token embedding:
//
//   dW[v] = scale * (sum of dY[t] over the tokens t that are v, in their order)
//
// written to the whole table, or added to the rows in use.
//
// The tokens are sorted first (one launch: a cluster of up to eight CTAs, a
// stable radix sort), so that a row's summands lie side by side and add up in
// registers in one fixed order: the same bits every time, no atomics. A warp
// adds up 8 to 32 sorted entries for 2 KB of a row. What begins or ends within
// them is written at once; a run that crosses to other warps' entries leaves
// fp32 parts, which the join kernel adds in order. Rows that no token uses are
// filled with zeros beside the sort, which keeps only a few SMs busy.
//
// Bound by HBM: dY is read once, the table written once.
#include "embed.cuh"
#include "tcgen.cuh"

namespace fsdp {
namespace embed {
namespace {

// ---------------------------------------------------------------- sort

constexpr int kSortThreads = 1024, kSortWarps = 32, kItems = 16;
constexpr uint32_t kTile = kSortThreads * kItems;  // entries of a CTA in one go
constexpr int kMostCtas = 8;                       // of the cluster (the portable limit)

struct SortShared {
    uint16_t count[kSortWarps][1 << kMostBits];  // entries of a warp with a digit; then those of the warps before it
    uint32_t total[1 << kMostBits];              // of the CTA (its peers read them)
    uint32_t base[1 << kMostBits];               // where its next entry with a digit goes
    uint32_t sums[kSortWarps];
};

__device__ __forceinline__ uint32_t load_peer(const uint32_t *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(tc::peer_addr(tma::smem_addr(p), rank)) : "memory");
    return v;
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
    if (warp == 0) {
        uint32_t all = sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, all, o);
            if (lane >= o) all += y;
        }
        sums[lane] = all;
    }
    __syncthreads();
    return sum - x + (warp > 0 ? sums[warp - 1] : 0u);
}

// One tile's entries in registers: a warp holds 32 * items consecutive ones.
struct SortTile {
    uint32_t key[kItems];
    uint32_t spot[kItems];  // digit << 16 | place among the warp's entries with that digit
    int items;
    uint32_t first;  // this lane's first entry (the next ones are 32 apart)
    uint32_t end;
};

__device__ __forceinline__ void load_tile(const SortArgs &a, int pass, uint32_t begin, uint32_t end, SortTile &t) {
    t.items = static_cast<int>((end - begin + kSortThreads - 1) / kSortThreads);
    t.first = begin + threadIdx.x / 32 * 32 * t.items + threadIdx.x % 32;
    t.end = end;
    const uint32_t *from = a.key[(pass + 1) % 2];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t at = t.first + 32 * i;
        if (i >= t.items || at >= end) continue;
        if (pass == 0) {
            const int64_t token = a.tokens[at];
            const bool none = token == a.ignore || token < 0 || token >= a.vocab;
            t.key[i] = none ? a.vocab : static_cast<uint32_t>(token);
        } else {
            t.key[i] = __ldcg(from + at);
        }
    }
}

// Every entry's digit and its place among the warp's; then, per digit, the
// warps' counts become what comes before them. Returns the count of the digit
// threadIdx.x over the tile.
__device__ __forceinline__ uint32_t rank_tile(SortShared &s, SortTile &t, int shift, uint32_t digits) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    for (uint32_t d = lane; d < digits; d += 32) s.count[warp][d] = 0;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (i >= t.items) break;  // (the same for all)
        const bool live = t.first + 32 * i < t.end;
        const uint32_t digit = live ? (t.key[i] >> shift) & (digits - 1) : 0xffffu;
        const uint32_t peers = __match_any_sync(0xffffffffu, digit);
        uint32_t before = 0;
        if (live) before = s.count[warp][digit];
        __syncwarp();
        if (live && lane == __ffs(peers) - 1) s.count[warp][digit] = static_cast<uint16_t>(before + __popc(peers));
        __syncwarp();
        t.spot[i] = digit << 16 | (before + __popc(peers & ((1u << lane) - 1)));
    }
    __syncthreads();
    uint32_t sum = 0;
    if (threadIdx.x < digits) {
#pragma unroll 8
        for (int w = 0; w < kSortWarps; ++w) {
            const uint32_t x = s.count[w][threadIdx.x];
            s.count[w][threadIdx.x] = static_cast<uint16_t>(sum);
            sum += x;
        }
    }
    return sum;
}

__device__ __forceinline__ void scatter_tile(const SortArgs &a, const SortShared &s, const SortTile &t, int pass) {
    const int warp = threadIdx.x / 32;
    const uint32_t *from = a.pos[(pass + 1) % 2];
    uint32_t *key = a.key[pass % 2], *pos = a.pos[pass % 2];
    uint32_t p[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t at = t.first + 32 * i;
        if (i < t.items && at < t.end) p[i] = pass == 0 ? at : __ldcg(from + at);
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        if (i >= t.items || t.first + 32 * i >= t.end) continue;
        const uint32_t digit = t.spot[i] >> 16;
        const uint32_t to = s.base[digit] + s.count[warp][digit] + (t.spot[i] & 0xffffu);
        key[to] = t.key[i];
        pos[to] = p[i];
    }
}

// A stable radix sort by digits of up to 10 bits. Each CTA has a stretch of the
// entries; the CTAs' counts of every digit tell where its entries go. Entries
// that are no token have the key `vocab` and come last.
__global__ void __launch_bounds__(kSortThreads, 1) sort_kernel(const __grid_constant__ SortArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    SortShared &s = *reinterpret_cast<SortShared *>(raw);
    const uint32_t rank = tc::cluster_rank(), ctas = cluster_size();
    const uint32_t each = (a.n + ctas - 1) / ctas;
    const uint32_t begin = min(rank * each, a.n), end = min(begin + each, a.n);
    const uint32_t digits = 1u << a.bits;
    const bool one = end - begin <= kTile;
    wait_previous();
    allow_next();
    for (int pass = 0; pass < a.passes; ++pass) {
        const int shift = pass * a.bits;
        SortTile t;
        uint32_t total = 0;
        for (uint32_t at = begin; at < end; at += kTile) {
            load_tile(a, pass, at, min(at + kTile, end), t);
            total += rank_tile(s, t, shift, digits);
            if (!one) __syncthreads();
        }
        if (threadIdx.x < digits) s.total[threadIdx.x] = total;
        tc::cluster_sync();
        uint32_t all = 0, before = 0;
        if (threadIdx.x < digits) {
#pragma unroll
            for (uint32_t c = 0; c < kMostCtas; ++c) {
                const uint32_t x = c < ctas ? load_peer(&s.total[threadIdx.x], c) : 0u;
                all += x;
                before += c < rank ? x : 0u;
            }
        }
        const uint32_t start = before_all(all, s.sums);
        if (threadIdx.x < digits) s.base[threadIdx.x] = start + before;
        __syncthreads();
        for (uint32_t at = begin; at < end; at += kTile) {
            uint32_t here = 0;
            if (!one) {
                load_tile(a, pass, at, min(at + kTile, end), t);
                here = rank_tile(s, t, shift, digits);
                __syncthreads();
            }
            scatter_tile(a, s, t, pass);
            if (!one) {
                __syncthreads();
                if (threadIdx.x < digits) s.base[threadIdx.x] += here;
            }
        }
        // the next pass reads what the cluster has written, and overwrites the totals
        __threadfence();
        tc::cluster_sync();
    }
}

// ---------------------------------------------------------------- rows that no token uses

constexpr int kFillThreads = 1024;
constexpr int64_t kWindow = 16384;  // rows whose use is known at a time

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
__global__ void __launch_bounds__(kFillThreads, 1) fill_kernel(const __grid_constant__ FillArgs a) {
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

// A lane's columns of one row's sum to the gradient: times scale, and added to
// what is there.
template <int DT, bool VEC>
__device__ __forceinline__ void write_row(const SumArgs &a, uint32_t key, int64_t col0,
                                          float (&sum)[Slice<DT, VEC>::kWords][Slice<DT, VEC>::kElems]) {
    using S = Slice<DT, VEC>;
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
            const float4 x = *reinterpret_cast<const float4 *>(p + e);
            f[e] += x.x, f[e + 1] += x.y, f[e + 2] += x.z, f[e + 3] += x.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] += p[e];
    }
}

constexpr int kTogether = 4;  // rows whose loads go out together

template <int DT, bool VEC> __global__ void __launch_bounds__(kThreads) sum_kernel(const __grid_constant__ SumArgs a) {
    using S = Slice<DT, VEC>;
    const int lane = threadIdx.x % 32;
    const int64_t at = int64_t(blockIdx.x) * kWarps + threadIdx.x / 32;
    const uint32_t chunk = static_cast<uint32_t>(at / a.slices);
    const int64_t col0 = (at - int64_t(chunk) * a.slices) * S::kCols + lane * S::kElems;
    wait_previous();
    allow_next();
    if (chunk >= a.chunks) return;
    const uint32_t first = chunk * static_cast<uint32_t>(a.chunk);
    const uint32_t n = min(static_cast<uint32_t>(a.chunk), a.n - first);
    const uint32_t key = lane < n ? a.key[first + lane] : a.vocab;
    const uint32_t pos = lane < n ? a.pos[first + lane] : 0u;
    const uint32_t before = first > 0 ? a.key[first - 1] : a.vocab;
    const uint32_t after = first + n < a.n ? a.key[first + n] : a.vocab;
    const int count = __popc(__ballot_sync(0xffffffffu, key < a.vocab));  // (what is no token comes last)
    if (count == 0) return;
    const uint32_t next = __shfl_down_sync(0xffffffffu, key, 1);
    // entries that end a run here; runs that began before, or go on after
    const uint32_t ends = __ballot_sync(0xffffffffu, lane < count && (lane + 1 == count || next != key));
    const bool from_before = before == __shfl_sync(0xffffffffu, key, 0);
    const bool goes_on = after == __shfl_sync(0xffffffffu, key, count - 1);
    const int first_end = __ffs(ends) - 1;
    float sum[S::kWords][S::kElems];
#pragma unroll
    for (int j = 0; j < S::kWords; ++j)
#pragma unroll
        for (int e = 0; e < S::kElems; ++e) sum[j][e] = 0.0f;
    for (int i0 = 0; i0 < count; i0 += kTogether) {
        Word<DT, VEC> w[kTogether][S::kWords];
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
            // (past the end: the last row again, not added)
            const uint8_t *row = a.d_out + int64_t(__shfl_sync(0xffffffffu, pos, min(i0 + u, count - 1))) * a.out_bytes;
#pragma unroll
            for (int j = 0; j < S::kWords; ++j) {
                const int64_t col = col0 + j * 32 * S::kElems;
                if (col < a.dim) w[u][j].load(row, col);
            }
        }
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
            const int i = i0 + u;
            if (i >= count) break;
#pragma unroll
            for (int j = 0; j < S::kWords; ++j) {
                float f[S::kElems];
                w[u][j].widen(f);
#pragma unroll
                for (int e = 0; e < S::kElems; ++e) sum[j][e] += f[e];
            }
            if (!(ends >> i & 1u)) continue;
            const bool head = i == first_end && from_before, tail = i + 1 == count && goes_on;
            if (head || tail) {
                float *part = a.part + (int64_t(chunk) * 2 + (head ? 0 : 1)) * a.ld_part;
#pragma unroll
                for (int j = 0; j < S::kWords; ++j) {
                    const int64_t col = col0 + j * 32 * S::kElems;
                    if (col < a.dim) store_floats<S::kElems>(part + col, sum[j]);
                }
            } else {
                write_row<DT, VEC>(a, __shfl_sync(0xffffffffu, key, i), col0, sum);
            }
#pragma unroll
            for (int j = 0; j < S::kWords; ++j)
#pragma unroll
                for (int e = 0; e < S::kElems; ++e) sum[j][e] = 0.0f;
        }
    }
}

// The parts of a run that crosses chunks: the last part of the chunk it begins
// in and the first parts of the `length` chunks after it.
template <int DT, bool VEC>
__device__ __forceinline__ void add_parts(const SumArgs &a, uint32_t chunk, uint32_t length, int64_t col0, uint32_t begin,
                                          uint32_t step,
                                          float (&sum)[Slice<DT, VEC>::kWords][Slice<DT, VEC>::kElems]) {
    using S = Slice<DT, VEC>;
#pragma unroll
    for (int j = 0; j < S::kWords; ++j)
#pragma unroll
        for (int e = 0; e < S::kElems; ++e) sum[j][e] = 0.0f;
#pragma unroll 2
    for (uint32_t i = begin; i <= length; i += step) {
        const float *part = a.part + (int64_t(chunk + i) * 2 + (i == 0 ? 1 : 0)) * a.ld_part;
#pragma unroll
        for (int j = 0; j < S::kWords; ++j) {
            const int64_t col = col0 + j * 32 * S::kElems;
            if (col < a.dim) add_floats<S::kElems>(part + col, sum[j]);
        }
    }
}

constexpr uint32_t kAlone = 16;  // parts that a warp adds up by itself

// A warp looks at a chunk: whether a run that crosses its end begins in it, and
// over how many more chunks it goes. It adds up a short run itself; the
// block's warps share a long one (each every eighth part, then the warps' sums
// in order).
template <int DT, bool VEC> __global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ SumArgs a) {
    using S = Slice<DT, VEC>;
    __shared__ float sums[kWarps][32][S::kWords * S::kElems + 1];
    __shared__ uint32_t lengths[kWarps], keys[kWarps];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const uint32_t chunk0 = blockIdx.x * kWarps, chunk = chunk0 + warp;
    const int64_t col0 = int64_t(blockIdx.y) * S::kCols + lane * S::kElems;
    wait_previous();
    allow_next();
    uint32_t length = 0, key = a.vocab;
    const uint64_t next = (uint64_t(chunk) + 1) * a.chunk;
    if (next < a.n) {
        const uint32_t first = chunk * static_cast<uint32_t>(a.chunk);
        key = a.key[next - 1];
        const bool begins = a.key[first] != key || first == 0 || a.key[first - 1] != key;
        if (key < a.vocab && begins && a.key[next] == key) {
            uint32_t lo = chunk + 1, hi = a.chunks;  // the last chunk that begins with the key is in [lo, hi)
            while (hi - lo > 1) {
                const uint32_t mid = lo + (hi - lo) / 2;
                if (a.key[uint64_t(mid) * a.chunk] == key)
                    lo = mid;
                else
                    hi = mid;
            }
            length = lo - chunk;
        }
    }
    float sum[S::kWords][S::kElems];
    if (length > 0 && length < kAlone) {
        add_parts<DT, VEC>(a, chunk, length, col0, 0, 1, sum);
        write_row<DT, VEC>(a, key, col0, sum);
        length = 0;
    }
    if (lane == 0) {
        lengths[warp] = length;
        keys[warp] = key;
    }
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) {
        if (lengths[i] == 0) continue;  // (the same for all)
        add_parts<DT, VEC>(a, chunk0 + i, lengths[i], col0, warp, kWarps, sum);
#pragma unroll
        for (int j = 0; j < S::kWords; ++j)
#pragma unroll
            for (int e = 0; e < S::kElems; ++e) sums[warp][lane][j * S::kElems + e] = sum[j][e];
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < kWarps; ++w)
#pragma unroll
                for (int j = 0; j < S::kWords; ++j)
#pragma unroll
                    for (int e = 0; e < S::kElems; ++e) sum[j][e] += sums[w][lane][j * S::kElems + e];
            write_row<DT, VEC>(a, keys[i], col0, sum);
        }
        __syncthreads();
    }
}

template <int DT, bool VEC> fsdp_status launch_type(const SumArgs &a, cudaStream_t s) {
    const int64_t blocks = (int64_t(a.chunks) * a.slices + kWarps - 1) / kWarps;
    if (blocks > 0x7fffffff || a.slices > 65535) return FSDP_ERR_INVALID_ARG;
    fsdp_status st = launch_chained(sum_kernel<DT, VEC>, static_cast<unsigned>(blocks), kThreads, 0, s, a);
    if (st != FSDP_OK || a.chunks == 1) return st;
    const dim3 grid((a.chunks + kWarps - 1) / kWarps, a.slices);
    return launch_chained(join_kernel<DT, VEC>, grid, kThreads, 0, s, a);
}

}  // namespace

fsdp_status launch_sort(const SortArgs &a, cudaStream_t s) {
    static PerDeviceOnce once;
    const int dev = current_device();
    if (!once.is_done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(sizeof(SortShared)));
        if (e != cudaSuccess) return cuda_status(e);
        once.mark(dev);
    }
    // a thread each for up to 8192 entries: a pass is mostly waiting
    unsigned ctas = 1;
    while (ctas < kMostCtas && ctas * kSortThreads < a.n) ctas *= 2;
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
    return cuda_status(cudaLaunchKernelEx(&config, sort_kernel, a));
}

fsdp_status launch_fill(const FillArgs &a, cudaStream_t s) {
    const int64_t sms = sm_count() > 0 ? sm_count() : 1, most = (a.vocab + 31) / 32;
    return launch_chained(fill_kernel, static_cast<unsigned>(sms < most ? sms : most), kFillThreads, 0, s, a);
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
