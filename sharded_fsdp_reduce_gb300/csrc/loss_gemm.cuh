// loss_gemm.cuh -- the matrix product of the head loss on CTA pairs.
//
// One kernel text for three products, by the operands' orders:
//   logits  L = X W^T        A = X  [T,D] K-major,  B = W [V,D] K-major
//   dX      = d W            A = d  [T,V] K-major,  B = W [V,D] N-major (K = V)
//   dW      = d^T X          A = d  [T,V] M-major,  B = X [T,D] N-major (K = T)
// so none of the operands is ever transposed in memory.
//
// A pair of CTAs (one cluster) works on a 256 x 256 tile of the result: each
// loads 128 rows of A and 128 of B per 64-wide K block by TMA (32 KB a stage,
// five or six stages), the even CTA issues the tcgen05 products for both
// (M = N = 256, K = 16), and each CTA's tensor memory holds 128 rows of the
// accumulator in fp32, twice (2 x 256 columns): the epilogue of one tile runs
// while the next one's products are issued. Against single CTAs of 128 x 256
// the pair takes a third off the operand bytes that shared memory and L2 must
// deliver. Persistent: one CTA per SM, tiles taken in a fixed order that keeps
// the reused operand in L2.
//
// Bound by the tensor pipes where K is long (2048 x 32000 x 5120: 354 us, 97.9 %
// active, 1.90 PFLOP/s; under the power cap 4096 x 128000 x 8192 runs at 1.50 to
// 1.70), by the operands' latency where a tile has few K blocks (1021 x 50257 x
// 768: 59 us, 67 % active).
//
// Roles by warp: 0 loads A and 3 loads B, 1 issues the products, 2 owns tensor
// memory, 4-19 are the epilogue: warp w reads lanes 32 (w % 4) .. + 31 (one
// row per thread), columns 64 ((w - 4) / 4) .. + 63.
//
// An fp32 operand is held as three bf16 planes (its leading, middle and last
// 8 bits). A stage then holds all three planes of both operands (96 KB, two
// stages), and each K block issues the six plane pairs whose products reach
// 2^-16 of the leading one, smallest first, into the same accumulator. What it
// leaves out is below 2^-23 of the product of the operands' magnitudes. (K
// loops over one pair after the other read every plane twice: 512 x 32000 x
// 1280 with its gradients 610 us, with planes side by side 573.)
//
// Every wait gives up after about a second, records itself and makes the pair
// leave; the result is then incomplete and the counter says so.
#pragma once

#include <float.h>

#include "loss.cuh"
#include "tcgen.cuh"

namespace fsdp {
namespace loss {

constexpr int kThreads = 640;
constexpr int kEpilogueWarps = 16;
// Stages of operands in shared memory. One more each would fit: 4096 x 128000 x
// 8192 with its gradients takes 15.4 to 15.6 ms either way, the hidden gradient
// of 1021 x 50257 x 768, a split product of few tiles, 62 us with these and 55
// with one more (of 215 in all), its other products the same.
constexpr int stages(int epilogue, int planes) { return planes == 3 ? 2 : epilogue == kExp ? 5 : 6; }
constexpr int kMaxStages = 6;
// K blocks summed in tensor memory before the sum moves to registers. The
// tensor cores' own sum loses bits at every K = 16 (a chain of 5120 / 16 adds
// left a loss 2.4e-6 off, 64 bits against it); chains of 512 / 16 joined by
// rounded fp32 adds do not show in fp32 results, chains of 2048 / 16 not in
// 16-bit ones. A move every 8 blocks costs up to 4 % against every 16 where K
// is split (the hidden gradient of 4096 x 50257 x 1280 358 us against 344) and
// nothing that shows elsewhere (4096 x 128000 x 8192 15.4 to 15.6 ms in all).
constexpr int chunk_blocks(int epilogue, int dtype, int planes) {
    return planes == 3 ? 1 : epilogue == kScale && dtype != FSDP_F32 ? 32 : 8;  // (a block of planes is 24 adds)
}
constexpr uint32_t kHalfBytes = 128 * kBlockK * 2;       // one plane of one operand's half tile: 16 KB
constexpr uint32_t stage_bytes(int planes) { return 2 * planes * kHalfBytes; }  // per CTA
constexpr uint32_t kTensorCols = 512;                    // two accumulators of 256 columns
constexpr long long kWaitCycles = 2000000000ll;          // about one second of SM clocks

struct Barriers {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tensor_base;
    int32_t gave_up;
};

constexpr uint32_t kBoxBytes = 32 * 64;                  // one warp's store box: 32 rows of 64 bytes
constexpr size_t smem_bytes(int epilogue, int planes) {
    return 1024 + stages(epilogue, planes) * stage_bytes(planes) + (epilogue == kExp ? kEpilogueWarps * kBoxBytes : 0) +
           sizeof(Barriers);
}
static_assert(smem_bytes(kExp, 1) <= 232448 && smem_bytes(kScale, 1) <= 232448 && smem_bytes(kExp, 3) <= 232448, "shared memory of one block");

// The products of one K block of three planes: the (A, B) planes of each, low
// nibble first.
constexpr uint32_t kPlanesA = 0x001021, kPlanesB = 0x010201;
constexpr int plane_products(int planes) { return planes == 3 ? 6 : 1; }
constexpr uint32_t plane_of(uint32_t list, int planes, int product) {
    return planes == 3 ? (list >> (4 * product)) & 15 : 0;
}

struct Tile {
    int m, n, split;
};

__device__ __forceinline__ Tile tile_at(const GemmArgs &g, int t) {
    const int per = g.tiles_m * g.tiles_n;
    Tile r;
    r.split = t / per;
    t -= r.split * per;
    const int fast = g.m_fast ? g.tiles_m : g.tiles_n, slow = g.m_fast ? g.tiles_n : g.tiles_m;
    const int first = t / (g.group * slow) * g.group;
    t -= first * slow;
    const int width = min(g.group, fast - first);
    const int f = first + t % width, s = t / width;
    r.m = g.m_fast ? f : s;
    r.n = g.m_fast ? s : f;
    return r;
}

// The K blocks of a split.
__device__ __forceinline__ void k_range(const GemmArgs &g, int split, int &begin, int &end) {
    begin = split * g.k_each + min(split, g.k_more);
    end = begin + g.k_each + (split < g.k_more ? 1 : 0);
}

// Bounded wait of a whole warp: all of its lanes get the same answer, since
// what follows (tensor-memory reads, elections) needs them together. False
// once any wait of this CTA has given up; `timeouts` counts the warps whose
// time ran out.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, Barriers *b, uint32_t *timeouts,
                                     long long limit = kWaitCycles) {
    constexpr uint32_t kAll = 0xffffffffu;
    if (__all_sync(kAll, tma::mbar_try_wait(bar, parity))) return true;
    const long long t0 = clock64();
    volatile int32_t *gave_up = &b->gave_up;
    while (!__all_sync(kAll, tma::mbar_try_wait(bar, parity))) {
        // one lane's flag and clock decide for all
        const int state = __shfl_sync(kAll, *gave_up ? 1 : clock64() - t0 > limit ? 2 : 0, 0);
        if (state == 0) continue;
        if (state == 2 && threadIdx.x % 32 == 0) {
            *gave_up = 1;
            if (timeouts) atomicAdd(timeouts, 1u);
        }
        return false;
    }
    return true;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// One row's 64 values (a thread's) to a gradient, rounded to DT: each thread
// writes 128 or 256 contiguous bytes, in the widest stores that the result's
// base and stride allow. Straight from registers: a gradient's tile is
// written once in many K blocks, at any alignment.
__device__ __forceinline__ void store32(void *p, uint4 a, uint4 b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

template <int DT> __device__ __forceinline__ uint4 pack16(const float *v) {
    if constexpr (DT == FSDP_F32)
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
        return make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7]));
}

template <int DT>
__device__ __forceinline__ void store_span(const GemmArgs &g, int64_t row, int64_t col0, int split, const float *v) {
    if (row >= g.M) return;
    constexpr int kSize = Dtype<DT>::kSize, kPer16 = 16 / kSize;
    const int64_t at = split * g.split_stride + row * g.ld_out + col0;
    uint8_t *out = static_cast<uint8_t *>(g.out) + at * kSize;
    if (g.store_bytes == 32 && col0 + kSpan <= g.store_cols) {
#pragma unroll
        for (int j = 0; j < kSpan; j += 2 * kPer16)
            store32(out + j * kSize, pack16<DT>(v + j), pack16<DT>(v + j + kPer16));
        return;
    }
#pragma unroll
    for (int j = 0; j < kSpan; j += kPer16) {
        if (g.store_bytes >= 16 && col0 + j + kPer16 <= g.store_cols) {
            *reinterpret_cast<uint4 *>(out + j * kSize) = pack16<DT>(v + j);
        } else {
#pragma unroll
            for (int e = 0; e < kPer16; ++e)
                if (col0 + j + e < g.store_cols) Dtype<DT>::store(out, j + e, v[j + e]);
        }
    }
}

// One warp's 32 rows x 64 columns of exponentials, by TMA from a small box in
// shared memory (64-byte rows, 64-byte swizzle), part after part: written on
// every tile of few K blocks, stores from registers took 67 us where this
// takes 60 (1021 x 50257 x 768).
template <int DT>
__device__ __forceinline__ void store_exponentials(const CUtensorMap *map, uint8_t *box, int lane, int64_t row0,
                                                   int64_t col0, const float *v) {
    constexpr int kPer16 = 16 / Dtype<DT>::kSize, kCols = 4 * kPer16;
    uint8_t *row = box + lane * 64;
    const int turn = (lane >> 1) & 3;
#pragma unroll
    for (int c = 0; c < kSpan; c += kCols) {
        if (lane == 0) tma::bulk_wait_read<0>();  // the last store has read the box
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4 *>(row + ((i ^ turn) << 4)) = pack16<DT>(v + c + i * kPer16);
        tma::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tc::store_tile(map, static_cast<int>(col0 + c), static_cast<int>(row0), 0, box);
            tma::bulk_commit();
        }
    }
}

// v[j] of 64 registers: a tree of selections, group after group, so that few
// of them wait.
__device__ __forceinline__ float pick(const float *v, int j) {
    float group[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float *x = v + 8 * i;
        const float a = j & 1 ? x[1] : x[0], b = j & 1 ? x[3] : x[2], c = j & 1 ? x[5] : x[4], d = j & 1 ? x[7] : x[6];
        const float e = j & 2 ? b : a, f = j & 2 ? d : c;
        group[i] = j & 4 ? f : e;
    }
    const float a = j & 8 ? group[1] : group[0], b = j & 8 ? group[3] : group[2];
    const float c = j & 8 ? group[5] : group[4], d = j & 8 ? group[7] : group[6];
    const float e = j & 16 ? b : a, f = j & 16 ? d : c;
    return j & 32 ? f : e;
}

// Softmax statistics (and exponentials) of one warp's 32 rows x 64 columns. A
// span's exponentials are against its own largest logit, subtracted as it is:
// the largest one is then exactly 1, the sum at least 1 and a row's loss
// neither negative nor, for a row that is sure of its target, the difference
// of two roundings (log2(e) times the largest would be rounded once more, and
// past 2^31 by more than exponentials can hold). In fp16 they are stored times
// 2^15: 11 bits down to 2^-29 of the span's largest (what is smaller is below
// 2^-40 of it).
//
// SOFT: the exponentials are of the logits over a temperature, and the logits
// of the teacher's entries are stored. `target` holds the row's first entry of
// the span and the first one after it, id the first one's token.
template <int EP, int DT, bool SOFT>
__device__ __forceinline__ void softmax_span(const GemmArgs &g, const CUtensorMap *map, uint8_t *box, int lane,
                                             float *v, int64_t row0, int64_t col0, int64_t target, int id) {
    const float kLog2e = SOFT ? g.log2e : 1.44269504088896340736f;
    const int64_t row = row0 + lane;
    const bool live = row < g.M;
    if constexpr (SOFT) {
        const uint32_t end = static_cast<uint32_t>(target) >> 16;
        const int32_t *ids = g.ids + row * g.top;
        float *to = g.at + row * g.top;
#pragma unroll 1
        for (uint32_t k = static_cast<uint32_t>(target) & 0xffffu; k < end;) {
            to[k] = pick(v, id - static_cast<int>(col0));
            if (++k < end) id = ids[k];
        }
    } else {
        const int64_t at = target - col0;
        if (at >= 0 && at < kSpan && at + col0 < g.N) {
            float t = 0.0f;
#pragma unroll
            for (int j = 0; j < kSpan; ++j)
                if (at == j) t = v[j];
            g.target_logit[row] = t;
        }
    }
    if (col0 + kSpan > g.N) {
        const int cols = static_cast<int>(g.N - col0);
#pragma unroll
        for (int j = 0; j < kSpan; ++j)
            if (j >= cols) v[j] = -INFINITY;
    }
    float t0 = -FLT_MAX, t1 = -FLT_MAX;
#pragma unroll
    for (int j = 0; j < kSpan; j += 2) {
        t0 = fmaxf(t0, v[j]);
        t1 = fmaxf(t1, v[j + 1]);
    }
    const float top = fmaxf(t0, t1);
    float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
    for (int j = 0; j < kSpan; ++j) v[j] = exp2_fast((v[j] - top) * kLog2e);
#pragma unroll
    for (int j = 0; j < kSpan; j += 4) {
        s0 += v[j];
        s1 += v[j + 1];
        s2 += v[j + 2];
        s3 += v[j + 3];
    }
    if (live) {
        const int64_t to = col0 / kSpan * g.ld_rows + row;
        g.off[to] = top;
        g.sum[to] = (s0 + s1) + (s2 + s3);
    }
    if constexpr (EP == kExp && DT == FSDP_F16) {
#pragma unroll
        for (int j = 0; j < kSpan; ++j) v[j] *= kExpGain;
    }
    if constexpr (EP == kExp) store_exponentials<DT>(map, box, lane, row0, col0, v);
}

// scale * (accumulator + earlier) of one warp's 32 rows x 64 columns.
template <int DT>
__device__ __forceinline__ void scaled_span(const GemmArgs &g, float *v, int64_t row, int64_t col0, int split,
                                            float scale) {
    if (g.earlier != nullptr && row < g.M) {
        const float *e = g.earlier + row * g.ld_earlier + col0;  // 16-byte aligned, padded to 64 columns
#pragma unroll
        for (int j = 0; j < kSpan; j += 4) {
            if (col0 + j < g.N) {
                const float4 x = *reinterpret_cast<const float4 *>(e + j);
                v[j] += x.x;
                v[j + 1] += x.y;
                v[j + 2] += x.z;
                v[j + 3] += x.w;
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kSpan; ++j) v[j] *= scale;
    store_span<DT>(g, row, col0, split, v);
}

// One operand's loads, by one warp of each CTA: its 128 rows of every K block
// of every tile, into the stages in turn. Each operand has a warp of its own,
// and the whole warp runs the loop while one elected thread issues, so that
// what it issues with stays in uniform registers: a single thread's loop over
// both operands took 830 cycles a K block, over one 500; the products take 512
// and a load that comes late has to be made up.
template <int MN, bool A, int P, int kStages>
__device__ __forceinline__ void load_operand(const GemmArgs &g, const CUtensorMap *map, uint8_t *smem, Barriers *b,
                                             uint32_t rank, int first, int total, int step) {
    const uint32_t full = tc::peer_addr(tc::smem_addr(&b->full[0]), 0), to = tc::smem_addr(smem);
    const bool expects = A && rank == 0;
    uint32_t *timeouts = g.timeouts;
    int stage = 0;
    uint32_t phase = 1;
    for (int t = first; t < total; t += step) {
        const Tile x = tile_at(g, t);
        int k0, k1;
        k_range(g, x.split, k0, k1);
        const int at = (A ? x.m * kTileM : x.n * kTileN) + static_cast<int>(rank) * 128;
        for (int k = k0; k < k1; ++k) {
            if (!wait(&b->empty[stage], phase, b, timeouts)) return;
            const uint32_t bar = full + stage * static_cast<uint32_t>(sizeof(uint64_t));
            const uint32_t dst = to + stage * stage_bytes(P);
            if (tc::elect_one()) {
                if (expects) tma::mbar_arrive_expect_tx(&b->full[stage], 2 * stage_bytes(P));
                // boxes hold all planes: K-major 128 rows each, MN-major twice 64 columns
                if constexpr (MN) {
                    tc::load_tile(dst, map, at, k * kBlockK, 0, bar);
                    tc::load_tile(dst + P * (kHalfBytes / 2), map, at + 64, k * kBlockK, 0, bar);
                } else {
                    tc::load_tile(dst, map, k * kBlockK, at, 0, bar);
                }
            }
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
    }
    // the last use of every stage has been consumed: no copy of this CTA is in
    // flight and no product still signals its barriers
    for (int s = 0; s < kStages; ++s) {
        if (!wait(&b->empty[stage], phase, b, timeouts)) return;
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
        }
    }
}

// The products of every tile, by one warp of the even CTA for the pair. The
// whole warp runs the loop and one elected thread issues: what it issues with
// then stays in uniform registers (a single thread's loop moved every operand
// there first, 560 cycles a K block against the products' 512).
template <int AMN, int BMN, int P, int kStages, int kChunk>
__device__ __forceinline__ void issue_products(const GemmArgs &g, uint8_t *smem, Barriers *b, uint32_t tensor,
                                               int first, int total, int step) {
    const uint32_t idesc = tc::instruction(0, AMN, BMN, kTileM, kTileN) |
                           (static_cast<uint32_t>(g.operand_type) << 7) |
                           (static_cast<uint32_t>(g.operand_type) << 10);
    // per K = 16: 32 bytes along a K-major row, two groups of eight K otherwise
    constexpr uint32_t kStepA = (AMN ? 2048 : 32) >> 4, kStepB = (BMN ? 2048 : 32) >> 4;
    constexpr uint32_t kHigh = tc::operand_high(1024);
    const uint32_t sa = tc::smem_addr(smem);
    const uint32_t a0 = tc::operand_low(sa, AMN ? P * (kHalfBytes / 2) : 16);
    const uint32_t b0 = tc::operand_low(sa + P * kHalfBytes, BMN ? P * (kHalfBytes / 2) : 16);
    // from one plane of an operand to the next
    constexpr uint32_t kPlaneA = (AMN ? kHalfBytes / 2 : kHalfBytes) >> 4;
    constexpr uint32_t kPlaneB = (BMN ? kHalfBytes / 2 : kHalfBytes) >> 4;
    const int tiles = g.tiles_m * g.tiles_n, splits = g.splits;
    uint32_t *timeouts = g.timeouts;
    int k0, k1;
    k_range(g, 0, k0, k1);
    int stage = 0, buf = 0;
    uint32_t phase = 0, acc_phase = 1;
    for (int t = first; t < total; t += step) {
        if (splits > 1) k_range(g, t / tiles, k0, k1);
        for (int c = k0; c < k1; c += kChunk) {
            if (!wait(&b->acc_empty[buf], acc_phase, b, timeouts)) return;
            tc::fence_after();
            const int end = min(c + kChunk, k1);
            const uint32_t d = tensor + buf * kTileN;
            for (int k = c; k < end; ++k) {
                if (!wait(&b->full[stage], phase, b, timeouts)) return;
                tc::fence_after();
                const uint32_t da = a0 + stage * (stage_bytes(P) >> 4), db = b0 + stage * (stage_bytes(P) >> 4);
                if (tc::elect_one()) {
#pragma unroll
                    for (int q = 0; q < plane_products(P); ++q)
#pragma unroll
                        for (int j = 0; j < kBlockK / 16; ++j)
                            tc::mma_pair(d, da + plane_of(kPlanesA, P, q) * kPlaneA + j * kStepA,
                                         db + plane_of(kPlanesB, P, q) * kPlaneB + j * kStepB, kHigh, idesc,
                                         k > c || q > 0 || j > 0);
                    tc::commit_pair(&b->empty[stage]);
                    if (k + 1 == end) tc::commit_pair(&b->acc_full[buf]);
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            buf ^= 1;
            acc_phase ^= buf == 0;
        }
    }
}

template <int AMN, int BMN, int EP, int DT, int P, bool SOFT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                const __grid_constant__ CUtensorMap map_out, const __grid_constant__ GemmArgs g) {
    constexpr int kStages = stages(EP, P), kChunk = chunk_blocks(EP, DT, P);
    extern __shared__ uint8_t raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    uint8_t *boxes = smem + kStages * stage_bytes(P);
    Barriers *b = reinterpret_cast<Barriers *>(boxes + (EP == kExp ? kEpilogueWarps * kBoxBytes : 0));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0), lane = threadIdx.x % 32;  // (uniform)
    const uint32_t rank = tc::cluster_rank();
    const int total = g.tiles_m * g.tiles_n * g.splits;
    const int first = blockIdx.x / 2, step = gridDim.x / 2;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
            tma::mbar_init(&b->full[s], 1);
            tma::mbar_init(&b->empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            tma::mbar_init(&b->acc_full[s], 1);
            tma::mbar_init(&b->acc_empty[s], 2 * kEpilogueWarps);
        }
        b->gave_up = 0;
        tma::fence_mbar_init();
        tc::prefetch_map(&map_a);
        tc::prefetch_map(&map_b);
    }
    __syncwarp();
    if (warp == 2) tc::alloc_pair(&b->tensor_base, kTensorCols);
    wait_previous();
    allow_next();
    if constexpr (EP != kScale) {
        if (blockIdx.x == 0 && threadIdx.x == 96 && g.ticket != nullptr) *g.ticket = 0;
    }
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();  // both CTAs' barriers exist before either signals the other's
    tc::fence_after();
    const uint32_t tensor = b->tensor_base;

    // registers: 56 a thread for the first four warps, 104 for the epilogue's
    // sixteen (a row of 64 sums each): 128 * 56 + 512 * 104 = 60,416 of the
    // 640 * 96 = 61,440 the block was launched with
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0)
            load_operand<AMN, true, P, kStages>(g, &map_a, smem, b, rank, first, total, step);
        else if (warp == 3)
            load_operand<BMN, false, P, kStages>(g, &map_b, smem + P * kHalfBytes, b, rank, first, total, step);
        else if (warp == 1 && rank == 0)
            issue_products<AMN, BMN, P, kStages, kChunk>(g, smem, b, tensor, first, total, step);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
        const int quarter = warp % 4, part = (warp - 4) / 4;
        float scale = 1.0f;
        if constexpr (EP == kScale) scale = g.scale_const * (g.scale != nullptr ? *g.scale : 1.0f);
        int buf = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        for (int t = first; t < total && ok; t += step) {
            const Tile x = tile_at(g, t);
            int k0, k1;
            k_range(g, x.split, k0, k1);
            const int64_t row0 = int64_t(x.m) * kTileM + rank * 128 + quarter * 32;
            const int64_t col0 = int64_t(x.n) * kTileN + part * kSpan;
            int64_t target = SOFT ? 0 : -1;  // loaded while the products run
            int id = 0;
            if constexpr (EP != kScale && SOFT) {
                if (row0 + lane < g.M && col0 < g.N) {
                    const uint16_t *first = g.first + (row0 + lane) * g.ld_first + col0 / kSpan;
                    const uint32_t begin = first[0], end = first[1];
                    target = static_cast<uint32_t>(begin | end << 16);
                    if (begin < end) id = g.ids[(row0 + lane) * g.top + begin];
                }
            } else if constexpr (EP != kScale) {
                if (row0 + lane < g.M) target = g.targets[row0 + lane];
            }
            float v[kSpan];
#pragma unroll
            for (int j = 0; j < kSpan; ++j) v[j] = 0.0f;
            for (int k = k0; k < k1; k += kChunk) {
                if (!(ok = wait(&b->acc_full[buf], acc_phase, b, g.timeouts))) break;
                tc::fence_after();
                const uint32_t acc =
                    tensor + buf * kTileN + part * kSpan + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
                for (int c = 0; c < kSpan; c += 32) {
                    float r[32];
                    __syncwarp();
                    tc::load_cols32(acc + c, r);
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[c + j] += r[j];
                }
                tc::fence_before();
                __syncwarp();
                if (lane == 0) tc::arrive_cluster(tc::peer_addr(tc::smem_addr(&b->acc_empty[buf]), 0));
                buf ^= 1;
                acc_phase ^= buf == 0;
            }
            if (ok && row0 < g.M && col0 < g.N) {
                if constexpr (EP == kScale)
                    scaled_span<DT>(g, v, row0 + lane, col0, x.split, scale);
                else
                    softmax_span<EP, DT, SOFT>(g, &map_out, boxes + (warp - 4) * kBoxBytes, lane, v, row0, col0, target,
                                               id);
            }
        }
    }
    if constexpr (EP == kExp) {
        if (warp >= 4 && lane == 0) tma::bulk_wait<0>();
    }
    // a wait gave up: let copies and products that are only slow land before
    // the shared and tensor memory go
    __syncwarp();
    if (*static_cast<volatile int32_t *>(&b->gave_up)) {
        const long long t0 = clock64();
        while (clock64() - t0 < kWaitCycles) __nanosleep(1000);
    }
    tc::fence_before();
    __syncthreads();
    tc::cluster_sync();
    __syncwarp();
    if (warp == 2) tc::free_pair(tensor, kTensorCols);
}

template <int AMN, int BMN, int EP, int DT, int P, bool SOFT = false>
fsdp_status launch_kernel(const CUtensorMap &a, const CUtensorMap &b, const CUtensorMap &out, GemmArgs g,
                          cudaStream_t s) {
    g.k_each = g.kblocks / g.splits;
    g.k_more = g.kblocks % g.splits;
    static PerDeviceOnce once;
    const int dev = current_device();
    if (!once.is_done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(gemm_kernel<AMN, BMN, EP, DT, P, SOFT>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(smem_bytes(EP, P)));
        if (e != cudaSuccess) return cuda_status(e);
        once.mark(dev);
    }
    const int64_t total = int64_t(g.tiles_m) * g.tiles_n * g.splits;
    if (total < 1 || total > 0x3fffffff) return FSDP_ERR_INVALID_ARG;  // (the kernel's tile counter adds to it)
    const int64_t pairs = sm_count() / 2;
    const unsigned grid = static_cast<unsigned>(2 * (total < pairs ? total : (pairs > 0 ? pairs : 1)));
    return launch_chained(gemm_kernel<AMN, BMN, EP, DT, P, SOFT>, grid, kThreads, smem_bytes(EP, P), s, a, b, out, g);
}

}  // namespace loss
}  // namespace fsdp
