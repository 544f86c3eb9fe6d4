// clip_norm.cu -- the global L2 norm of many gradients in one pass, with the
// ranks' average formed and (when asked) kept on the way.
//
//   g = c * (G_0 + G_1 + ... + G_{N-1})   fp32, ranks in order
//   norm = |scale| * sqrt(sum over all units and elements of g^2)
//
// Bound by HBM (708 M bf16 elements 231 us, 6.2 TB/s; 85 M of eight ranks with
// the average written 252 us, 6.7 TB/s): N gradients are read (16-byte
// streaming loads) and, for the clipped step of many ranks, the fp32 average
// is written. Up to 32 squares (chunks_together) are added in fp32, which is
// within 9 roundings of 2^-24, those sums in pairs of floats (the sum and what
// its rounding lost) per thread and warp, and in fp64 per block and call, in
// an order fixed by the sizes, so the norm is the same bits every time: this
// part's fp64 units take 64 cycles for a warp's add, and adds per chunk held a
// pass over one bf16 list at 2.4 TB/s. Squares that overflow fp32, or are too
// small for it to hold their bits, are formed again at a scale where they
// fit, so the norm is right wherever its value is a finite fp32. The last
// block to finish (one counter, left at zero) adds the blocks' sums.
#include "clip.cuh"
#include "rsa_impl.cuh"

namespace fsdp {
namespace clip {
namespace {

// Sum of squares of eight averages.
__device__ __forceinline__ float squares(const float *g) {
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        s0 = fmaf(g[e], g[e], s0);
        s1 = fmaf(g[e + 1], g[e + 1], s1);
    }
    return s0 + s1;
}

// Whether an fp32 sum of squares kept fp32's bits, and may be added to a
// block's others: far from overflow, and nothing that mattered lost below
// fp32's smallest values.
__device__ __forceinline__ bool in_range(float s) { return s > 1e-30f && s < 1e30f; }

// A sum and what its roundings lost.
struct Pair {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float t = __fadd_rn(hi, x), b = __fsub_rn(t, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(t, b)), __fsub_rn(x, b)));
        hi = t;
    }
    __device__ __forceinline__ double value() const { return static_cast<double>(hi) + static_cast<double>(lo); }
};

// The same for any eight values, at a scale where their squares fit. By
// value: an address would keep every caller's values in local memory.
__device__ __noinline__ double squares_any(float4 lo, float4 hi) {
    const float g[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    float s = squares(g);
    if (in_range(s)) return s;
    float top = 0.0f;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        top = fmaxf(top, fabsf(g[e]));
        bad |= isnan(g[e]);
    }
    if (bad) return NAN;
    if (top == 0.0f) return 0.0;
    if (isinf(top)) return INFINITY;
    // large: top is 2^48 to 2^128; small: it is below 2^-49, down to 2^-149
    const float by = top > 1.0f ? 0x1p-70f : 0x1p100f;
    s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(g[e] * by, g[e] * by, s);
    return static_cast<double>(s) * (top > 1.0f ? 0x1p140 : 0x1p-200);
}
__device__ __forceinline__ double squares_any(const float *g) {
    return squares_any(make_float4(g[0], g[1], g[2], g[3]), make_float4(g[4], g[5], g[6], g[7]));
}

// The average of one chunk's gradients.
template <int NW, int GD>
__device__ __forceinline__ void average_of(float c, const rsa::GradRegs<NW, GD> &r, float *g) {
    rsa::widen8<GD>(r.w[0], g);
#pragma unroll
    for (int q = 1; q < NW; ++q) {
        float f[8];
        rsa::widen8<GD>(r.w[q], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = __fadd_rn(g[e], f[e]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = __fmul_rn(g[e], c);
}

// Stored where the update will read it; plain stores, kept in L2 where it fits.
template <int W> __device__ __forceinline__ void keep_average(const NormUnit<W> &u, int64_t j0, const float *g) {
    if (u.average == nullptr) return;
    *reinterpret_cast<float4 *>(u.average + j0) = make_float4(g[0], g[1], g[2], g[3]);
    *reinterpret_cast<float4 *>(u.average + j0 + 4) = make_float4(g[4], g[5], g[6], g[7]);
}

// The chunk [j0, j0 + 8) cut to [0, numel), zeros elsewhere: any rank count,
// any alignment.
template <int GD, int W>
__device__ __forceinline__ void cut_chunk(const NormUnit<W> &u, int world, float c, int64_t j0, float *g) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int64_t j = j0 + e;
        g[e] = 0.0f;
        if (j < 0 || j >= u.numel) continue;
        float acc = Dtype<GD>::load(u.grads[0], j);
        for (int q = 1; q < world; ++q) acc = __fadd_rn(acc, Dtype<GD>::load(u.grads[q], j));
        g[e] = __fmul_rn(acc, c);
        if (u.average != nullptr) u.average[j] = g[e];
    }
}

__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const float hi = __shfl_xor_sync(0xffffffffu, x.hi, o), lo = __shfl_xor_sync(0xffffffffu, x.lo, o);
        x.add(hi);
        x.lo = __fadd_rn(x.lo, lo);
    }
    return x;
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// One whole chunk of any number of ranks, by 16-byte loads.
template <int NW, int GD, int W>
__device__ __forceinline__ void whole_chunk(const NormUnit<W> &u, int world, float c, int64_t j0, float *g) {
    if constexpr (NW > 0) {
        rsa::GradRegs<NW, GD> r;
#pragma unroll
        for (int q = 0; q < NW; ++q) rsa::load_grad8<GD>(u.grads[q], j0, r.w[q]);
        average_of<NW, GD>(c, r, g);
    } else {
#pragma unroll 4
        for (int q = 0; q < world; ++q) {
            uint4 w[rsa::GradRegs<1, GD>::kWords];
            rsa::load_grad8<GD>(u.grads[q], j0, w);
            float f[8];
            rsa::widen8<GD>(w, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = q == 0 ? f[e] : __fadd_rn(g[e], f[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = __fmul_rn(g[e], c);
    }
    keep_average(u, j0, g);
}

// Chunks whose loads a thread has in flight together, their squares one fp32
// sum: eight 16-byte loads, but four for a single 16-bit tensor list, whose
// arithmetic per byte wants a fifth block per SM more (708 M bf16 elements
// 237 us against 281).
template <int NW, int GD> constexpr int chunks_together() {
    constexpr int kLoads = NW * rsa::GradRegs<1, GD>::kWords;
    return kLoads == 0 || kLoads >= 8 ? 1 : kLoads == 1 ? 4 : 8 / kLoads;
}

template <int NW, int GD, int W, int CAP>
__global__ void __launch_bounds__(kThreads, NW == 1 && GD != FSDP_F32 ? 5 : 4)
    norm_kernel(const __grid_constant__ NormArgs<W, CAP> a) {
    __shared__ Pair pairs[kThreads / 32];
    __shared__ double rare[kThreads / 32];
    __shared__ bool last;
    const NormUnit<W> &u = a.u[unit_of(a.u, a.n, blockIdx.x)];
    const int64_t first = (blockIdx.x - u.cta_begin) * (int64_t(8) * kThreads * a.per_thread) - u.lead;
    constexpr int U = chunks_together<NW, GD>();
    wait_previous();
    allow_next();
    Pair sum;
    double out_of_range = 0.0;  // what was summed at another scale
    bool any_rare = false;
    uint32_t bad = 0;
    auto rest = [&](const float *g) {
        out_of_range += squares_any(g);
        any_rare = true;
#pragma unroll
        for (int e = 0; e < 8; ++e) bad += isfinite(g[e]) ? 0u : 1u;
    };
    for (int i = 0; i < a.per_thread; i += U) {
        const int64_t j0 = first + 8 * (int64_t(i) * kThreads + threadIdx.x);
        if (j0 >= u.numel) break;
        if constexpr (U > 1) {
            const int64_t last_j = j0 + 8 * int64_t(U - 1) * kThreads;
            if (u.vec && j0 >= 0 && last_j + 8 <= u.numel && i + U <= a.per_thread) {
                rsa::GradRegs<NW, GD> r[U];
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int q = 0; q < NW; ++q)
                        rsa::load_grad8<GD>(u.grads[q], j0 + 8 * int64_t(k) * kThreads, r[k].w[q]);
                float all = 0.0f;
#pragma unroll
                for (int k = 0; k < U; ++k) {
                    float g[8];
                    average_of<NW, GD>(a.c, r[k], g);
                    keep_average(u, j0 + 8 * int64_t(k) * kThreads, g);
                    all += squares(g);
                }
                if (in_range(all)) {
                    sum.add(all);
                } else {
#pragma unroll
                    for (int k = 0; k < U; ++k) {
                        float g[8];
                        average_of<NW, GD>(a.c, r[k], g);
                        rest(g);
                    }
                }
                continue;
            }
        }
#pragma unroll 1
        for (int k = 0; k < U && i + k < a.per_thread; ++k) {
            const int64_t j = j0 + 8 * int64_t(k) * kThreads;
            if (j >= u.numel) break;
            float g[8];
            if (u.vec && j >= 0 && j + 8 <= u.numel) {
                whole_chunk<NW, GD, W>(u, a.world, a.c, j, g);
            } else {
                cut_chunk<GD, W>(u, a.world, a.c, j, g);
            }
            const float s = squares(g);
            if (in_range(s)) {
                sum.add(s);
            } else {
                rest(g);
            }
        }
    }
    if (a.out.nonfinite != nullptr) {
        const uint32_t total = __reduce_add_sync(0xffffffffu, bad);
        if (threadIdx.x % 32 == 0 && total) atomicAdd(a.out.nonfinite, total);
    }
    sum = warp_sum(sum);
    const int warp = threadIdx.x / 32;
    if (threadIdx.x % 32 == 0) pairs[warp] = sum;
    const bool has_rare = __syncthreads_or(any_rare);
    if (has_rare) {
        out_of_range = warp_sum(out_of_range);
        if (threadIdx.x % 32 == 0) rare[warp] = out_of_range;
        __syncthreads();
    }
    if (warp == 0) {
        Pair x;
        if (threadIdx.x < kThreads / 32) x = pairs[threadIdx.x];
        x = warp_sum(x);
        if (threadIdx.x == 0) {
            double all = x.value();
            if (has_rare)
                for (int w = 0; w < kThreads / 32; ++w) all += rare[w];
            a.out.part[a.out.part_begin + blockIdx.x] = all;
            __threadfence();
            last = atomicAdd(a.out.ticket, 1u) + 1 == static_cast<uint32_t>(a.out.part_count);
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double all = 0.0;
    for (int64_t i = threadIdx.x; i < a.out.part_count; i += kThreads) all += __ldcg(a.out.part + i);
    all = warp_sum(all);
    if (threadIdx.x % 32 == 0) rare[warp] = all;
    __syncthreads();
    if (threadIdx.x == 0) {
        all = 0.0;
        for (int w = 0; w < kThreads / 32; ++w) all += rare[w];
        *a.out.norm = static_cast<float>(sqrt(all) * static_cast<double>(a.out.scale));
        *a.out.ticket = 0;
    }
}

template <int NW, int W, int CAP>
fsdp_status launch_capacity(const NormArgs<W, CAP> &a, int dtype, unsigned grid, cudaStream_t s) {
    auto kernel = dtype == FSDP_BF16  ? norm_kernel<NW, FSDP_BF16, W, CAP>
                  : dtype == FSDP_F16 ? norm_kernel<NW, FSDP_F16, W, CAP>
                                      : norm_kernel<NW, FSDP_F32, W, CAP>;
    return launch_chained(kernel, grid, kThreads, 0, s, a);
}

template <int NW, int W> fsdp_status launch(const NormArgs<W> &a, int dtype, int64_t grid, cudaStream_t s) {
    if (a.n < 1 || a.n > NormArgs<W>::kUnits || grid < 1 || grid > 0x7fffffff) return FSDP_ERR_INVALID_ARG;
    if (a.n <= kFew) {
        NormArgs<W, kFew> few;
        few_of(a, few);
        return launch_capacity<NW>(few, dtype, static_cast<unsigned>(grid), s);
    }
    return launch_capacity<NW>(a, dtype, static_cast<unsigned>(grid), s);
}

}  // namespace

static_assert(sizeof(NormArgs<1>) < 32764 && sizeof(NormArgs<8>) < 32764 && sizeof(NormArgs<FSDP_MAX_WORLD>) < 32764,
              "kernel parameter space");

fsdp_status launch_norm(const NormArgs<1> &a, int dtype, int64_t grid, cudaStream_t s) {
    return launch<1>(a, dtype, grid, s);
}
fsdp_status launch_norm(const NormArgs<2> &a, int dtype, int64_t grid, cudaStream_t s) {
    return launch<2>(a, dtype, grid, s);
}
fsdp_status launch_norm(const NormArgs<4> &a, int dtype, int64_t grid, cudaStream_t s) {
    return launch<4>(a, dtype, grid, s);
}
fsdp_status launch_norm(const NormArgs<8> &a, int dtype, int64_t grid, cudaStream_t s) {
    return launch<8>(a, dtype, grid, s);
}
fsdp_status launch_norm(const NormArgs<FSDP_MAX_WORLD> &a, int dtype, int64_t grid, cudaStream_t s) {
    return launch<0>(a, dtype, grid, s);
}

}  // namespace clip
}  // namespace fsdp
