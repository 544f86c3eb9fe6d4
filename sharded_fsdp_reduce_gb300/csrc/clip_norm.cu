// clip_norm.cu -- the global L2 norm of many gradients in one pass, with the
// ranks' average formed and (when asked) kept on the way.
//
//   g = c * (G_0 + G_1 + ... + G_{N-1})   fp32, ranks in order
//   norm = |scale| * sqrt(sum over all units and elements of g^2)
//
// Bound by HBM: N gradients are read (16-byte streaming loads) and, for the
// clipped step of many ranks, the fp32 average is written. Squares of a
// thread's eight values are added in fp32, those sums in fp64 per thread,
// block and call, in an order fixed by the sizes, so the norm is the same
// bits every time. Eight squares that overflow fp32, or are too small for it
// to hold their bits, are formed again at a scale where they fit, so the norm
// is right wherever its value is a finite fp32. The last block to finish
// (one counter, left at zero) adds the blocks' sums.
#include "clip.cuh"
#include "rsa_impl.cuh"

namespace fsdp {
namespace clip {
namespace {

// Sum of squares of eight averages.
__device__ __forceinline__ double squares(const float *g) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(g[e], g[e], s);
    if (s > 1e-30f && s < 1e38f) return s;
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
    // large: top is 2^61 to 2^128; small: it is below 2^-49, down to 2^-149
    const float by = top > 1.0f ? 0x1p-70f : 0x1p100f;
    s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(g[e] * by, g[e] * by, s);
    return static_cast<double>(s) * (top > 1.0f ? 0x1p140 : 0x1p-200);
}

// One chunk: the elements [j0, j0 + 8) of the unit, cut to [0, numel).
template <int NW, int GD, int W>
__device__ __forceinline__ double chunk(const NormUnit<W> &u, int world, float c, int64_t j0, uint32_t &bad) {
    float g[8];
    if (u.vec && j0 >= 0 && j0 + 8 <= u.numel) {
        float acc[8];
        if constexpr (NW > 0) {
            rsa::GradRegs<NW, GD> r;
#pragma unroll
            for (int q = 0; q < NW; ++q) rsa::load_grad8<GD>(u.grads[q], j0, r.w[q]);
            rsa::widen8<GD>(r.w[0], acc);
#pragma unroll
            for (int q = 1; q < NW; ++q) {
                float f[8];
                rsa::widen8<GD>(r.w[q], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = __fadd_rn(acc[e], f[e]);
            }
        } else {
#pragma unroll 4
            for (int q = 0; q < world; ++q) {
                uint4 w[rsa::GradRegs<1, GD>::kWords];
                rsa::load_grad8<GD>(u.grads[q], j0, w);
                float f[8];
                rsa::widen8<GD>(w, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] = q == 0 ? f[e] : __fadd_rn(acc[e], f[e]);
            }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = __fmul_rn(acc[e], c);
        if (u.average != nullptr) {
            // read again by the update: kept in L2 where it fits
            *reinterpret_cast<float4 *>(u.average + j0) = make_float4(g[0], g[1], g[2], g[3]);
            *reinterpret_cast<float4 *>(u.average + j0 + 4) = make_float4(g[4], g[5], g[6], g[7]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t j = j0 + e;
            g[e] = 0.0f;
            if (j < 0 || j >= u.numel) continue;
            float acc = Dtype<GD>::load(u.grads[0], j);
            const int n = NW > 0 ? NW : world;
            for (int q = 1; q < n; ++q) acc = __fadd_rn(acc, Dtype<GD>::load(u.grads[q], j));
            g[e] = __fmul_rn(acc, c);
            if (u.average != nullptr) u.average[j] = g[e];
        }
    }
    const double s = squares(g);
    if (!isfinite(s)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) bad += isfinite(g[e]) ? 0u : 1u;
    }
    return s;
}

__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// The block's sum in thread 0.
__device__ __forceinline__ double block_sum(double x, double *shared) {
    x = warp_sum(x);
    if (threadIdx.x % 32 == 0) shared[threadIdx.x / 32] = x;
    __syncthreads();
    if (threadIdx.x < 32) x = warp_sum(threadIdx.x < kThreads / 32 ? shared[threadIdx.x] : 0.0);
    return x;
}

template <int NW, int GD, int W>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ NormArgs<W> a) {
    __shared__ double shared[kThreads / 32];
    __shared__ bool last;
    const NormUnit<W> &u = a.u[unit_of(a.u, a.n, blockIdx.x)];
    const int64_t first = (blockIdx.x - u.cta_begin) * (int64_t(8) * kThreads * a.per_thread) - u.lead;
    double sum = 0.0;
    uint32_t bad = 0;
#pragma unroll 2
    for (int i = 0; i < a.per_thread; ++i) {
        const int64_t j0 = first + 8 * (int64_t(i) * kThreads + threadIdx.x);
        if (j0 < u.numel) sum += chunk<NW, GD, W>(u, a.world, a.c, j0, bad);
    }
    if (a.out.nonfinite != nullptr) {
        const uint32_t total = __reduce_add_sync(0xffffffffu, bad);
        if (threadIdx.x % 32 == 0 && total) atomicAdd(a.out.nonfinite, total);
    }
    sum = block_sum(sum, shared);
    if (threadIdx.x == 0) {
        a.out.part[a.out.part_begin + blockIdx.x] = sum;
        __threadfence();
        last = atomicAdd(a.out.ticket, 1u) + 1 == static_cast<uint32_t>(a.out.part_count);
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    double all = 0.0;
    for (int64_t i = threadIdx.x; i < a.out.part_count; i += kThreads) all += __ldcg(a.out.part + i);
    all = block_sum(all, shared);
    if (threadIdx.x == 0) {
        *a.out.norm = static_cast<float>(sqrt(all) * static_cast<double>(a.out.scale));
        *a.out.ticket = 0;
    }
}

template <int NW, int W> fsdp_status launch(const NormArgs<W> &a, int dtype, int64_t grid, cudaStream_t s) {
    if (a.n < 1 || a.n > NormArgs<W>::kUnits || grid < 1 || grid > 0x7fffffff) return FSDP_ERR_INVALID_ARG;
    const unsigned n = static_cast<unsigned>(grid);
    switch (dtype) {
        case FSDP_BF16: norm_kernel<NW, FSDP_BF16, W><<<n, kThreads, 0, s>>>(a); break;
        case FSDP_F16: norm_kernel<NW, FSDP_F16, W><<<n, kThreads, 0, s>>>(a); break;
        default: norm_kernel<NW, FSDP_F32, W><<<n, kThreads, 0, s>>>(a);
    }
    return check_launch();
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
