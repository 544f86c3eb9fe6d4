// clip_scale.cu -- many tensors times one factor that is known on the device
// only: y = x * (scale * min(1, max_norm / (norm + 1e-6))), in place or into
// other tensors (views of a flat gradient buffer, at any alignment).
//
// Bound by HBM: one read, one write. The blocks run from the end of the list
// to its start: what the norm read last is still in L2 and is read first (50 M
// bf16 elements, norm and scaling, 61 us against 65 in the other order). 708 M
// bf16 elements: 396 us, 7.1 TB/s.
#include "clip.cuh"
#include "rsa_impl.cuh"

namespace fsdp {
namespace clip {
namespace {

template <int DT> __device__ __forceinline__ void store8(void *base, int64_t j, const float *v) {
    if constexpr (DT == FSDP_F32) {
        float *p = static_cast<float *>(base) + j;
        st_state(p, make_float4(v[0], v[1], v[2], v[3]));
        st_state(p + 4, make_float4(v[4], v[5], v[6], v[7]));
    } else {
        st_stream(static_cast<uint16_t *>(base) + j, make_uint4(pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]),
                                                                pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])));
    }
}

// The coherent form of load_grad8: in place, this kernel writes what it reads.
template <int DT> __device__ __forceinline__ void load8(const void *base, int64_t j, uint4 *w) {
    if constexpr (DT == FSDP_F32) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + j);
        w[0] = __ldcs(p);
        w[1] = __ldcs(p + 1);
    } else {
        w[0] = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + j));
    }
}

template <int DT, int CAP>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ ScaleArgsOf<CAP> a) {
    const int64_t cta = gridDim.x - 1 - blockIdx.x;
    const ScaleUnit &u = a.u[unit_of(a.u, a.n, cta)];
    const int64_t first = (cta - u.cta_begin) * (int64_t(8) * kThreads * kScaleChunks) - u.lead;
    constexpr int kWords = rsa::GradRegs<1, DT>::kWords;
    wait_previous();
    allow_next();
    const float f = __fmul_rn(a.scale, coefficient(*a.norm, a.max_norm));
    if (a.in_place && f == 1.0f) return;
    uint4 w[kScaleChunks][kWords];
#pragma unroll
    for (int i = 0; i < kScaleChunks; ++i) {
        const int64_t j = first + 8 * (int64_t(i) * kThreads + threadIdx.x);
        if (u.vec && j >= 0 && j + 8 <= u.numel) load8<DT>(u.src, j, w[i]);
    }
#pragma unroll
    for (int i = 0; i < kScaleChunks; ++i) {
        const int64_t j = first + 8 * (int64_t(i) * kThreads + threadIdx.x);
        if (j >= u.numel) continue;
        if (j >= 0 && j + 8 <= u.numel) {
            float v[8];
            if (u.vec) {
                rsa::widen8<DT>(w[i], v);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = Dtype<DT>::load(u.src, j + e);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __fmul_rn(v[e], f);
            store8<DT>(u.dst, j, v);
        } else {
            for (int e = 0; e < 8; ++e)
                if (j + e >= 0 && j + e < u.numel)
                    Dtype<DT>::store(u.dst, j + e, __fmul_rn(Dtype<DT>::load(u.src, j + e), f));
        }
    }
}

template <int CAP>
fsdp_status launch_capacity(const ScaleArgsOf<CAP> &a, int dtype, unsigned grid, cudaStream_t s) {
    auto kernel = dtype == FSDP_BF16  ? scale_kernel<FSDP_BF16, CAP>
                  : dtype == FSDP_F16 ? scale_kernel<FSDP_F16, CAP>
                                      : scale_kernel<FSDP_F32, CAP>;
    return launch_chained(kernel, grid, kThreads, 0, s, a);
}

}  // namespace

static_assert(sizeof(ScaleArgs) < 32764, "kernel parameter space");

fsdp_status launch_scale(const ScaleArgs &a, int dtype, int64_t grid, cudaStream_t s) {
    if (a.n < 1 || a.n > ScaleArgs::kUnits || grid < 1 || grid > 0x7fffffff) return FSDP_ERR_INVALID_ARG;
    if (a.n <= kFew) {
        ScaleArgsOf<kFew> few;
        few_of(a, few);
        return launch_capacity(few, dtype, static_cast<unsigned>(grid), s);
    }
    return launch_capacity(a, dtype, static_cast<unsigned>(grid), s);
}

}  // namespace clip
}  // namespace fsdp
