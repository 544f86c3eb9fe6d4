// loss_few.cu -- the head loss of a few rows (scoring single tokens): the
// logits' statistics by dot products, without tensor cores.
//
// A few rows read the whole weight for 2 to 16 operations an element: bound
// by HBM, and a 256-row tile would be nearly empty. A warp takes four
// vocabulary rows at a time, 16 bytes of each per lane and step, multiplies
// them with up to eight rows' hidden values (cached in L1: a few KB that all
// warps read) in fp32, and adds up over its lanes; more rows go in groups of
// eight whose blocks run side by side and share the weight in L2. Softmax
// statistics run along in registers; a block leaves one (reference, sum) per
// row, which the row kernel joins as it joins the spans of the matrix product.
// fp32 heads and rows off 16 bytes are read as they are, where the product
// would pack them first. One row of 50257 x 768 bf16: 12 us in the kernel (6.4
// TB/s); of 32000 x 4096 49 us with the row kernel (5.4 TB/s).
#include <float.h>
#include <math.h>

#include "loss.cuh"

namespace fsdp {
namespace loss {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kTake = 4;  // vocabulary rows of a warp's step
constexpr float kLog2e = 1.44269504088896340736f;

// sum * 2^top with one more term 2^x.
__device__ __forceinline__ void take(float &top, float &sum, float x) {
    const float most = fmaxf(top, x);
    sum = sum * exp2f(top - most) + exp2f(x - most);
    top = most;
}
__device__ __forceinline__ void join(float &top, float &sum, float other_top, float other_sum) {
    const float most = fmaxf(top, other_top);
    sum = sum * exp2f(top - most) + other_sum * exp2f(other_top - most);
    top = most;
}

// Lane group 8 r .. 8 r + 7 gets the sum over all lanes of v[r].
__device__ __forceinline__ float sum4(const float *v, int lane) {
    const bool hi = lane & 16, mid = lane & 8;
    float a = hi ? v[2] : v[0], b = hi ? v[3] : v[1];
    a += __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
    b += __shfl_xor_sync(0xffffffffu, hi ? v[1] : v[3], 16);
    float c = mid ? b : a;
    c += __shfl_xor_sync(0xffffffffu, mid ? a : b, 8);
#pragma unroll
    for (int o = 4; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
    return c;
}

// E consecutive values from k of a row, as fp32: one 16-byte load, or E of
// them cut at the row's end.
template <int DT, int E> __device__ __forceinline__ uint4 load_whole(const uint8_t *base, int64_t k) {
    return __ldg(reinterpret_cast<const uint4 *>(base + k * Dtype<DT>::kSize));
}
template <int DT, int E> __device__ __forceinline__ void widen(const uint4 &w, float *f) {
    if constexpr (DT == FSDP_F32) {
        f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y);
        f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
    } else {
        unpack8<DT>(w, f);
    }
}
template <int DT, int E>
__device__ __forceinline__ void load_cut(const uint8_t *base, int64_t k, int64_t D, float *f) {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = k + e < D ? Dtype<DT>::load(base, k + e) : 0.0f;
}

template <int DT, int R, bool VEC> __global__ void __launch_bounds__(kThreads, 2) few_kernel(const FewArgs a) {
    __shared__ float tops[kWarps][R], sums[kWarps][R];
    constexpr int kSize = Dtype<DT>::kSize, E = 16 / kSize;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    wait_previous();
    allow_next();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    // the groups of R rows that read the same part of the weight run side by side
    const int64_t groups = (a.rows + R - 1) / R, block = blockIdx.x / groups, row0 = blockIdx.x % groups * R;
    const int rows = static_cast<int>(min(int64_t(R), a.rows - row0));
    const uint8_t *x = static_cast<const uint8_t *>(a.hidden) + row0 * a.ld_hidden * kSize;
    const uint8_t *w = static_cast<const uint8_t *>(a.weight);
    int64_t y[R];
    float top[R], sum[R];
#pragma unroll
    for (int t = 0; t < R; ++t) {
        y[t] = t < rows ? a.targets[row0 + t] : -1;
        top[t] = -FLT_MAX;
        sum[t] = 0.0f;
    }
    for (int64_t v0 = kTake * (block * kWarps + warp); v0 < a.vocab; v0 += kTake * kWarps * a.blocks) {
        const uint8_t *row[kTake];
#pragma unroll
        for (int r = 0; r < kTake; ++r) row[r] = w + min(v0 + r, a.vocab - 1) * a.ld_weight * kSize;
        float acc[R][kTake] = {};
        int64_t k = lane * E;
        if constexpr (VEC) {
            // whole steps of the warp, no bounds in them: the loads of two go out together
            const int64_t whole = a.dim / (32 * E) * (32 * E);
#pragma unroll 2
            for (; k < whole; k += 32 * E) {
                uint4 wv[kTake], xv[R];
#pragma unroll
                for (int r = 0; r < kTake; ++r) wv[r] = load_whole<DT, E>(row[r], k);
#pragma unroll
                for (int t = 0; t < R; ++t)
                    xv[t] = load_whole<DT, E>(x + (t < rows ? t : 0) * a.ld_hidden * kSize, k);
                float f[kTake][E];
#pragma unroll
                for (int r = 0; r < kTake; ++r) widen<DT, E>(wv[r], f[r]);
#pragma unroll
                for (int t = 0; t < R; ++t) {
                    float h[E];
                    widen<DT, E>(xv[t], h);
#pragma unroll
                    for (int r = 0; r < kTake; ++r)
#pragma unroll
                        for (int e = 0; e < E; ++e) acc[t][r] = fmaf(f[r][e], h[e], acc[t][r]);
                }
            }
        }
#pragma unroll 1
        for (; k < a.dim; k += 32 * E) {
            float f[kTake][E];
#pragma unroll
            for (int r = 0; r < kTake; ++r) load_cut<DT, E>(row[r], k, a.dim, f[r]);
#pragma unroll
            for (int t = 0; t < R; ++t) {
                float h[E];
                load_cut<DT, E>(x + (t < rows ? t : 0) * a.ld_hidden * kSize, k, a.dim, h);
#pragma unroll
                for (int r = 0; r < kTake; ++r)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[t][r] = fmaf(f[r][e], h[e], acc[t][r]);
            }
        }
        const int64_t v = v0 + lane / 8;
#pragma unroll
        for (int t = 0; t < R; ++t) {
            const float logit = sum4(acc[t], lane);
            if (v < a.vocab) {
                if (v == y[t] && lane % 8 == 0) a.target_logit[row0 + t] = logit;
                take(top[t], sum[t], logit * kLog2e);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < R; ++t) {
#pragma unroll
        for (int o = 16; o >= 8; o >>= 1)
            join(top[t], sum[t], __shfl_xor_sync(0xffffffffu, top[t], o), __shfl_xor_sync(0xffffffffu, sum[t], o));
        if (lane == 0) {
            tops[warp][t] = top[t];
            sums[warp][t] = sum[t];
        }
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < rows) {
        float m = tops[0][t], s = sums[0][t];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) join(m, s, tops[i][t], sums[i][t]);
        a.off[block * a.ld_rows + row0 + t] = m;
        a.sum[block * a.ld_rows + row0 + t] = s;
    }
}

template <int DT, int R> fsdp_status launch_rows(const FewArgs &a, cudaStream_t s) {
    const bool vec = aligned(a.hidden, 16) && aligned(a.weight, 16) && a.ld_hidden * Dtype<DT>::kSize % 16 == 0 &&
                     a.ld_weight * Dtype<DT>::kSize % 16 == 0;
    return launch_chained(vec ? few_kernel<DT, R, true> : few_kernel<DT, R, false>,
                          static_cast<unsigned>(a.blocks * ((a.rows + R - 1) / R)), kThreads, 0, s, a);
}

template <int DT> fsdp_status launch_type(const FewArgs &a, cudaStream_t s) {
    return a.rows <= 1   ? launch_rows<DT, 1>(a, s)
           : a.rows <= 2 ? launch_rows<DT, 2>(a, s)
           : a.rows <= 4 ? launch_rows<DT, 4>(a, s)
                         : launch_rows<DT, 8>(a, s);
}

}  // namespace

// Enough blocks to keep every SM's loads in flight, no more than there are
// vocabulary rows for.
int64_t few_blocks(int64_t vocab) {
    const int64_t most = int64_t(sm_count()) * 4, need = (vocab + kTake * kWarps - 1) / (kTake * kWarps);
    return need < most ? need : most;
}

fsdp_status launch_few(const FewArgs &a, int dtype, cudaStream_t s) {
    switch (dtype) {
        case FSDP_BF16: return launch_type<FSDP_BF16>(a, s);
        case FSDP_F16: return launch_type<FSDP_F16>(a, s);
        default: return launch_type<FSDP_F32>(a, s);
    }
}

}  // namespace loss
}  // namespace fsdp
