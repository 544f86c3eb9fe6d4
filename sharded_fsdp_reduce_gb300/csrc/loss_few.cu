// loss_few.cu -- the head loss of a few rows (scoring single tokens): the
// logits' statistics by dot products, without tensor cores.
//
// Up to eight rows read the whole weight for 2 to 16 operations an element:
// bound by HBM, and a 256-row tile would be nearly empty. A warp takes four
// vocabulary rows at a time, 16 bytes of each per lane and step, multiplies
// them with every row's hidden values (cached in L1: a few KB that all warps
// read) in fp32, and adds up over its lanes. Softmax statistics run along in
// registers; a block leaves one (reference, sum) per row, which the row
// kernel joins as it joins the spans of the matrix product. fp32 heads and
// rows off 16 bytes are read as they are, where the product would pack them
// first. One row of 50257 x 768 bf16: 12 us (6.4 TB/s) against 24 for the product.
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

// E consecutive values from k of a row of D, as fp32 (zeros past the end).
template <int DT, bool VEC, int E>
__device__ __forceinline__ void load(const void *base, int64_t k, int64_t D, float *f) {
    if (VEC && k + E <= D) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + k * Dtype<DT>::kSize));
        if constexpr (DT == FSDP_F32) {
            f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y);
            f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
        } else {
            unpack8<DT>(w, f);
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = k + e < D ? Dtype<DT>::load(base, k + e) : 0.0f;
    }
}

template <int DT, int R, bool VEC> __global__ void __launch_bounds__(kThreads) few_kernel(const FewArgs a) {
    __shared__ float tops[kWarps][R], sums[kWarps][R];
    constexpr int kSize = Dtype<DT>::kSize, E = 16 / kSize;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    wait_previous();
    allow_next();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    const uint8_t *x = static_cast<const uint8_t *>(a.hidden), *w = static_cast<const uint8_t *>(a.weight);
    int64_t y[R];
    float top[R], sum[R];
#pragma unroll
    for (int t = 0; t < R; ++t) {
        y[t] = t < a.rows ? a.targets[t] : -1;
        top[t] = -FLT_MAX;
        sum[t] = 0.0f;
    }
    for (int64_t v0 = kTake * (int64_t(blockIdx.x) * kWarps + warp); v0 < a.vocab;
         v0 += int64_t(kTake) * kWarps * gridDim.x) {
        const uint8_t *row[kTake];
#pragma unroll
        for (int r = 0; r < kTake; ++r) row[r] = w + min(v0 + r, a.vocab - 1) * a.ld_weight * kSize;
        float acc[R][kTake] = {};
#pragma unroll 3
        for (int64_t k = lane * E; k < a.dim; k += 32 * E) {
            float f[kTake][E];
#pragma unroll
            for (int r = 0; r < kTake; ++r) load<DT, VEC, E>(row[r], k, a.dim, f[r]);
#pragma unroll
            for (int t = 0; t < R; ++t) {
                float h[E];
                load<DT, VEC, E>(x + (t < a.rows ? t : 0) * a.ld_hidden * kSize, k, a.dim, h);
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
                if (v == y[t] && lane % 8 == 0) a.target_logit[t] = logit;
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
    if (t < R && t < a.rows) {
        float m = tops[0][t], s = sums[0][t];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) join(m, s, tops[i][t], sums[i][t]);
        a.off[blockIdx.x * a.ld_rows + t] = m;
        a.sum[blockIdx.x * a.ld_rows + t] = s;
    }
}

template <int DT, int R> fsdp_status launch_rows(const FewArgs &a, cudaStream_t s) {
    const bool vec = aligned(a.hidden, 16) && aligned(a.weight, 16) && a.ld_hidden * Dtype<DT>::kSize % 16 == 0 &&
                     a.ld_weight * Dtype<DT>::kSize % 16 == 0;
    return launch_chained(vec ? few_kernel<DT, R, true> : few_kernel<DT, R, false>,
                          static_cast<unsigned>(a.blocks), kThreads, 0, s, a);
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
