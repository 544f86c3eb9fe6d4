// loss_few.cu -- the head loss of a few rows (scoring single tokens): the
// logits' statistics by dot products, without tensor cores.
//
// A few rows read the whole weight for 2 to 16 operations an element: bound
// by HBM, and a 256-row tile would be nearly empty. A warp takes four
// vocabulary rows at a time, 16 bytes of each per lane and step, multiplies
// them with up to eight rows' hidden values (cached in L1: a few KB that all
// warps read) in fp32, and adds up over its lanes; more rows go in groups of
// eight whose blocks run side by side and share the weight in L2. Softmax
// statistics run along in registers; a block leaves one (largest, sum) per
// row, which the row kernel joins as it joins the spans of the matrix product.
// fp32 heads and rows off 16 bytes are read as they are, where the product
// would pack them first. One row of 50257 x 768 bf16: 10 us in the kernel where
// the weight is partly in L2, 20 where it is not (3.9 TB/s), 15.5 with the row
// kernel in a loop; of 32000 x 4096 49 us with it (5.4 TB/s).
//
// Gradients of up to eight rows of an fp32 head go the same way (few_dx_kernel,
// few_dw_kernel), from the logits that this pass leaves: the products' way
// packs the weight (10 bytes an element) for a tile that is mostly padding.
#include <float.h>
#include <math.h>

#include "loss.cuh"

namespace fsdp {
namespace loss {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32, kTake = 4;  // vocabulary rows of a warp's step
constexpr float kLog2e = 1.44269504088896340736f;

// e^x, or of x over a temperature; e^0 is exactly 1.
__device__ __forceinline__ float exp_of(float x, float log2e = kLog2e) { return exp2f(x * log2e); }

// sum * e^top with one more term e^logit.
__device__ __forceinline__ void take(float &top, float &sum, float logit, float log2e) {
    const float most = fmaxf(top, logit);
    sum = sum * exp_of(top - most, log2e) + exp_of(logit - most, log2e);
    top = most;
}
__device__ __forceinline__ void join(float &top, float &sum, float other_top, float other_sum, float log2e) {
    const float most = fmaxf(top, other_top);
    sum = sum * exp_of(top - most, log2e) + other_sum * exp_of(other_top - most, log2e);
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
    __shared__ int64_t target[R];
    constexpr int kSize = Dtype<DT>::kSize, E = 16 / kSize;
    constexpr int kTogether = R < 4 ? R : 4;  // hidden rows loaded together
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    wait_previous();
    allow_next();
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
    // the groups of R rows that read the same part of the weight run side by side
    const int64_t groups = (a.rows + R - 1) / R, block = blockIdx.x / groups, row0 = blockIdx.x % groups * R;
    const int rows = static_cast<int>(min(int64_t(R), a.rows - row0));
    const uint8_t *x = static_cast<const uint8_t *>(a.hidden) + row0 * a.ld_hidden * kSize;
    const uint8_t *w = static_cast<const uint8_t *>(a.weight);
    if (threadIdx.x < R) target[threadIdx.x] = threadIdx.x < rows && a.targets != nullptr ? a.targets[row0 + threadIdx.x] : -1;
    __syncthreads();
    float top[R], sum[R];
#pragma unroll
    for (int t = 0; t < R; ++t) {
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
                uint4 wv[kTake];
#pragma unroll
                for (int r = 0; r < kTake; ++r) wv[r] = load_whole<DT, E>(row[r], k);
                float f[kTake][E];
#pragma unroll
                for (int r = 0; r < kTake; ++r) widen<DT, E>(wv[r], f[r]);
#pragma unroll
                for (int t0 = 0; t0 < R; t0 += kTogether) {
                    uint4 xv[kTogether];
#pragma unroll
                    for (int i = 0; i < kTogether; ++i)
                        xv[i] = load_whole<DT, E>(x + (t0 + i < rows ? t0 + i : 0) * a.ld_hidden * kSize, k);
#pragma unroll
                    for (int i = 0; i < kTogether; ++i) {
                        float h[E];
                        widen<DT, E>(xv[i], h);
#pragma unroll
                        for (int r = 0; r < kTake; ++r)
#pragma unroll
                            for (int e = 0; e < E; ++e) acc[t0 + i][r] = fmaf(f[r][e], h[e], acc[t0 + i][r]);
                    }
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
        const int64_t v = v0 + lane / (32 / kTake);
        const bool first = lane % (32 / kTake) == 0;
#pragma unroll
        for (int t = 0; t < R; ++t) {
            const float logit = sum4(acc[t], lane);
            if (v < a.vocab) {
                if (first && v == target[t]) a.target_logit[row0 + t] = logit;
                if (first && a.logits != nullptr && t < rows) a.logits[(row0 + t) * a.ld_logits + v] = logit;
                take(top[t], sum[t], logit, a.log2e);
            }
        }
    }
#pragma unroll
    for (int t = 0; t < R; ++t) {
#pragma unroll
        for (int o = 16; o >= 32 / kTake; o >>= 1)
            join(top[t], sum[t], __shfl_xor_sync(0xffffffffu, top[t], o), __shfl_xor_sync(0xffffffffu, sum[t], o), a.log2e);
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
        for (int i = 1; i < kWarps; ++i) join(m, s, tops[i][t], sums[i][t], a.log2e);
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

// ---------------------------------------------------------------- gradients of a few fp32 rows

// d[t, v] from a stored logit.
__device__ __forceinline__ float d_of(const FewGradArgs &a, int64_t t, int64_t v) {
    if (t >= a.rows || v >= a.vocab) return 0.0f;
    if (a.soft) return a.logits[t * a.ld_logits + v];
    const int64_t y = a.targets[t];
    if (y == a.ignore) return 0.0f;
    if (y < 0 || y >= a.vocab) return NAN;
    const float2 state = a.row_state[t];
    const float p = exp_of(a.logits[t * a.ld_logits + v] - state.x) / state.y;
    return v == y ? p - 1.0f : p;
}

// Four consecutive values from k of a row of D (zeros past its end), and back.
template <bool VEC> __device__ __forceinline__ float4 load4(const float *row, int64_t k, int64_t D) {
    if (VEC && k + 4 <= D) return *reinterpret_cast<const float4 *>(row + k);
    return make_float4(k < D ? row[k] : 0.0f, k + 1 < D ? row[k + 1] : 0.0f, k + 2 < D ? row[k + 2] : 0.0f,
                       k + 3 < D ? row[k + 3] : 0.0f);
}
template <bool VEC> __device__ __forceinline__ void store4(float *row, int64_t k, int64_t D, float4 x) {
    if (VEC && k + 4 <= D) {
        *reinterpret_cast<float4 *>(row + k) = x;
    } else {
        if (k < D) row[k] = x.x;
        if (k + 1 < D) row[k + 1] = x.y;
        if (k + 2 < D) row[k + 2] = x.z;
        if (k + 3 < D) row[k + 3] = x.w;
    }
}

constexpr int kCols = 128;   // of a block: a warp's lanes times four
constexpr int kVocab = 64;   // vocabulary rows whose d is in shared memory at a time

// dX of R rows: a block adds up d W over its part of the vocabulary for 128
// columns, each warp every eighth vocabulary row; the warps' sums and, in the
// join kernel, the parts' add up in a fixed order.
template <int R, bool VEC> __global__ void __launch_bounds__(kThreads) few_dx_kernel(const FewGradArgs a) {
    __shared__ __align__(16) float d[kVocab][R];
    __shared__ __align__(16) float all[R][kCols];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t k = blockIdx.x * int64_t(kCols) + lane * 4, row0 = blockIdx.z * int64_t(R);
    const int64_t each = (a.vocab + gridDim.y - 1) / gridDim.y;
    const int64_t begin = blockIdx.y * each, end = min(begin + each, a.vocab);
    wait_previous();
    allow_next();
    float4 acc[R];
#pragma unroll
    for (int t = 0; t < R; ++t) acc[t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int64_t v0 = begin; v0 < end; v0 += kVocab) {
        __syncthreads();
        for (int i = threadIdx.x; i < kVocab * R; i += kThreads) {
            const int t = i / kVocab, v = i % kVocab;
            d[v][t] = v0 + v < end ? d_of(a, row0 + t, v0 + v) : 0.0f;
        }
        __syncthreads();
#pragma unroll 4
        for (int i = 0; i < kVocab / kWarps; ++i) {
            const int v = i * kWarps + warp;
            const float4 w = load4<VEC>(a.weight + min(v0 + v, a.vocab - 1) * a.ld_weight, k, a.dim);
            const bool live = v0 + v < end;
#pragma unroll
            for (int t = 0; t < R; ++t) {
                // a row past the part adds nothing, whatever its weight holds
                const float c = d[v][t];
                if (live) {
                    acc[t].x = fmaf(c, w.x, acc[t].x);
                    acc[t].y = fmaf(c, w.y, acc[t].y);
                    acc[t].z = fmaf(c, w.z, acc[t].z);
                    acc[t].w = fmaf(c, w.w, acc[t].w);
                }
            }
        }
    }
    for (int i = 0; i < kWarps; ++i) {
        __syncthreads();
        if (warp == i) {
#pragma unroll
            for (int t = 0; t < R; ++t) {
                float4 *p = reinterpret_cast<float4 *>(&all[t][lane * 4]);
                const float4 x = i > 0 ? *p : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                *p = make_float4(x.x + acc[t].x, x.y + acc[t].y, x.z + acc[t].z, x.w + acc[t].w);
            }
        }
    }
    __syncthreads();
    for (int t = warp; t < R && row0 + t < a.rows; t += kWarps)
        if (k < a.ld_part)  // padded to 64 columns
            *reinterpret_cast<float4 *>(a.part + (blockIdx.y * a.rows + row0 + t) * a.ld_part + k) =
                *reinterpret_cast<const float4 *>(&all[t][lane * 4]);
}

// dW: a block writes 64 vocabulary rows x 128 columns from all rows' d and
// hidden values in shared memory. Bound by the write.
template <bool VEC> __global__ void __launch_bounds__(kThreads) few_dw_kernel(const FewGradArgs a) {
    extern __shared__ __align__(16) float shared[];
    float *d = shared, *x = shared + a.rows * kVocab;  // [rows][64], [rows][128]
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t k = blockIdx.y * int64_t(kCols) + lane * 4, v0 = blockIdx.x * int64_t(kVocab);
    const int rows = static_cast<int>(a.rows);
    wait_previous();
    allow_next();
    for (int i = threadIdx.x; i < rows * kVocab; i += kThreads) d[i] = d_of(a, i / kVocab, v0 + i % kVocab);
    for (int t = warp; t < rows; t += kWarps) {
        // an ignored row has no gradient, whatever its hidden values are
        const bool counts = a.targets[t] != a.ignore;
        const float4 h = load4<VEC>(a.hidden + t * a.ld_hidden, k, a.dim);
        *reinterpret_cast<float4 *>(x + t * kCols + lane * 4) = counts ? h : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __syncthreads();
    float4 acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
    for (int t = 0; t < rows; ++t) {
        const float4 h = *reinterpret_cast<const float4 *>(x + t * kCols + lane * 4);
        const float4 lo = *reinterpret_cast<const float4 *>(d + t * kVocab + warp * 8);
        const float4 hi = *reinterpret_cast<const float4 *>(d + t * kVocab + warp * 8 + 4);
        const float c[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            acc[i].x = fmaf(c[i], h.x, acc[i].x);
            acc[i].y = fmaf(c[i], h.y, acc[i].y);
            acc[i].z = fmaf(c[i], h.z, acc[i].z);
            acc[i].w = fmaf(c[i], h.w, acc[i].w);
        }
    }
    const float f = *a.scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int64_t v = v0 + warp * 8 + i;
        if (v < a.vocab)
            store4<VEC>(a.d_weight + v * a.ld_d_weight, k, a.dim,
                        make_float4(acc[i].x * f, acc[i].y * f, acc[i].z * f, acc[i].w * f));
    }
}

template <int R> fsdp_status launch_dx(const FewGradArgs &a, cudaStream_t s) {
    const bool vec = aligned(a.weight, 16) && a.ld_weight % 4 == 0;
    const dim3 grid(static_cast<unsigned>((a.dim + kCols - 1) / kCols), static_cast<unsigned>(a.parts),
                    static_cast<unsigned>((a.rows + R - 1) / R));
    return launch_chained(vec ? few_dx_kernel<R, true> : few_dx_kernel<R, false>, grid, kThreads, 0, s, a);
}

}  // namespace

// Enough blocks to keep every SM's loads in flight, no more than there are
// vocabulary rows for.
int64_t few_blocks(int64_t vocab) {
    const int64_t most = int64_t(sm_count()) * 4, need = (vocab + 4 * kWarps - 1) / (4 * kWarps);
    return need < most ? need : most;
}

// Parts of the vocabulary in the hidden gradient: blocks for every SM, each
// with a few steps of 64 rows.
int64_t few_parts(int64_t vocab, int64_t dim) {
    const int64_t tiles = (dim + kCols - 1) / kCols;
    int64_t parts = (int64_t(sm_count()) * 4 + tiles - 1) / tiles;
    const int64_t most = (vocab + 4 * kVocab - 1) / (4 * kVocab);
    if (parts > most) parts = most;
    return parts < 1 ? 1 : parts > 256 ? 256 : parts;
}

fsdp_status launch_few(const FewArgs &a, int dtype, cudaStream_t s) {
    switch (dtype) {
        case FSDP_BF16: return launch_type<FSDP_BF16>(a, s);
        case FSDP_F16: return launch_type<FSDP_F16>(a, s);
        default: return launch_type<FSDP_F32>(a, s);
    }
}

fsdp_status launch_few_dx(const FewGradArgs &a, cudaStream_t s) {
    return a.rows <= 4 ? launch_dx<4>(a, s) : launch_dx<8>(a, s);
}

fsdp_status launch_few_dw(const FewGradArgs &a, cudaStream_t s) {
    const bool vec = aligned(a.hidden, 16) && a.ld_hidden % 4 == 0 && aligned(a.d_weight, 16) && a.ld_d_weight % 4 == 0;
    const size_t smem = static_cast<size_t>(a.rows) * (kVocab + kCols) * 4;
    const dim3 grid(static_cast<unsigned>((a.vocab + kVocab - 1) / kVocab),
                    static_cast<unsigned>((a.dim + kCols - 1) / kCols));
    return launch_chained(vec ? few_dw_kernel<true> : few_dw_kernel<false>, grid, kThreads, smem, s, a);
}

}  // namespace loss
}  // namespace fsdp
