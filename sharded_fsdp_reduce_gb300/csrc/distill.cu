// distill.cu -- the loss of a linear head against a teacher's top logits:
// fsdp_head_distill.
//
//   p[t,k] = softmax over the row's entries k of a[t,k] / tau
//   q[t,v] = softmax over the vocabulary of l[t,v] / tau,   l = X W^T
//   loss_t = tau^2 sum_k p[t,k] (log p[t,k] - log q[t,id_k])
//   d[t,v] = tau (q[t,v] - sum over the entries k of token v of p[t,k])
//
// The products and the passes between them are the cross entropy's (loss.cu).
// What is particular to a teacher is done here, before them: each row's
// entries get their probabilities and are put in the order of their tokens,
// and a table tells where each span of 64 columns begins among them. A thread
// of the logits product's epilogue, which has a row's 64 logits of a span in
// registers, then finds its entries with one load, and leaves their logits in
// fp32: gathering the rows of W again would read top * dim values a token.
#include <math.h>

#include "loss.cuh"

namespace fsdp {
namespace loss {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xffffffffu;
constexpr uint64_t kNone = ~uint64_t(0);
constexpr int64_t kMostTop = FSDP_MAX_TEACHER_TOP;

__device__ __forceinline__ float teacher_logit(const SoftArgs &a, int64_t at) {
    switch (a.teacher_dtype) {
        case FSDP_BF16: return Dtype<FSDP_BF16>::load(a.teacher, at);
        case FSDP_F16: return Dtype<FSDP_F16>::load(a.teacher, at);
        default: return Dtype<FSDP_F32>::load(a.teacher, at);
    }
}
__device__ __forceinline__ int64_t teacher_token(const SoftArgs &a, int64_t at) {
    return a.wide ? static_cast<const int64_t *>(a.given)[at] : static_cast<const int32_t *>(a.given)[at];
}
__device__ __forceinline__ float logit_of(uint64_t entry) { return __uint_as_float(static_cast<uint32_t>(entry)); }
__device__ __forceinline__ uint64_t entry_of(uint64_t token, float logit) {
    return token << 32 | __float_as_uint(logit);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, o));
    return x;
}

// A warp puts its 32 N values in order: the i-th of lane l is the (32 i + l)-th.
template <int N> __device__ __forceinline__ void sort_warp(uint64_t (&x)[N]) {
    const int lane = threadIdx.x % 32;
#pragma unroll
    for (int run = 2; run <= 32 * N; run *= 2) {
#pragma unroll
        for (int apart = run / 2; apart >= 32; apart /= 2) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int o = i ^ (apart / 32);
                if (o < i) continue;
                const bool up = ((32 * i) & run) == 0;  // (run > 32: the same for all lanes)
                const uint64_t a = x[i], b = x[o];
                x[i] = (a > b) == up ? b : a;
                x[o] = (a > b) == up ? a : b;
            }
        }
#pragma unroll
        for (int apart = run / 2 < 32 ? run / 2 : 16; apart > 0; apart /= 2) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool up = ((32 * i + lane) & run) == 0, low = (lane & apart) == 0;
                const uint64_t a = x[i], b = __shfl_xor_sync(kAll, a, apart);
                x[i] = (a > b) == (up == low) ? b : a;
            }
        }
    }
}

// A warp per row of at most 32 N entries, N a power of two. An entry that does
// not count: token -1, or a logit of minus infinity, or one so small that its
// probability is 0. `late`: the kernel before this one on the stream does not
// touch what it reads or writes, and what came before that has ended; so this
// one waits for it last. Bound by the sort's exchanges where the entries are many:
// 4096 rows of 64 entries 16 us, of 256 31, of 512 48, of 1024 (32 a lane, in two
// registers each) 106.
template <int N>
__global__ void __launch_bounds__(kThreads)
    prepare_kernel(const __grid_constant__ SoftArgs a, int64_t row0, int64_t rows, bool late) {
    extern __shared__ uint64_t lists[];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    uint64_t *list = lists + warp * 32 * N;
    const int64_t r = int64_t(blockIdx.x) * kWarps + warp, row = row0 + r;
    if (!late) {
        wait_previous();
        allow_next();
    }
    if (r < rows) {
        int64_t token[N];
        float logit[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int k = 32 * i + lane;
            token[i] = k < a.top ? teacher_token(a, row * a.ld_given + k) : -1;
            logit[i] = k < a.top ? teacher_logit(a, row * a.ld_teacher + k) : -INFINITY;
        }
        bool bad = false, any = false;
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const bool of_vocab = token[i] >= 0 && token[i] < a.vocab;
            if (!of_vocab) {
                bad |= token[i] != -1;
                logit[i] = -INFINITY;
            }
            if (logit[i] != -INFINITY) {
                bad |= !(logit[i] < INFINITY);
                any = true;
                most = fmaxf(most, logit[i]);
            }
        }
        bad = __any_sync(kAll, bad);
        any = __any_sync(kAll, any);
        if (lane == 0) a.targets[row] = bad ? a.vocab : any ? 0 : kIgnored;
        if (a.ids != nullptr) {
            most = warp_max(most);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (logit[i] != -INFINITY) sum += expf((logit[i] - most) * a.inverse);
            sum = warp_sum(sum);
            const float log_sum = logf(sum), least = bad || !any ? INFINITY : 0.0f;
            uint64_t entry[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool counts = logit[i] != -INFINITY && expf((logit[i] - most) * a.inverse) / sum > least;
                entry[i] = counts ? entry_of(static_cast<uint64_t>(token[i]), logit[i]) : kNone;
            }
            sort_warp<N>(entry);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int k = 32 * i + lane;
                list[k] = entry[i];
                if (k < a.top) {
                    const bool there = entry[i] != kNone;
                    const float x = (logit_of(entry[i]) - most) * a.inverse;
                    a.ids[r * a.top + k] = there ? static_cast<int32_t>(entry[i] >> 32) : kNoEntry;
                    a.prob[r * a.top + k] = there ? make_float2(expf(x) / sum, x - log_sum) : make_float2(0.0f, 0.0f);
                }
            }
            __syncwarp();
            if (a.first != nullptr) {
                // entries before column 64 s, four spans of a lane at a time
                uint16_t *first = a.first + r * a.ld_first;
                for (int64_t s0 = lane; s0 <= a.spans; s0 += 4 * 32) {
                    int at[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int step = 32 * N / 2; step > 0; step /= 2)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            if (list[at[u] + step - 1] < static_cast<uint64_t>((s0 + 32 * u) * kSpan) << 32) at[u] += step;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint64_t limit = static_cast<uint64_t>((s0 + 32 * u) * kSpan) << 32;
                        if (s0 + 32 * u <= a.spans) first[s0 + 32 * u] = static_cast<uint16_t>(at[u] + (list[at[u]] < limit));
                    }
                }
            }
        }
    }
    if (late) {
        wait_previous();
        allow_next();
    }
}

// Few rows' logits become d, a thread per column.
__global__ void __launch_bounds__(kThreads) few_soft_kernel(const __grid_constant__ FewSoftArgs a) {
    const int64_t v = int64_t(blockIdx.x) * kThreads + threadIdx.x, row = blockIdx.y;
    wait_previous();
    allow_next();
    if (v >= a.vocab) return;
    float *at = a.logits + row * a.ld_logits + v;
    const int64_t target = a.targets[row];
    float d = 0.0f;
    if (target == 0) {
        const int32_t *ids = a.ids + row * a.top;
        int64_t lo = 0, hi = a.top;
        while (lo < hi) {
            const int64_t mid = (lo + hi) / 2;
            if (ids[mid] < v)
                lo = mid + 1;
            else
                hi = mid;
        }
        float p = 0.0f;
        for (; lo < a.top && ids[lo] == v; ++lo) p += a.prob[row * a.top + lo].x;
        const float2 state = a.row_state[row];
        d = exp2f((*at - state.x) * a.log2e) / state.y - p;
    } else if (target != kIgnored) {
        d = NAN;
    }
    *at = d;
}

// The call as the cross entropy's, whose targets are the workspace's.
fsdp_head_loss_args head_of(const fsdp_head_distill_args &d) {
    fsdp_head_loss_args a = {};
    a.hidden = d.hidden;
    a.ld_hidden = d.ld_hidden;
    a.weight = d.weight;
    a.ld_weight = d.ld_weight;
    a.tokens = d.tokens;
    a.vocab = d.vocab;
    a.dim = d.dim;
    a.band = d.band;
    a.dtype = d.dtype;
    a.reduction = d.reduction;
    a.grad_scale = d.grad_scale;
    a.loss = d.loss;
    a.token_loss = d.token_loss;
    a.d_hidden = d.d_hidden;
    a.ld_d_hidden = d.ld_d_hidden;
    a.d_weight = d.d_weight;
    a.ld_d_weight = d.ld_d_weight;
    a.wait_timeouts = d.wait_timeouts;
    return a;
}

fsdp_status check(const fsdp_head_distill_args *d) {
    if (!d || d->reserved != 0) return FSDP_ERR_INVALID_ARG;
    if (!dtype_valid(d->teacher_dtype)) return FSDP_ERR_UNSUPPORTED_DTYPE;
    if (d->id_bits != 32 && d->id_bits != 64) return FSDP_ERR_UNSUPPORTED_DTYPE;
    if (d->top < 1 || d->top > kMostTop || !(d->temperature >= 1e-3f && d->temperature <= 1e3f))
        return FSDP_ERR_INVALID_ARG;
    constexpr int64_t kMostLd = int64_t(1) << 34, kMostArea = int64_t(1) << 50;  // (products of sizes stay inside 64 bits)
    if (d->tokens < 0 || d->ld_teacher_logits < d->top || d->ld_teacher_logits > kMostLd || d->ld_teacher_ids < d->top ||
        d->ld_teacher_ids > kMostLd || d->tokens > kMostArea / d->ld_teacher_logits ||
        d->tokens > kMostArea / d->ld_teacher_ids || !isfinite(d->grad_scale * d->temperature))
        return FSDP_ERR_INVALID_ARG;
    const size_t entry = d->teacher_dtype == FSDP_F32 ? 4 : 2, token = d->id_bits / 8;
    const int64_t rows = d->tokens;
    const void *in[2] = {d->teacher_logits, d->teacher_ids};
    const size_t nin[2] = {rows > 0 ? ((rows - 1) * d->ld_teacher_logits + d->top) * entry : 0,
                           rows > 0 ? ((rows - 1) * d->ld_teacher_ids + d->top) * token : 0};
    const fsdp_status st = check_head(head_of(*d), in, nin, 2);
    if (st != FSDP_OK) return st;
    return aligned(in[0], entry) && aligned(in[1], token) ? FSDP_OK : FSDP_ERR_ALIGNMENT;
}

}  // namespace

namespace {

template <int N> fsdp_status prepare(const SoftArgs &a, int64_t row0, int64_t rows, bool late, cudaStream_t s) {
    constexpr size_t kShared = 32 * N * kWarps * sizeof(uint64_t);
    static PerDeviceOnce once;
    const int dev = current_device();
    if (!once.is_done(dev)) {
        const cudaError_t e = cudaFuncSetAttribute(prepare_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(kShared));
        if (e != cudaSuccess) return cuda_status(e);
        once.mark(dev);
    }
    return launch_chained(prepare_kernel<N>, static_cast<unsigned>((rows + kWarps - 1) / kWarps), kThreads, kShared, s, a,
                          row0, rows, late);
}

}  // namespace

fsdp_status launch_prepare(const SoftArgs &a, int64_t row0, int64_t rows, bool late, cudaStream_t s) {
    return a.top <= 32    ? prepare<1>(a, row0, rows, late, s)
           : a.top <= 64  ? prepare<2>(a, row0, rows, late, s)
           : a.top <= 128 ? prepare<4>(a, row0, rows, late, s)
           : a.top <= 256 ? prepare<8>(a, row0, rows, late, s)
           : a.top <= 512 ? prepare<16>(a, row0, rows, late, s)
                          : prepare<32>(a, row0, rows, late, s);
}

fsdp_status launch_few_soft(const FewSoftArgs &a, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>((a.vocab + kThreads - 1) / kThreads), static_cast<unsigned>(a.rows));
    return launch_chained(few_soft_kernel, grid, kThreads, 0, s, a);
}

}  // namespace loss
}  // namespace fsdp

using namespace fsdp;

extern "C" {

FSDP_API fsdp_status fsdp_head_distill_workspace(const fsdp_head_distill_args *args, int64_t *bytes_out) {
    const fsdp_status st = loss::check(args);
    return st == FSDP_OK ? loss::soft_workspace(loss::head_of(*args), args->top, bytes_out) : st;
}

FSDP_API fsdp_status fsdp_head_distill(const fsdp_head_distill_args *args, void *workspace, int64_t workspace_bytes,
                                       void *stream) {
    const fsdp_status st = loss::check(args);
    if (st != FSDP_OK) return st;
    loss::SoftArgs soft = {};
    soft.teacher = args->teacher_logits;
    soft.given = args->teacher_ids;
    soft.ld_teacher = args->ld_teacher_logits;
    soft.ld_given = args->ld_teacher_ids;
    soft.teacher_dtype = args->teacher_dtype;
    soft.wide = args->id_bits == 64;
    soft.top = args->top;
    soft.temperature = args->temperature;
    soft.inverse = static_cast<float>(1.0 / args->temperature);
    soft.log2e = static_cast<float>(1.44269504088896340736 / args->temperature);
    return loss::soft_run(loss::head_of(*args), soft, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
