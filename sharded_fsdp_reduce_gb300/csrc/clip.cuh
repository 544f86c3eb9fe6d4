// clip.cuh -- internal arguments of the global gradient norm, the scaling of
// tensors to a largest norm, and the clipped model step.
#pragma once

#include <stddef.h>
#include <string.h>

#include "chain.cuh"

namespace fsdp {
namespace clip {

constexpr int kThreads = 256;
constexpr float kNormEps = 1e-6f;  // under the clipping quotient

// min(1, max_norm / (norm + eps)); a NaN norm gives NaN, an infinite one 0.
__device__ __forceinline__ float coefficient(float norm, float max_norm) {
    const float q = __fdiv_rn(max_norm, __fadd_rn(norm, kNormEps));
    return q >= 1.0f ? 1.0f : q;
}

// Descriptors travel by value in the kernel's parameter space; a launch takes
// as many as fit about 28 KB. Up to kFew go in a struct of that size: a short
// launch does not pay for copying the long one's.
constexpr int capacity(size_t descriptor) {
    const size_t n = 28000 / descriptor;
    return static_cast<int>(n < 512 ? n : 512);
}
constexpr int kFew = 16;

// The first a.n <= kFew descriptors of `a`, and all that lies before them.
template <class Args, class Few> void few_of(const Args &a, Few &few) {
    memcpy(static_cast<void *>(&few), &a, offsetof(Args, u));
    memcpy(static_cast<void *>(few.u), a.u, sizeof(a.u[0]) * static_cast<size_t>(a.n));
}

// ---------------------------------------------------------------- norm

// One tensor, or one unit's W rank gradients. Elements are visited in chunks
// of eight that start `lead` elements before the first, so that whole chunks
// lie on 16-byte boundaries of the gradients.
template <int W> struct NormUnit {
    const void *grads[W];
    float *average;      // fp32 averaged gradient, written when not NULL
    int64_t numel;
    int64_t cta_begin;   // the unit's first CTA in the launch
    int32_t lead;
    int32_t vec;         // whole chunks by 16-byte loads (and stores of the average)
};

// Where the blocks' sums go and how they end as the norm.
struct NormOut {
    double *part;        // one per CTA of all the call's launches
    uint32_t *ticket;    // zero between calls
    int64_t part_begin;  // this launch's first
    int64_t part_count;  // of the call
    float scale;         // |scale| of the result
    float *norm;
    uint32_t *nonfinite; // count of averaged values that are not finite, or NULL
};

template <int W, int CAP = capacity(sizeof(NormUnit<W>))> struct NormArgs {
    static constexpr int kUnits = CAP;
    NormOut out;
    float c;             // average = c * sum over the ranks
    int32_t n, world;
    int32_t per_thread;  // chunks per thread
    NormUnit<W> u[kUnits];
};

// Elements one CTA visits.
inline int64_t norm_span(int per_thread) { return int64_t(8) * kThreads * per_thread; }
inline int64_t norm_ctas(int64_t numel, int lead, int per_thread) {
    const int64_t span = norm_span(per_thread), n = (numel + lead + span - 1) / span;
    return n > 0 ? n : 1;
}

// Chunks per thread of a norm pass over this many elements.
int norm_per_thread(int64_t elements);

// W = 1, 2, 4, 8 ranks, or up to FSDP_MAX_WORLD of them (the last form).
fsdp_status launch_norm(const NormArgs<1> &a, int dtype, int64_t grid, cudaStream_t s);
fsdp_status launch_norm(const NormArgs<2> &a, int dtype, int64_t grid, cudaStream_t s);
fsdp_status launch_norm(const NormArgs<4> &a, int dtype, int64_t grid, cudaStream_t s);
fsdp_status launch_norm(const NormArgs<8> &a, int dtype, int64_t grid, cudaStream_t s);
fsdp_status launch_norm(const NormArgs<FSDP_MAX_WORLD> &a, int dtype, int64_t grid, cudaStream_t s);

// ---------------------------------------------------------------- scaling

struct ScaleUnit {
    const void *src;
    void *dst;
    int64_t numel;
    int64_t cta_begin;
    int32_t lead;    // of dst
    int32_t vec;     // src lies as dst does on 16 bytes
};

template <int CAP> struct ScaleArgsOf {
    static constexpr int kUnits = CAP;
    const float *norm;
    float max_norm, scale;
    int32_t n;
    int32_t in_place;  // every dst is its src: nothing to do for a factor of 1
    ScaleUnit u[kUnits];
};
using ScaleArgs = ScaleArgsOf<capacity(sizeof(ScaleUnit))>;

constexpr int kScaleChunks = 4;  // chunks per thread
inline int64_t scale_ctas(int64_t numel, int lead) { return norm_ctas(numel, lead, kScaleChunks); }

fsdp_status launch_scale(const ScaleArgs &a, int dtype, int64_t grid, cudaStream_t s);

// ---------------------------------------------------------------- clipped update

constexpr int kUpdateWorld = 4;  // ranks whose gradients are read again
constexpr int kUpdateFull = 8;   // gathered buffers written by the update

struct UpdateUnit {
    const void *grads[kUpdateWorld];  // the ranks' gradients, or the fp32 average alone
    void *full[kUpdateFull];
    float *master, *m, *v;
    void *out;
    int64_t numel;
    int64_t cta_begin;
    int32_t n_full;
    int32_t vec;
};

template <int CAP> struct UpdateArgsOf {
    static constexpr int kUnits = CAP;
    AdamScalars s;   // c: the average's factor, 1 for an average
    const float *norm;
    float max_norm;
    int32_t n, world;
    UpdateUnit u[kUnits];
};
using UpdateArgs = UpdateArgsOf<capacity(sizeof(UpdateUnit))>;

inline int64_t update_ctas(int64_t numel) { return (numel + 8 * kThreads - 1) / (8 * kThreads); }

// `host_state`: master, m and v in host memory (fp32 averages only).
fsdp_status launch_update_bf16(const UpdateArgs &a, int out_dtype, int64_t grid, cudaStream_t s);
fsdp_status launch_update_f16(const UpdateArgs &a, int out_dtype, int64_t grid, cudaStream_t s);
fsdp_status launch_update_f32(const UpdateArgs &a, int out_dtype, bool host_state, int64_t grid, cudaStream_t s);

// The unit of a CTA: the last one whose first CTA is at or before it.
template <class Unit> __device__ __forceinline__ int unit_of(const Unit *u, int n, int64_t cta) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (u[mid].cta_begin <= cta) {
            lo = mid;
        } else {
            hi = mid - 1;
        }
    }
    return lo;
}

}  // namespace clip
}  // namespace fsdp
