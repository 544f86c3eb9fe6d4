// clip.cu -- the entry points over a list of gradient tensors:
// fsdp_grad_norm and fsdp_clip_grads. The model step's own norm and clipping
// (fsdp_clip_plan_*) are in abi.cu, with the units' validation.
#include "clip.cuh"

#include <math.h>
#include <string.h>

#include <algorithm>
#include <memory>
#include <new>
#include <vector>

namespace fsdp {
namespace clip {

// Chunks of a norm pass's thread: one while that leaves SMs idle, more as the
// work grows, so that a block's sum and its turn at the counter stay small
// beside its loads.
int norm_per_thread(int64_t elements) {
    const int64_t blocks = elements / (8 * kThreads), enough = int64_t(sm_count()) * 32;
    int n = 1;  // a power of two: whole groups of the chunks a thread loads together
    while (n < 64 && blocks / (2 * n) >= enough) n *= 2;
    return n;
}

namespace {

constexpr int64_t kHeader = 256;  // the counter

struct Span {
    uintptr_t lo, hi;
    int index;
};

int64_t total_of(const int64_t *numels, int n) {
    int64_t total = 0;
    for (int k = 0; k < n; ++k) total += numels[k];
    return total;
}

fsdp_status check_list(const void *const *tensors, const int64_t *numels, const int32_t *dtypes, int n) {
    if (n < 0 || (n > 0 && (!numels || !dtypes))) return FSDP_ERR_INVALID_ARG;
    int64_t total = 0;
    for (int k = 0; k < n; ++k) {
        if (!dtype_valid(dtypes[k])) return FSDP_ERR_UNSUPPORTED_DTYPE;
        if (numels[k] < 0 || numels[k] > (int64_t(1) << 56) - total) return FSDP_ERR_INVALID_ARG;
        total += numels[k];
        if (!tensors || numels[k] == 0) continue;
        if (!tensors[k]) return FSDP_ERR_INVALID_ARG;
        if (!aligned(tensors[k], static_cast<size_t>(dtype_size(dtypes[k])))) return FSDP_ERR_ALIGNMENT;
    }
    return FSDP_OK;
}

// Elements by which p lies past a 16-byte boundary.
int lead_of(const void *p, int dtype) {
    return static_cast<int>(reinterpret_cast<uintptr_t>(p) % 16) / dtype_size(dtype);
}

int64_t blocks_of(const int64_t *numels, int n) {
    const int per = norm_per_thread(total_of(numels, n));
    int64_t blocks = 0;
    for (int k = 0; k < n; ++k)
        if (numels[k] > 0) blocks += norm_ctas(numels[k], 7, per);
    return blocks;
}

template <class Body> fsdp_status guarded(Body &&body) noexcept {
    try {
        return body();
    } catch (...) {
        return FSDP_ERR_HOST_MEMORY;
    }
}

}  // namespace
}  // namespace clip
}  // namespace fsdp

using namespace fsdp;
using namespace fsdp::clip;

extern "C" {

FSDP_API fsdp_status fsdp_grad_norm_workspace(const int64_t *numels, const int32_t *dtypes, int n_tensors,
                                              int64_t *bytes_out) {
    if (!bytes_out) return FSDP_ERR_INVALID_ARG;
    const fsdp_status st = check_list(nullptr, numels, dtypes, n_tensors);
    if (st != FSDP_OK) return st;
    *bytes_out = kHeader + 8 * blocks_of(numels, n_tensors);
    return FSDP_OK;
}

FSDP_API fsdp_status fsdp_grad_norm(const void *const *tensors, const int64_t *numels, const int32_t *dtypes,
                                    int n_tensors, float scale, float *norm_out, void *workspace,
                                    int64_t workspace_bytes, void *stream) {
    return guarded([&]() -> fsdp_status {
        if (n_tensors > 0 && !tensors) return FSDP_ERR_INVALID_ARG;
        fsdp_status st = check_list(tensors, numels, dtypes, n_tensors);
        if (st != FSDP_OK) return st;
        if (!norm_out || !isfinite(scale)) return FSDP_ERR_INVALID_ARG;
        if (!aligned(norm_out, 4)) return FSDP_ERR_ALIGNMENT;
        const cudaStream_t s = static_cast<cudaStream_t>(stream);
        const int64_t blocks = blocks_of(numels, n_tensors);
        if (blocks == 0) return cuda_status(cudaMemsetAsync(norm_out, 0, 4, s));
        if (!workspace || workspace_bytes < kHeader + 8 * blocks || blocks > 0x7fffffff) return FSDP_ERR_INVALID_ARG;
        if (!aligned(workspace, 16)) return FSDP_ERR_ALIGNMENT;
        const size_t ws_bytes = static_cast<size_t>(kHeader + 8 * blocks);
        if (overlaps(norm_out, 4, workspace, ws_bytes)) return FSDP_ERR_INVALID_ARG;
        for (int k = 0; k < n_tensors; ++k) {
            const size_t bytes = static_cast<size_t>(numels[k]) * dtype_size(dtypes[k]);
            if (overlaps(tensors[k], bytes, workspace, ws_bytes) || overlaps(tensors[k], bytes, norm_out, 4))
                return FSDP_ERR_INVALID_ARG;
        }
        const int per = norm_per_thread(total_of(numels, n_tensors));
        // the blocks that will run: at each tensor's own alignment
        int64_t count = 0;
        for (int k = 0; k < n_tensors; ++k)
            if (numels[k] > 0) count += norm_ctas(numels[k], lead_of(tensors[k], dtypes[k]), per);
        std::unique_ptr<NormArgs<1>> a(new NormArgs<1>);  // up to 28 KB: not on the caller's stack
        a->out = NormOut();
        a->out.ticket = static_cast<uint32_t *>(workspace);
        a->out.part = reinterpret_cast<double *>(static_cast<uint8_t *>(workspace) + kHeader);
        a->out.part_count = count;
        a->out.scale = fabsf(scale);
        a->out.norm = norm_out;
        a->c = 1.0f;
        a->world = 1;
        a->per_thread = per;
        for (int dt = FSDP_F32; dt <= FSDP_F16; ++dt) {
            int64_t grid = 0;
            a->n = 0;
            for (int k = 0; k <= n_tensors; ++k) {
                if (k < n_tensors && (dtypes[k] != dt || numels[k] == 0)) continue;
                if (k < n_tensors) {
                    NormUnit<1> &u = a->u[a->n++];
                    u.grads[0] = tensors[k];
                    u.average = nullptr;
                    u.numel = numels[k];
                    u.cta_begin = grid;
                    u.lead = lead_of(tensors[k], dt);
                    u.vec = 1;
                    grid += norm_ctas(numels[k], u.lead, per);
                }
                if (a->n == NormArgs<1>::kUnits || (k == n_tensors && a->n > 0)) {
                    st = launch_norm(*a, dt, grid, s);
                    if (st != FSDP_OK) return st;
                    a->out.part_begin += grid;
                    a->n = 0;
                    grid = 0;
                }
            }
        }
        return FSDP_OK;
    });
}

FSDP_API fsdp_status fsdp_clip_grads(const void *const *tensors, void *const *outs, const int64_t *numels,
                                     const int32_t *dtypes, int n_tensors, const float *norm, float max_norm,
                                     float scale, void *stream) {
    return guarded([&]() -> fsdp_status {
        if (n_tensors > 0 && (!tensors || !outs)) return FSDP_ERR_INVALID_ARG;
        fsdp_status st = check_list(tensors, numels, dtypes, n_tensors);
        if (st == FSDP_OK) st = check_list(outs, numels, dtypes, n_tensors);
        if (st != FSDP_OK) return st;
        if (!norm || !(max_norm > 0.0f) || !isfinite(scale)) return FSDP_ERR_INVALID_ARG;
        if (!aligned(norm, 4)) return FSDP_ERR_ALIGNMENT;
        // written ranges are disjoint; a tensor overlaps a written range only
        // where that is the tensor itself
        std::vector<Span> w;
        bool in_place = true;
        for (int k = 0; k < n_tensors; ++k) {
            if (numels[k] == 0) continue;
            const uintptr_t bytes = static_cast<uintptr_t>(numels[k]) * dtype_size(dtypes[k]);
            const uintptr_t at = reinterpret_cast<uintptr_t>(outs[k]);
            if (overlaps(outs[k], bytes, norm, 4)) return FSDP_ERR_INVALID_ARG;
            in_place = in_place && outs[k] == tensors[k];
            w.push_back({at, at + bytes, k});
        }
        std::sort(w.begin(), w.end(), [](const Span &x, const Span &y) { return x.lo < y.lo; });
        for (size_t i = 1; i < w.size(); ++i)
            if (w[i].lo < w[i - 1].hi) return FSDP_ERR_INVALID_ARG;
        if (!in_place) {
            for (int k = 0; k < n_tensors; ++k) {
                if (numels[k] == 0) continue;
                const uintptr_t lo = reinterpret_cast<uintptr_t>(tensors[k]);
                const uintptr_t hi = lo + static_cast<uintptr_t>(numels[k]) * dtype_size(dtypes[k]);
                for (auto it = std::upper_bound(w.begin(), w.end(), lo,
                                                [](uintptr_t x, const Span &y) { return x < y.hi; });
                     it != w.end() && it->lo < hi; ++it)
                    if (it->index != k || outs[k] != tensors[k]) return FSDP_ERR_INVALID_ARG;
            }
        }
        std::unique_ptr<ScaleArgs> a(new ScaleArgs);
        a->norm = norm;
        a->max_norm = max_norm;
        a->scale = scale;
        a->in_place = in_place ? 1 : 0;
        // from the last tensor to the first, as the blocks run within a launch
        for (int dt = FSDP_F16; dt >= FSDP_F32; --dt) {
            std::vector<int> list;
            for (int k = 0; k < n_tensors; ++k)
                if (dtypes[k] == dt && numels[k] > 0) list.push_back(k);
            for (int end = static_cast<int>(list.size()); end > 0;) {
                const int begin = end > ScaleArgs::kUnits ? end - ScaleArgs::kUnits : 0;
                int64_t grid = 0;
                a->n = end - begin;
                for (int i = begin; i < end; ++i) {
                    const int k = list[static_cast<size_t>(i)];
                    ScaleUnit &u = a->u[i - begin];
                    u.src = tensors[k];
                    u.dst = outs[k];
                    u.numel = numels[k];
                    u.cta_begin = grid;
                    u.lead = lead_of(outs[k], dt);
                    u.vec = lead_of(tensors[k], dt) == u.lead;
                    grid += scale_ctas(numels[k], u.lead);
                }
                st = launch_scale(*a, dt, grid, static_cast<cudaStream_t>(stream));
                if (st != FSDP_OK) return st;
                end = begin;
            }
        }
        return FSDP_OK;
    });
}

}  // extern "C"
