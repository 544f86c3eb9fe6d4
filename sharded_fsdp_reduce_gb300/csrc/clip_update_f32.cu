// The clipped update from fp32 averages, or fp32 gradients of up to two ranks
// (see clip_update.cuh).
#include "clip_update.cuh"

namespace fsdp {
namespace clip {

static_assert(sizeof(UpdateArgs) < 32764, "kernel parameter space");

fsdp_status launch_update_f32(const UpdateArgs &a, int out_dtype, bool host_state, int64_t grid, cudaStream_t s) {
    if (host_state) {
        if (a.world != 1) return FSDP_ERR_INVALID_ARG;
        return launch_out<1, FSDP_F32, true>(a, out_dtype, grid, s);
    }
    switch (a.world) {
        case 1: return launch_out<1, FSDP_F32, false>(a, out_dtype, grid, s);
        case 2: return launch_out<2, FSDP_F32, false>(a, out_dtype, grid, s);
        default: return FSDP_ERR_INVALID_ARG;
    }
}

}  // namespace clip
}  // namespace fsdp
