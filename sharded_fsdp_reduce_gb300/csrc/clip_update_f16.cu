// The clipped update from f16 gradients (see clip_update.cuh).
#include "clip_update.cuh"

namespace fsdp {
namespace clip {

fsdp_status launch_update_f16(const UpdateArgs &a, int out_dtype, int64_t grid, cudaStream_t s) {
    return launch_ranks<FSDP_F16>(a, out_dtype, grid, s);
}

}  // namespace clip
}  // namespace fsdp
