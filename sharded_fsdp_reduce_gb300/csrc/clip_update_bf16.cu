// The clipped update from bf16 gradients (see clip_update.cuh).
#include "clip_update.cuh"

namespace fsdp {
namespace clip {

fsdp_status launch_update_bf16(const UpdateArgs &a, int out_dtype, int64_t grid, cudaStream_t s) {
    return launch_ranks<FSDP_BF16>(a, out_dtype, grid, s);
}

}  // namespace clip
}  // namespace fsdp
