// The head loss's gradient products with f32 outputs (see loss_gemm.cuh).
#include "loss_gemm.cuh"

namespace fsdp {
namespace loss {

fsdp_status launch_grad_f32(Orders o, const CUtensorMap &a, const CUtensorMap &b, const GemmArgs &g, cudaStream_t s) {
    // an fp32 head's gradients, or the fp32 partial sums of a 16-bit head's
    if (g.planes == 3)
        return o == kHiddenGrad ? launch_kernel<0, 1, kScale, FSDP_F32, 3>(a, b, a, g, s)
                                : launch_kernel<1, 1, kScale, FSDP_F32, 3>(a, b, a, g, s);
    return o == kHiddenGrad ? launch_kernel<0, 1, kScale, FSDP_F32, 1>(a, b, a, g, s)
                            : launch_kernel<1, 1, kScale, FSDP_F32, 1>(a, b, a, g, s);
}

}  // namespace loss
}  // namespace fsdp
