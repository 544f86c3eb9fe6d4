// The head loss's gradient products with f16 outputs (see loss_gemm.cuh).
#include "loss_gemm.cuh"

namespace fsdp {
namespace loss {

fsdp_status launch_grad_f16(Orders o, const CUtensorMap &a, const CUtensorMap &b, const GemmArgs &g, cudaStream_t s) {
    return o == kHiddenGrad ? launch_kernel<0, 1, kScale, FSDP_F16, 1>(a, b, a, g, s)
                            : launch_kernel<1, 1, kScale, FSDP_F16, 1>(a, b, a, g, s);
}

}  // namespace loss
}  // namespace fsdp
