// The distillation loss's logits product (see loss_gemm.cuh).
#include "loss_gemm.cuh"

namespace fsdp {
namespace loss {

fsdp_status launch_soft_logits(Epilogue ep, bool f32, const CUtensorMap &a, const CUtensorMap &b,
                               const CUtensorMap &exponentials, const GemmArgs &g, cudaStream_t s) {
    if (ep == kStats)
        return f32 ? launch_kernel<0, 0, kStats, FSDP_F32, 3, true>(a, b, exponentials, g, s)
                   : launch_kernel<0, 0, kStats, FSDP_F16, 1, true>(a, b, exponentials, g, s);
    return f32 ? launch_kernel<0, 0, kExp, FSDP_F32, 3, true>(a, b, exponentials, g, s)
               : launch_kernel<0, 0, kExp, FSDP_F16, 1, true>(a, b, exponentials, g, s);
}

}  // namespace loss
}  // namespace fsdp
