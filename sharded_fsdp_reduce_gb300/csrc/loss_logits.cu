// The head loss's logits product, and the self-test of the products' bounded
// waits (see loss_gemm.cuh).
#include "loss_gemm.cuh"

namespace fsdp {
namespace loss {

fsdp_status launch_logits(Epilogue ep, bool f32, const CUtensorMap &a, const CUtensorMap &b,
                          const CUtensorMap &exponentials, const GemmArgs &g, cudaStream_t s) {
    if (ep == kStats)
        return f32 ? launch_kernel<0, 0, kStats, FSDP_F32, 3>(a, b, exponentials, g, s)
                   : launch_kernel<0, 0, kStats, FSDP_F16, 1>(a, b, exponentials, g, s);
    return f32 ? launch_kernel<0, 0, kExp, FSDP_F32, 3>(a, b, exponentials, g, s)
               : launch_kernel<0, 0, kExp, FSDP_F16, 1>(a, b, exponentials, g, s);
}

namespace {

constexpr int kWaitingWarps = 4;

__global__ void __launch_bounds__(32 * (kWaitingWarps + 1))
    wait_check_kernel(long long limit, long long arrive_after, int32_t *outcomes, uint32_t *timeouts) {
    __shared__ Barriers b;
    if (threadIdx.x == 0) {
        tma::mbar_init(&b.full[0], 1);
        b.gave_up = 0;
        tma::fence_mbar_init();
    }
    __syncthreads();
    if (threadIdx.x < 32 * kWaitingWarps) {
        outcomes[threadIdx.x] = wait(&b.full[0], 0, &b, timeouts, limit);
    } else if (threadIdx.x % 32 == 0 && arrive_after >= 0) {
        const long long t0 = clock64();
        while (clock64() - t0 < arrive_after) {
        }
        tma::mbar_arrive(&b.full[0]);
    }
    __syncthreads();
}

}  // namespace

fsdp_status launch_wait_check(long long limit, long long arrive_after, int32_t *outcomes, uint32_t *timeouts,
                              cudaStream_t s) {
    wait_check_kernel<<<1, 32 * (kWaitingWarps + 1), 0, s>>>(limit, arrive_after, outcomes, timeouts);
    return check_launch();
}

}  // namespace loss
}  // namespace fsdp
