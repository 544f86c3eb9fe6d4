// clip_update.cuh -- the clipped step's second pass: AdamW and cast (and the
// first all-gather) from the averaged gradient times the clipping coefficient.
//
//   g = (c * (G_0 + ... + G_{N-1})) * min(1, max_norm / (norm + 1e-6))
//   then the fused step's update, operation by operation (rsa_impl.cuh)
//
// so that a coefficient of 1 gives the unclipped step's bits. The norm is
// known only after every gradient has been read once, so something is read
// twice: the N gradients again where they are at most 8 bytes an element (N
// up to 4 in 16 bits, 2 in fp32), else the fp32 average that the norm pass
// has written (4 bytes written, 4 read). Eight ranks in bf16: 50 bytes an
// element against 58; two: 34 bytes against 38 (160 M elements 826 us against
// 919); four the same either way (1003 and 1011 us). Bound by HBM; launched over
// the units from the last to the first, since the norm pass leaves the end of
// its traffic in L2.
#pragma once

#include "clip.cuh"
#include "rsa_impl.cuh"

namespace fsdp {
namespace clip {

// SPLIT: the lane-interleaved chunks of state in host memory (rsa_impl.cuh);
// a CTA then has eight warp blocks of 256 elements, the same 2048 in all.
template <int NW, int GD, int OD, bool SPLIT, int CAP>
__global__ void __launch_bounds__(kThreads, SPLIT ? 1 : 3)
    update_kernel(const __grid_constant__ UpdateArgsOf<CAP> a) {
    const int64_t cta = gridDim.x - 1 - blockIdx.x;
    const UpdateUnit &u = a.u[unit_of(a.u, a.n, cta)];
    const int64_t first = (cta - u.cta_begin) * (8 * kThreads);
    const int64_t block = first + 256 * (threadIdx.x / 32);
    const int64_t j_lo = SPLIT ? block + 4 * (threadIdx.x % 32) : first + 8 * int64_t(threadIdx.x);
    const int64_t j_hi = j_lo + (SPLIT ? 128 : 4);
    RsaArgs r;  // the fields the shared code reads
    r.master = u.master;
    r.m = u.m;
    r.v = u.v;
    r.out = u.out;
    r.s = a.s;
    if (u.vec && (SPLIT ? block + 256 : j_lo + 8) <= u.numel) {
        // the norm pass before this kernel does not touch the state: its loads
        // need not wait for it
        const float4 p0 = ld_state(u.master + j_lo), p1 = ld_state(u.master + j_hi);
        const float4 m0 = ld_state(u.m + j_lo), m1 = ld_state(u.m + j_hi);
        const float4 v0 = ld_state(u.v + j_lo), v1 = ld_state(u.v + j_hi);
        wait_previous();
        allow_next();
        rsa::GradRegs<NW, GD> w;
#pragma unroll
        for (int q = 0; q < NW; ++q) rsa::load_grad8<GD, SPLIT>(u.grads[q], j_lo, j_hi, w.w[q]);
        r.s.c = coefficient(*a.norm, a.max_norm);
        float acc[8];
        rsa::widen8<GD>(w.w[0], acc);
#pragma unroll
        for (int q = 1; q < NW; ++q) {
            float f[8];
            rsa::widen8<GD>(w.w[q], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = __fadd_rn(acc[e], f[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = __fmul_rn(acc[e], a.s.c);
        rsa::finish_chunk<OD, true, SPLIT>(r, j_lo, j_hi, acc, p0, p1, m0, m1, v0, v1, u.full, u.n_full);
        return;
    }
    // elements after the last whole chunk, and units off 16 bytes
    wait_previous();
    allow_next();
    const float coef = coefficient(*a.norm, a.max_norm);
    for (int e = 0; e < 8; ++e) {
        const int64_t j = SPLIT ? block + 32 * e + threadIdx.x % 32 : j_lo + e;
        if (j >= u.numel) break;
        float acc = Dtype<GD>::load(u.grads[0], j);
        for (int q = 1; q < NW; ++q) acc = __fadd_rn(acc, Dtype<GD>::load(u.grads[q], j));
        float p = u.master[j], m = u.m[j], v = u.v[j];
        rsa::adamw(__fmul_rn(__fmul_rn(acc, a.s.c), coef), p, m, v, a.s);
        u.master[j] = p;
        u.m[j] = m;
        u.v[j] = v;
        Dtype<OD>::store(u.out, j, p);
        for (int d = 0; d < u.n_full; ++d) Dtype<OD>::store(u.full[d], j, p);
    }
}

template <int NW, int GD, bool SPLIT, int CAP>
fsdp_status launch_capacity(const UpdateArgsOf<CAP> &a, int out_dtype, unsigned grid, cudaStream_t s) {
    auto kernel = out_dtype == FSDP_BF16  ? update_kernel<NW, GD, FSDP_BF16, SPLIT, CAP>
                  : out_dtype == FSDP_F16 ? update_kernel<NW, GD, FSDP_F16, SPLIT, CAP>
                                          : update_kernel<NW, GD, FSDP_F32, SPLIT, CAP>;
    return launch_chained(kernel, grid, kThreads, 0, s, a);
}

template <int NW, int GD, bool SPLIT>
fsdp_status launch_out(const UpdateArgs &a, int out_dtype, int64_t grid, cudaStream_t s) {
    if (a.n < 1 || a.n > UpdateArgs::kUnits || grid < 1 || grid > 0x7fffffff) return FSDP_ERR_INVALID_ARG;
    if (a.n <= kFew) {
        UpdateArgsOf<kFew> few;
        few_of(a, few);
        return launch_capacity<NW, GD, SPLIT>(few, out_dtype, static_cast<unsigned>(grid), s);
    }
    return launch_capacity<NW, GD, SPLIT>(a, out_dtype, static_cast<unsigned>(grid), s);
}

// 16-bit gradients of up to four ranks.
template <int GD> fsdp_status launch_ranks(const UpdateArgs &a, int out_dtype, int64_t grid, cudaStream_t s) {
    switch (a.world) {
        case 1: return launch_out<1, GD, false>(a, out_dtype, grid, s);
        case 2: return launch_out<2, GD, false>(a, out_dtype, grid, s);
        case 3: return launch_out<3, GD, false>(a, out_dtype, grid, s);
        case 4: return launch_out<4, GD, false>(a, out_dtype, grid, s);
        default: return FSDP_ERR_INVALID_ARG;
    }
}

}  // namespace clip
}  // namespace fsdp
