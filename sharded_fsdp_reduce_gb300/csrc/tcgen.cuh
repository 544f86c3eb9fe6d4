// tcgen.cuh -- inline-PTX wrappers of the fifth-generation tensor cores
// (tcgen05, accumulators in tensor memory) and of the tiled TMA copies, as the
// CTA-pair products use them: two CTAs of a cluster hold one half each of
// both operand tiles, the even CTA issues the instructions for both, and each
// CTA's tensor memory holds its half of the accumulator's rows.
//
// Rules the callers keep: the innermost tile coordinate times the element
// size is a multiple of 16 bytes; no store starts at a negative coordinate;
// both operands of one instruction have the same 16-bit type; every wait is
// bounded.
#pragma once

#include <cuda.h>  // CUtensorMap
#include <stdint.h>

#include "tma.cuh"

namespace fsdp {
namespace tc {

using tma::smem_addr;

// ---------------------------------------------------------------- cluster

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// The address of the same shared-memory object in the CTA of rank `rank`.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// Arrive on a barrier of either CTA (a shared::cluster address). What it
// orders are tensor-memory reads that a tcgen05 fence has closed: the CTA
// scope of the default form is enough, and a cluster-scope release would
// wait for this thread's global stores.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---------------------------------------------------------------- tiled TMA

// Load one box at (x, y, z) into this CTA's shared memory (dst: its address
// there); the bytes count on `bar`, a shared::cluster address (the pair's even
// CTA's barrier).
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void store_tile(const CUtensorMap *map, int x, int y, int z, const void *src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map),
                 "r"(x), "r"(y), "r"(z), "r"(smem_addr(src))
                 : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---------------------------------------------------------------- tensor memory

// One warp of each CTA of the pair allocates / frees `cols` columns together.
__device__ __forceinline__ void alloc_pair(uint32_t *dst, uint32_t cols) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}

__device__ __forceinline__ void free_pair(uint32_t addr, uint32_t cols) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

// 32 columns of the warp's 32 lanes: thread l gets lane l's values, complete
// on return.
__device__ __forceinline__ void load_cols32(uint32_t addr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---------------------------------------------------------------- the products

// Shared-memory operand descriptor, 128-byte swizzle, 1024-byte atoms of
// eight 128-byte rows. `lead` and `stride` in bytes: K-major operands (rows of
// 64 K elements) use stride between groups of eight rows; MN-major ones (rows
// of 64 M or N elements) use stride between groups of eight K and lead
// between blocks of 64 M or N. The address is in the low word, which is all
// that changes from one product to the next.
__device__ __forceinline__ uint32_t operand_low(uint32_t addr, uint32_t lead) {
    return ((addr & 0x3ffff) >> 4) | ((lead >> 4) << 16);
}
constexpr uint32_t operand_high(uint32_t stride) { return (stride >> 4) | (1u << 14) | (2u << 29); }

// Instruction descriptor of kind::f16: fp32 accumulator, operand type 0 (fp16)
// or 1 (bf16) for both, majorness per operand (1: MN-major).
constexpr uint32_t instruction(int type, int a_mn, int b_mn, int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(type) << 7) | (static_cast<uint32_t>(type) << 10) |
           (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// D (+)= A B over K = 16 by the pair; one thread of the even CTA issues it.
// Operands as the low words of their descriptors; `high` is both's high word.
__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t b, uint32_t high, uint32_t idesc,
                                         bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "mov.b64 x, {%1, %3};\n\t"
        "mov.b64 y, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(high), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}

// Arrive on the barrier at this offset in both CTAs once every product issued
// so far has finished.
__device__ __forceinline__ void commit_pair(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// True in one thread of the (whole) warp: always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

}  // namespace tc
}  // namespace fsdp
