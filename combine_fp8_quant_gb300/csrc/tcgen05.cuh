// tcgen05.cuh -- thin wrappers of the sm_103a instructions the matrix kernels
// use: clusters, tensor-map (TMA) loads, tensor memory and tcgen05.mma.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace moeperm {

// ---------------------------------------------------------------------------
// Clusters
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One lane of a converged warp (the instruction's operands stay warp-uniform).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// ---------------------------------------------------------------------------
// CTA pairs. Address of the same shared-memory offset in CTA `rank` of the
// cluster, and an arrival on an mbarrier there. What the arrival hands over is
// read by the asynchronous proxy or by tcgen05 instructions in the arriving CTA,
// so a proxy fence or tcgen05.fence before it orders it; release at cluster scope
// on top of that cost about 2000 cycles an arrival.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t map_to_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_arrive_mapped(uint32_t mapped) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(mapped) : "memory");
}

// 16 bytes to another CTA's shared memory, counted on an mbarrier there (both
// mapped addresses).
__device__ __forceinline__ void store_async16(uint32_t mapped, uint32_t a, uint32_t b, uint32_t c, uint32_t d,
                                              uint32_t mapped_bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
               ::"r"(mapped), "r"(a), "r"(b), "r"(c), "r"(d), "r"(mapped_bar)
               : "memory");
}

// ---------------------------------------------------------------------------
// Tensor-map loads (global -> this CTA's shared memory). The mbarrier that
// counts the bytes may be the pair's other CTA's (a mapped address).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
               " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
               " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2,
                                            int c3, int c4) {
  asm volatile("cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
               " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst), "l"(m), "r"(bar), "r"(c0), "r"(c1),
               "r"(c2), "r"(c3), "r"(c4)
               : "memory");
}

// ---------------------------------------------------------------------------
// Tensor memory
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t cols) {  // one whole warp
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t cols) {  // the same warp
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 32 columns of this warp's 32 lanes (lane = lane, register j = column j).
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
// 32 columns of 16 lanes as 8x8 blocks: register 4 i + h + 2 g of lane l holds
// lane l / 4 + 8 g, column 8 i + 2 (l % 4) + h (the fragments stmatrix takes).
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
// Four 8x8 blocks of 16-bit fragments, stored (loaded) transposed: lane l gives
// the shared-memory address of row l % 8 of block l / 8.
__device__ __forceinline__ void stmatrix_trans(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t saddr, uint32_t (&v)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(saddr)
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------------------
// Matrix products. Operands are described by 64-bit shared-memory descriptors
// in the 128-byte swizzle that the tensor maps write.
//   K-major   128 bytes of the reduction per row, 8 rows = 1024 bytes, the next
//             8 rows 1024 bytes on; +32 bytes steps one instruction's reduction.
//   MN-major  64 16-bit elements of the row dimension per 128-byte line, one
//             line per reduction index, 8 lines = 1024 bytes; the next 64 elements
//             `atom` bytes on; +2048 bytes steps 16 reduction indices.
// ---------------------------------------------------------------------------
// A descriptor's high word (8-line stride, version, swizzle) is a constant; its
// low word is the address / 16 and, for MN-major operands, the 64-element
// stride / 16 in the upper half, so one 32-bit addition steps it.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t atom) {
  return ((saddr & 0x3FFFF) >> 4) | ((atom >> 4) << 16);
}
// Unswizzled rows of 16 bytes, 8 rows = 128 bytes (the scale words).
constexpr uint32_t kDescPlainHi = (128u >> 4) | (1u << 14);

// Instruction descriptors: fp32 accumulators, M = 256 (128 lanes of each CTA of
// the pair), N = n (each CTA's shared memory holds half of the n rows).
__device__ __forceinline__ uint32_t idesc_16bit(bool bf16, bool a_mn, bool b_mn, int n) {
  const uint32_t f = bf16 ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(n >> 3) << 17) | ((256u >> 4) << 24);
}
// e4m3 operands with one UE8M0 scale per 32 reduction elements, byte `sf` of the scale words.
__device__ __forceinline__ uint32_t idesc_e4m3(int n, uint32_t sf) {
  return (sf << 4) | ((uint32_t)(n >> 3) << 17) | (1u << 23) | ((256u >> 4) << 24) | (sf << 29);
}

__device__ __forceinline__ void mma_16bit(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
               "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
               "tcgen05.mma.cta_group::2.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
               "r"(accumulate), "n"(kDescHi)
               : "memory");
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %6, 0;\n\t"
               "mov.b64 da, {%1, %7};\n\tmov.b64 db, {%2, %7};\n\t"
               "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], da, db, %3, [%4], [%5], p;"
               "\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "n"(kDescHi)
               : "memory");
}
// 32 rows of 16 bytes of shared memory to 4 tensor-memory columns, in all four
// lane quarters; in both CTAs of the pair, each from its own shared memory.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint32_t lo) {
  asm volatile("{\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\t"
               "tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(taddr), "r"(lo), "n"(kDescPlainHi)
               : "memory");
}
// Arrives on the mbarrier at this offset in the CTAs of the mask (by cluster
// rank) when this thread's matrix work issued so far has completed.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar, uint16_t both) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(bar), "h"(both)
               : "memory");
}

}  // namespace moeperm
