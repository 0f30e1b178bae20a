// sm100_mx4.cuh -- tcgen05 primitives of the MXFP4 (block-scaled E2M1) GEMM:
// the block-scaled instruction descriptor, MMA and scale copy for one CTA or a
// CTA pair, and the tensor copy of the scale blocks.  Written from the PTX ISA
// description of each instruction.
#pragma once
#include "sm100.cuh"

namespace vit {

// Instruction descriptor of kind::mxf4: E2M1 x E2M1, fp32 accumulation, E8M0
// scales (one per 32 elements, two per row and MMA), both operands K-major,
// K = 64 per MMA.  sf: which two bytes of the 32-bit scale words this MMA
// reads, 0 or 2.
__host__ __device__ constexpr uint32_t idesc_mx4(int M, int N, int sf) {
  return (uint32_t(sf & 3) << 4)      // B scale-factor byte
         | (1u << 7)                  // A format: E2M1
         | (1u << 10)                 // B format: E2M1
         | (uint32_t(N >> 3) << 17)   // N / 8
         | (1u << 23)                 // scale format: E8M0
         | (uint32_t(M >> 7) << 27)   // M / 128
         | (uint32_t(sf & 3) << 29);  // A scale-factor byte
}

// D[tmem] (+)= (A . 2^sfA)[smem desc] * (B . 2^sfB)[smem desc] over K = 64.
// The scale addresses carry the scale byte index in their top two bits.  PAIR:
// the CTA pair's MMA, issued by its leader; each CTA's tensor memory holds the
// scales of its own rows of A and of all of B.
template <bool PAIR>
__device__ __forceinline__ void mma_mx4_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                           uint32_t idesc, uint32_t sfa_tmem, uint32_t sfb_tmem,
                                           uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
        "[%6], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], "
        "[%6], p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sfa_tmem), "r"(sfb_tmem)
        : "memory");
}

// Shared memory -> TMEM copy of a 32-row x 16-byte scale block into all four
// lane quarters (see tmem_cp_32x128b_x4 of sm100_mx8.cuh); PAIR: in both CTAs
// of the pair, each from its own shared memory at the descriptor's address.
template <bool PAIR>
__device__ __forceinline__ void tmem_cp_scales(uint32_t dst_tmem, uint64_t src_desc) {
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(dst_tmem), "l"(src_desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(dst_tmem), "l"(src_desc)
                 : "memory");
}

// Asks for [p, p + bytes) to be brought into L2 (16-byte aligned, a multiple of 16).
__device__ __forceinline__ void prefetch_l2(const void *p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(reinterpret_cast<uint64_t>(p)),
               "r"(bytes)
               : "memory");
}

// The address of `addr`, a shared-memory address of this CTA, in the CTA of rank
// `cta` of the cluster, and 16 bytes from such an address.
__device__ __forceinline__ uint32_t map_addr_to_cta(uint32_t addr, uint32_t cta) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}
__device__ __forceinline__ float4 ld_cluster(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 3-D tiled bulk tensor copy global -> shared, completion on an mbarrier of
// this CTA, or (PAIR) on one of the pair's leader at a cluster address.
template <bool PAIR>
__device__ __forceinline__ void tma_load_3d(void *smem_dst, const CUtensorMap *map, uint32_t bar,
                                            int c0, int c1, int c2) {
  if constexpr (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

}  // namespace vit
