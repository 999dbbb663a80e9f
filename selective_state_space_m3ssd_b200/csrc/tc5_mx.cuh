// Block-scaled tcgen05 products: operands in microscaled formats (mx.cuh) in shared memory
// (128-byte swizzled canonical layouts, K-major), their scales in tensor memory.
#pragma once

#include <stdint.h>

#include "tc5.cuh"

namespace m3ssd {
namespace tc5 {

// Instruction descriptor of kind::mxf4 and kind::mxf8f6f4 with fp32 accumulation, both
// operands K-major: A / B format (bits 7-9 and 10-12; mxf4: 1 = E2M1; mxf8f6f4: 0 = E4M3,
// 5 = E2M1), N >> 3 (bits 17-22), scale format (bit 23: 1 = UE8M0), M >> 7 (bits 27-28).
// The scale-factor ids (which byte of a 32-bit scale column a product reads: bits 4-5 for
// B, 29-30 for A) are ORed in by idesc_mx_sf.
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, uint32_t a_fmt, uint32_t b_fmt) {
  return (a_fmt << 7) | (b_fmt << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 7) << 27);
}
__host__ __device__ constexpr uint32_t idesc_mx_sf(uint32_t idesc, uint32_t id) {
  return idesc | (id << 4) | (id << 29);
}

// D[tmem] (+)= (A . scales) * (B . scales): 64 E2M1 values of K, two UE8M0 scales a row.
__device__ __forceinline__ void mma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                         uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], "
      "p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u));
}
// The same for 8-bit containers: 32 values of K, one UE8M0 scale a row.
__device__ __forceinline__ void mma_mxf8f6f4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                             bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate ? 1u : 0u));
}

// Shared-memory descriptor without swizzle of 32 rows of 16 bytes, 8-row groups 128 bytes
// apart (one 512-byte tile of scales).
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(16 >> 4) << 16) |
         ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
// One tile of scales (128 rows x 4 blocks) into four TMEM columns, repeated for the four
// lane quarters.  In order with the products this thread issues afterwards.
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc)
               : "memory");
}

// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}"
               : "=r"(p));
  return p != 0;
}
// A thread-block cluster: this CTA's rank; a barrier of all its threads that orders what they
// wrote to shared memory before; another CTA's copy of a shared-memory address; a load there.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_ld4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

}  // namespace tc5
}  // namespace m3ssd
