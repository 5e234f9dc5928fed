// Tensor-core plumbing shared by the attention kernels (tcgen05, tensor memory,
// shared-memory matrix descriptors) and the unpacking of block codes to fp16.
#pragma once

#include "kvq_internal.h"
#include "ptx.cuh"

namespace kvq {

// Shared-memory matrix descriptor of a 128-byte-swizzled operand (atoms 1024-byte
// aligned, so the base offset is 0).
__device__ __forceinline__ uint64_t umma_desc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;   // descriptor version for sm_100
  d |= (uint64_t)2 << 61;   // layout: 128-byte swizzle
  return d;
}
// D (tensor memory) = A B (+ D when `accumulate` is nonzero), kind::f16, with A
// read from tensor memory (M rows in lanes, K along columns, two 16-bit elements
// per 32-bit column, the lower-indexed in the low half) and B from shared memory
// through its descriptor.
__device__ __forceinline__ void umma_f16_tmem_a(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive fp32 columns of this thread's TMEM lane (warp w: lanes 32(w%4)..),
// waited for inside the same statement so that no use of r can move above the wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t r[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t r[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One 32-channel block (block b of token t) of a page-head's K or V plane:
// its codes' low plane (lo, up to 32 bytes) and high plane (hi, up to 8 bytes).
// K planes are interleaved in 16-byte pieces (byte o of token t at
// ((o/16)*64 + t)*16 + o%16); V planes are row-major.  Every read is aligned.
template <int BITS, bool KPLANE>
__device__ __forceinline__ void block_planes(const uint8_t* codes, int cb, int t, int b, uint32_t lo[8],
                                             uint32_t hi[2]) {
  auto at = [&](int o) -> const uint8_t* {
    return KPLANE ? codes + ((((o >> 4) * PAGE + t) << 4) + (o & 15)) : codes + t * cb + o;
  };
  if (BITS == 8) {
    const uint4 a = *reinterpret_cast<const uint4*>(at(32 * b));
    const uint4 c = *reinterpret_cast<const uint4*>(at(32 * b + 16));
    lo[0] = a.x; lo[1] = a.y; lo[2] = a.z; lo[3] = a.w; lo[4] = c.x; lo[5] = c.y; lo[6] = c.z; lo[7] = c.w;
  } else if (BITS >= 4) {                          // 4, 5, 6: nibble plane first
    const uint4 a = *reinterpret_cast<const uint4*>(at(16 * b));
    lo[0] = a.x; lo[1] = a.y; lo[2] = a.z; lo[3] = a.w;
  } else {                                         // 2, 3: 2-bit plane first
    const uint2 a = *reinterpret_cast<const uint2*>(at(8 * b));
    lo[0] = a.x; lo[1] = a.y;
  }
  if (BITS == 6) {
    const uint2 h = *reinterpret_cast<const uint2*>(at(64 + 8 * b));
    hi[0] = h.x; hi[1] = h.y;
  } else if (BITS == 5) {
    hi[0] = *reinterpret_cast<const uint32_t*>(at(64 + 4 * b));
  } else if (BITS == 3) {
    hi[0] = *reinterpret_cast<const uint32_t*>(at(32 + 4 * b));
  }
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ __half2 as_h2(uint32_t w) { return *reinterpret_cast<const __half2*>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// The codes of channels 8J .. 8J+7 of a block as four fp16 pairs 1024 + u (bit
// pattern 0x6400 | u, exact for u < 1024): pair e holds channels 8J+2e (low
// half) and 8J+2e+1.  8- and 4-bit planes are spread with byte permutes (for
// nibbles, the sign-replicating selectors 8 + k give zero bytes: every byte is
// below 16); the other widths assemble their integer codes first.
template <int BITS, int J>
__device__ __forceinline__ void chunk_pairs(const uint32_t lo[8], const uint32_t hi[2], uint32_t W[4]) {
  if (BITS == 8) {
    const uint32_t a = lo[2 * J], c = lo[2 * J + 1];
    W[0] = prmt(a, 0x64646464u, 0x4140u);
    W[1] = prmt(a, 0x64646464u, 0x4342u);
    W[2] = prmt(c, 0x64646464u, 0x4140u);
    W[3] = prmt(c, 0x64646464u, 0x4342u);
  } else if (BITS == 4) {
    const uint32_t L = lo[J] & 0x0F0F0F0Fu, Hh = (lo[J] >> 4) & 0x0F0F0F0Fu;
    W[0] = prmt(L, Hh, 0xC480u) | 0x64006400u;
    W[1] = prmt(L, Hh, 0xD591u) | 0x64006400u;
    W[2] = prmt(L, Hh, 0xE6A2u) | 0x64006400u;
    W[3] = prmt(L, Hh, 0xF7B3u) | 0x64006400u;
  } else {
    uint32_t u[8];
    if (BITS >= 4) {
#pragma unroll
      for (int v = 0; v < 8; ++v) u[v] = (lo[J] >> (4 * v)) & 15u;
    } else {
      const uint32_t w = lo[J >> 1] >> (16 * (J & 1));
#pragma unroll
      for (int v = 0; v < 8; ++v) u[v] = (w >> (2 * v)) & 3u;
    }
    if (BITS == 6) {
      const uint32_t h = hi[J >> 1] >> (16 * (J & 1));
#pragma unroll
      for (int v = 0; v < 8; ++v) u[v] |= ((h >> (2 * v)) & 3u) << 4;
    } else if (BITS == 5 || BITS == 3) {
      const uint32_t h = hi[0] >> (8 * J);
#pragma unroll
      for (int v = 0; v < 8; ++v) u[v] |= ((h >> v) & 1u) << (BITS == 5 ? 4 : 2);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) W[e] = u[2 * e] | (u[2 * e + 1] << 16) | 0x64006400u;
  }
}

}  // namespace kvq
