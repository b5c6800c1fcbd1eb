// Block-scaled 8-bit tensor-core building blocks for sm_100a: the
// tcgen05.mma form whose operands carry a power-of-two scale per row and 32
// K elements, its scale factors in tensor memory, and cluster helpers.
#pragma once

#include "sm100_ptx.cuh"

namespace moe {
namespace ptx {

// True in one lane of a converged warp (the same lane each time).  Code under
// this predicate is known to run in a single lane, so descriptors and
// addresses stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// The descriptor of ptx::smem_desc_sw128 from its low word (address >> 4 and the
// leading offset): only that word changes from tile to tile and step to step,
// and adding to it alone saves the issuing thread the carries.
__device__ __forceinline__ uint32_t desc_sw128_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | (1u << 16);
}
__device__ __forceinline__ uint64_t desc_sw128(uint32_t lo) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  return (uint64_t)hi << 32 | lo;
}

// Instruction descriptor of tcgen05.mma kind::mxf8f6f4 with block scales:
// A and B E4M3 (format 0), both K-major, fp32 accumulator, scales E8M0 (bit
// 23), N >> 3 in bits 17-22, M >> 4 in bits 24-28.  The byte of each 32-bit
// scale word that the MMA reads is named in bits 4-5 (B) and 29-30 (A).
__host__ __device__ constexpr uint32_t idesc_mxf8(uint32_t M, uint32_t N) {
  return (1u << 23) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
__host__ __device__ constexpr uint32_t idesc_sf_byte(uint32_t a_byte, uint32_t b_byte) {
  return (b_byte << 4) | (a_byte << 29);
}

// D[tmem] (+)= (A * sfa) (B * sfb)^T over K = 32 E4M3 elements; one thread.
// Scale factors: row r of A has its E8M0 byte in TMEM lane r % 32 (repeated in
// each of the four lane quarters), column sfa + r / 32; B's rows the same
// way from sfb.  Both column addresses are multiples of four.
__device__ __forceinline__ void mma_mxf8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
      "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// 32 lanes x 32 bits, 1, 2, 4 or 8 consecutive columns: thread i of the warp
// writes TMEM lane (base lane + i).
__device__ __forceinline__ void tmem_st_x1(uint32_t taddr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r)
               : "memory");
}
__device__ __forceinline__ void tmem_st_x2(uint32_t taddr, uint32_t r0, uint32_t r1) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(taddr), "r"(r0),
               "r"(r1)
               : "memory");
}
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// Whether the aligned words that hold q[0 .. n-1] lie inside the array [lo, hi)
// of bytes, as they do everywhere but at an unaligned array's two ends.
__device__ __forceinline__ bool words_inside(const int8_t* q, int n, const int8_t* lo,
                                             const int8_t* hi) {
  const uintptr_t first = reinterpret_cast<uintptr_t>(q) & ~(uintptr_t)3;
  const uintptr_t end = (reinterpret_cast<uintptr_t>(q + n) + 3) & ~(uintptr_t)3;
  return first >= reinterpret_cast<uintptr_t>(lo) && end <= reinterpret_cast<uintptr_t>(hi);
}
// Bytes q[0 .. n-1] (at most four) as a word, byte by byte.
__device__ __forceinline__ uint32_t bytes_word(const int8_t* q, int n) {
  uint32_t v = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) v |= (uint32_t)(uint8_t)__ldcg(q + i) << (8 * i);
  return v;
}

// Whether the barrier's phase of this parity has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A barrier of a few warps whose wait is bounded: an mbarrier that one lane of
// each warp arrives on.  False when the wait gave up (as mbar_wait).
struct WarpBarrier {
  uint64_t* bar;
  uint32_t phase = 0;
  __device__ __forceinline__ bool sync(volatile int* abort, int lane) {
    __syncwarp();
    if (lane == 0)
      asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar))
                   : "memory");
    const bool ok = mbar_wait(bar, phase, abort);
    phase ^= 1u;
    return !__any_sync(0xffffffffu, !ok);
  }
};

// ---------------------------------------------------------------------------
// Clusters
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of every CTA of the cluster; orders their shared-memory
// accesses before it (release) with those after it (acquire).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The four floats at this CTA's shared address `addr` in CTA `rank` of the
// cluster.
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .u32 a;\n\t"
      "mapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

}  // namespace ptx
}  // namespace moe
