// bf16 rows -> E4M3 codes with one power-of-two exponent per 128 columns of
// each row, gathered by an optional row index on the way.
//
//   e[r, b]    = the smallest e in [-117, 120] with max|x[r, 128b ..]| <= 448 * 2^e
//                (0 for a block of zeros)
//   code[r, c] = E4M3(x[r, c] * 2^-e), round to nearest even
//
// x * 2^-e is exact in fp32 wherever the code is not zero, so each code has
// one rounding.  448 = 0.875 * 2^9: with max = 1.m * 2^p (bf16, 7 fraction
// bits), e = p - 8, or p - 7 when the fraction is above that of 448 = 1.75 *
// 2^8, which the integer sum below decides without branches.
#include <cuda_bf16.h>

#include "moe_internal.cuh"
#include "sm100_ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kQMinExp = -117;   // keeps 2^-e and the smallest step 2^(e-9) normal in fp32
constexpr uint32_t kAll = 0xffffffffu;

// Two floats -> two E4M3 bytes (lo in the low byte); NaN gives 0x7F.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Sixteen lanes own a block of 128 columns, eight columns (16 bytes) each; a
// warp takes two neighbouring blocks of a row at a time, and kUnroll such
// pairs are loaded before the first is used.
constexpr int kUnroll = 4;

__global__ void __launch_bounds__(kThreads) quantize_fp8_kernel(
    const uint16_t* __restrict__ x, int src_rows, const int32_t* __restrict__ idx, int R, int K,
    uint8_t* __restrict__ codes, int8_t* __restrict__ exps, int* status) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int KB = (K + 127) / 128;
  const int pairs = (KB + 1) / 2;               // 256-column units of a row
  const long long units = (long long)R * pairs;
  const int lane = threadIdx.x & 31;
  const long long warp = (blockIdx.x * (long long)kThreads + threadIdx.x) >> 5;
  const long long nwarps = ((long long)gridDim.x * kThreads) >> 5;
  int bad = 0;
  for (long long u0 = warp * kUnroll; u0 < units; u0 += nwarps * kUnroll) {
    uint4 v[kUnroll];
    long long row[kUnroll];
    int col[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const long long u = u0 + i;
      row[i] = u / pairs;
      col[i] = (int)(u - row[i] * pairs) * 256 + lane * 8;
      v[i] = make_uint4(0, 0, 0, 0);
      if (u < units && col[i] < K) {
        const int s = idx ? idx[row[i]] : (int)row[i];
        if (s >= 0 && s < src_rows)
          v[i] = *reinterpret_cast<const uint4*>(x + (size_t)s * K + col[i]);
        else
          bad |= kStBounds;
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      // largest finite magnitude as bf16 bits (they order like the values)
      uint32_t top = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int s = 0; s < 32; s += 16) {
          const uint32_t m = (w[q] >> s) & 0x7fffu;
          if (m >= 0x7f80u) bad |= kStNonFinite;
          else top = max(top, m);
        }
      }
#pragma unroll
      for (int off = 8; off; off >>= 1) top = max(top, __shfl_xor_sync(kAll, top, off));
      // p - 8 with p = (bits >> 7) - 127, one more when the fraction exceeds
      // 0.75 (0x60 of 0x80): adding 0x1f carries into the exponent exactly then
      int e = top ? max((int)((top + 0x1fu) >> 7) - 135, kQMinExp) : 0;
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
      uint32_t c[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t a = w[2 * q], b = w[2 * q + 1];
        uint32_t lo = e4m3x2(bf_lo(a) * inv, bf_hi(a) * inv);
        uint32_t hi = e4m3x2(bf_lo(b) * inv, bf_hi(b) * inv);
        // infinities are marked like NaN (the conversion would saturate them)
        if ((a & 0x7fffu) >= 0x7f80u) lo = (lo & 0xff00u) | 0x7fu;
        if (((a >> 16) & 0x7fffu) >= 0x7f80u) lo = (lo & 0x00ffu) | 0x7f00u;
        if ((b & 0x7fffu) >= 0x7f80u) hi = (hi & 0xff00u) | 0x7fu;
        if (((b >> 16) & 0x7fffu) >= 0x7f80u) hi = (hi & 0x00ffu) | 0x7f00u;
        c[q] = lo | (hi << 16);
      }
      if (u0 + i < units && col[i] < K) {
        *reinterpret_cast<uint2*>(codes + (size_t)row[i] * K + col[i]) = make_uint2(c[0], c[1]);
        if ((lane & 15) == 0) exps[(size_t)row[i] * KB + col[i] / 128] = (int8_t)e;
      }
    }
  }
  if (bad && status) atomicOr(status, bad);
}

}  // namespace

cudaError_t launch_quantize_fp8(const uint16_t* x, int src_rows, const int32_t* idx, int R, int K,
                                uint8_t* codes, int8_t* exps, int* status, cudaStream_t st) {
  const long long units = (long long)R * ((K + 255) / 256);
  const int per_block = kThreads / 32 * kUnroll;
  long long blocks = (units + per_block - 1) / per_block;
  const long long cap = 8ll * num_sms();
  if (blocks > cap) blocks = cap;
  return launch_pdl(quantize_fp8_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, st, x,
                    src_rows, idx, R, K, codes, exps, status);
}

}  // namespace moe
