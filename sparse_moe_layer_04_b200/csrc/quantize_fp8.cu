// bf16 rows -> E4M3 codes with one power-of-two exponent per 128 columns of
// each row, gathered by an optional row index on the way.
//
//   e[r, b]    = the smallest e in [-117, 120] with max|x[r, 128b ..]| <= 448 * 2^e
//                (0 for a block of zeros)
//   code[r, c] = E4M3(x[r, c] * 2^-e), round to nearest even
//
// x * 2^-e is exact in bf16 wherever the code is not zero, so each code has one
// rounding.  448 = 0.875 * 2^9: with max = 1.m * 2^p (bf16, 7 fraction
// bits), e = p - 8, or p - 7 when the fraction is above that of 448 = 1.75 *
// 2^8, which the integer sum below decides without branches.
//
// 32768 x 6144 rows gathered from 4096: 66 us, 600 MB through L2 (each row is
// read eight times, 50 MB of HBM reads and 203 MB of writes).  Without the loads
// 43, without the arithmetic 57, and the two overlap only as far as other warps
// are there to run: resident warps that walk rows with the next one on its way
// took 68, sixteen of them an SM fed by bulk copies 128.
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

// Two bf16 products.
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 32 bytes in one load (16-byte aligned addresses that are not 32-byte aligned
// take two).
__device__ __forceinline__ void load32(const uint16_t* p, bool wide, uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                   "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}

// A warp takes U chunks of 512 columns of one row: eight lanes own a block of
// 128 columns, sixteen columns (32 bytes) each.  All U loads are issued before
// the first is used.
template <int U>
__global__ void __launch_bounds__(kThreads) quantize_fp8_kernel(
    const uint16_t* __restrict__ x, int src_rows, const int32_t* __restrict__ idx, int R, int K,
    int KB, bool wide, uint8_t* __restrict__ codes, int8_t* __restrict__ exps, int* status) {
  ptx::pdl_launch_dependents();
  ptx::pdl_wait();
  const int lane = threadIdx.x & 31;
  const unsigned r = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);   // (R may end at 2^31)
  if (r >= (unsigned)R) return;
  const int col0 = blockIdx.y * (512 * U) + lane * 16;
  const int s = idx ? idx[r] : (int)r;
  int bad = 0;
  const bool ok = s >= 0 && s < src_rows;
  if (!ok) bad = kStBounds;
  const uint16_t* src = x + (size_t)(ok ? s : 0) * K + col0;
  uint32_t w[U][8];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (ok && col0 + 512 * i < K) {
      load32(src + 512 * i, wide, w[i]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) w[i][q] = 0;
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int col = col0 + 512 * i;
    // the largest magnitude of the block, as bf16 bits (they order like the values)
    uint32_t t2 = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) t2 = __vmaxu2(t2, w[i][q] & 0x7fff7fffu);
    uint32_t top = max(t2 & 0xffffu, t2 >> 16);
#pragma unroll
    for (int off = 4; off; off >>= 1) top = max(top, __shfl_xor_sync(kAll, top, off));
    const bool odd = top >= 0x7f80u;   // a NaN or an infinity in this block
    if (__any_sync(kAll, odd)) {
      // the largest finite magnitude instead
      if (odd) bad |= kStNonFinite;
      top = 0;
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const uint32_t m = (w[i][q / 2] >> (16 * (q & 1))) & 0x7fffu;
        if (m < 0x7f80u) top = max(top, m);
      }
#pragma unroll
      for (int off = 4; off; off >>= 1) top = max(top, __shfl_xor_sync(kAll, top, off));
    }
    // p - 8 with p = (bits >> 7) - 127, one more when the fraction exceeds
    // 0.75 (0x60 of 0x80): adding 0x1f carries into the exponent exactly then
    const int e = top ? max((int)((top + 0x1fu) >> 7) - 135, kQMinExp) : 0;
    const uint32_t inv = (uint32_t)(127 - e) * 0x00800080u;   // 2^-e as bf16, twice
    uint32_t c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t y = mul2(w[i][2 * q], inv), z = mul2(w[i][2 * q + 1], inv);
      c[q] = e4m3x2(bf_lo(y), bf_hi(y)) | (e4m3x2(bf_lo(z), bf_hi(z)) << 16);
    }
    if (odd) {
      // infinities are marked like NaN (the conversion saturates them)
#pragma unroll
      for (int q = 0; q < 16; ++q)
        if (((w[i][q / 2] >> (16 * (q & 1))) & 0x7fffu) >= 0x7f80u)
          c[q / 4] = (c[q / 4] & ~(0xffu << (8 * (q & 3)))) | (0x7fu << (8 * (q & 3)));
    }
    if (col < K) {
      *reinterpret_cast<uint4*>(codes + (size_t)r * K + col) = make_uint4(c[0], c[1], c[2], c[3]);
      if ((lane & 7) == 0) exps[(size_t)r * KB + (col >> 7)] = (int8_t)e;
    }
  }
  if (bad && status) atomicOr(status, bad);
}

}  // namespace

cudaError_t launch_quantize_fp8(const uint16_t* x, int src_rows, const int32_t* idx, int R, int K,
                                uint8_t* codes, int8_t* exps, int* status, cudaStream_t st) {
  const int chunks = (K + 511) / 512;
  const int warps = kThreads / 32;
  const unsigned gx = ((unsigned)R + warps - 1) / warps;
  // rows start on 32 bytes when the matrix does (K is a multiple of 16)
  const bool wide = (reinterpret_cast<uintptr_t>(x) & 31u) == 0;
  const int KB = (K + 127) / 128;
  // A chunk per warp while that is not much more than the SMs hold at once (104
  // rows of 6144: 1.9 us; 1000 rows: 4.1 against 4.6) or a row has no more (65536
  // rows of 256: 14 against 21); else two, whose loads a warp has in flight
  // together (32768 rows of 6144: 66 us, with one 77, with four 67; 16384 rows of
  // 1024: 7.5, 8.1, 11.6).
  if (chunks == 1 || (long long)gx * chunks <= 12ll * num_sms())
    return launch_pdl(quantize_fp8_kernel<1>, dim3(gx, chunks), dim3(kThreads), 0, st, x, src_rows,
                      idx, R, K, KB, wide, codes, exps, status);
  return launch_pdl(quantize_fp8_kernel<2>, dim3(gx, (chunks + 1) / 2), dim3(kThreads), 0, st, x,
                    src_rows, idx, R, K, KB, wide, codes, exps, status);
}

}  // namespace moe
