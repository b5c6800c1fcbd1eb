// Grouped products of E4M3 rows with E4M3 weights, one power-of-two exponent
// per 128 columns of a row and per 128 x 128 block of a weight matrix:
//
//   y[r, n]   = sum_k xq[r, k] 2^xe[r, k/128] * wq[g, n, k] 2^we[g, n/128, k/128]
//   act[r, n] = silu(y1[r, n]) * y3[r, n]        (gated: weights W1 and W3)
//
// for the rows offsets[g] <= r < offsets[g + 1] of each group g.
//
// The exponents are E8M0 scales as they stand (byte = e + 127), so the tensor
// core applies them itself: tcgen05.mma kind::mxf8f6f4 with block scales takes
// one scale per row and 32 K elements, and the 128 columns of an exponent are
// four such steps that name the same byte.  The sum over all of K then stays in
// one fp32 accumulator in tensor memory; no partial product is scaled or
// added outside the tensor core.
//
// The weights are the M = 128 operand and the rows the N operand, in steps
// of 16 up to NT: a group's ragged row count pads to 16 only, one thread of
// the epilogue holds one output column, and a warp stores 32 neighbouring
// columns of a row at a time.
//
// CTA structure (480 threads, tiles taken round-robin):
//   warp 0      weight producer: TMA of 128 x 128 codes a stage, 128-byte
//               swizzled, into a deep ring (the weights come from HBM)
//   warp 14     row producer: TMA of up to NT x 128 codes a stage into a ring
//               of its own (the rows are read again for every column tile, so
//               they come from L2)
//   warp 1      TMEM allocator and MMA issuer (one elected thread)
//   warps 2-9   epilogue: TMEM -> registers -> global, two warps for each lane
//               quarter, which take turns of 16 rows; two accumulators, so a
//               tile's epilogue overlaps the next tile's products (three
//               where a CTA takes two weight tiles at a time and they fit)
//   warps 10-13 scale writers: the exponents of sixteen K-blocks at a time,
//               loaded a row per thread while the sixteen before them are in
//               use, exchanged through shared memory, and written as 32-bit
//               words of four E8M0 bytes into one of two TMEM slots; each of
//               the four warps fills its lane quarter with the same words, as
//               the tensor core expects them
// Gated tiles hold 64 output columns: the 128 weight rows alternate 16 of W1
// and 16 of W3, so every warp's lanes 0-15 hold gates and lanes 16-31 the ups
// of the same columns, which one shuffle per pair of rows brings together.
//
// Few tiles (one row through one matrix): a cluster of CTAs shares a tile,
// each with its own range of K-blocks, and adds the partial tiles through
// distributed shared memory in rank order, so results do not depend on timing.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>

#include "ffn_common.cuh"
#include "gate.cuh"
#include "sm100_scaled.cuh"

namespace moe {
namespace {

constexpr int kBK = 128;                 // K elements of a stage = one exponent
constexpr int kWTile = 128 * kBK;        // weight tile bytes
constexpr int kEpiWarps = 8, kSfWarp0 = 2 + kEpiWarps, kRowWarp = kSfWarp0 + 4;
constexpr int kThreads = (kRowWarp + 1) * 32;
constexpr int kMaxStages = 11;          // of either ring
constexpr int kRingBytes = 208 * 1024;
constexpr int kMaxG = 1024;
constexpr unsigned kAll = 0xffffffffu;

struct alignas(64) GemmParams8 {
  CUtensorMap x;        // [R, K] codes, box XBOX x 128
  CUtensorMap w1, w3;   // [G * N, K] codes, box 128 (plain) or 16 (gated) x 128
  const int8_t* xe;     // [R, KB]
  const int8_t* w1e;    // [G, NB, KB]
  const int8_t* w3e;
  const int32_t* offsets;   // [G + 1]; nullptr: one group of all rows
  void* y;
  int y_bf16;
  int G, R, N, K, KB, NB;
  int nt;               // output column tiles of a group
  int split;            // CTAs per tile (cluster size)
  int* status;
};

// Row blocks of the groups: group g's rows are cut into equal blocks of at
// most NT rows (a multiple of 16).
struct GroupMap {
  int total;                 // row blocks of all groups
  int off[kMaxG + 1];
  int prefix[kMaxG + 1];
};

struct Tile8 {
  int g, n0, row0, rows;     // group, first output column, first row, rows
};

// NT: rows of a tile.  NW: weight tiles of 128 that share the rows of a stage (2:
// the rows are staged once for twice the products, which halves what a product
// draws from L2).
template <int NT, int NW>
struct Cfg {
  // rows of one TMA box of the row operand: a tile loads only as many boxes as
  // its rows need
  static constexpr int XBOX = NT % 48 == 0 ? 48 : 32;
  static constexpr int X_BYTES = NT * kBK;
  static constexpr int W_BYTES = NW * kWTile;
  // The rows come from L2, whose latency under this load takes five or six
  // K-blocks of one weight tile to cover; six stages of weights keep HBM busy.
  // (64 experts, 8192 rows, N = 2048, K = 6144 gated: 290 us with 5 + 6 stages of
  // rows and weights, 318 with 4 + 8.)
  static constexpr int XST = NW == 2 ? kRingBytes / (W_BYTES + X_BYTES) : NT > 160 ? 4 : NT > 144 ? 5 : 6;
  static constexpr int WST = NW == 2 ? XST
                             : (kRingBytes - XST * X_BYTES) / W_BYTES < kMaxStages
                                 ? (kRingBytes - XST * X_BYTES) / W_BYTES
                                 : kMaxStages;
  static constexpr int RING = WST * W_BYTES + XST * X_BYTES;
  static_assert(XST <= WST, "the weights' stages release the rows'");
  // scale columns of a slot: 4 for each weight tile, 8 for the rows
  static constexpr int SF_SLOT = 4 * NW + 8;
  // accumulators, used in turn: two, or the three that fit
  static constexpr int ACC = NW == 2 && 3 * NT + 2 * SF_SLOT <= 512 ? 3 : 2;
  static constexpr int COLS = ACC * NT + 2 * SF_SLOT;
  static constexpr uint32_t TMEM_COLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
  static_assert(COLS <= 512 && NT % 16 == 0 && NT <= 240, "tensor memory columns");
  static_assert(NT % XBOX == 0 && XBOX % 8 == 0 && X_BYTES % 1024 == 0, "row boxes");
};

struct Shared8 {
  // of the weights' stages; a K-block's rows arrive on the same barrier
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t sf_full[2], sf_empty[2];
  uint64_t acc_full[3], acc_empty[3];
  uint64_t drain;
  uint64_t sf_bar;             // barrier of the four scale warps
  uint32_t tmem_base;
  int abort;
  int bad;
  uint32_t sf_rows[2][4][256]; // scale words of sixteen K-blocks [set][row]
  GroupMap gm;
};

template <int NT, int NW>
constexpr int smem_bytes8() {
  return 1024 + Cfg<NT, NW>::RING + (int)sizeof(Shared8);
}

__device__ __forceinline__ int blocks_of(int rows, int nt) { return (rows + nt - 1) / nt; }

// Rows of the product's row operand: the tile's, in steps of 16.
__device__ __forceinline__ int mma_rows(int rows) { return max(16, (rows + 15) / 16 * 16); }

// One warp, offsets in gm.off: checks them and counts each group's row blocks.
// Offsets that are not increasing within [0, R] give no tiles and raise
// kStBounds.
template <int NT>
__device__ void build_groups(GroupMap& gm, const GemmParams8& p, int lane) {
  int carry = 0;
  bool bad = false;
  for (int base = 0; base < p.G; base += 32) {
    const int g = base + lane;
    int cnt = 0;
    if (g < p.G) {
      const int a = gm.off[g], b = gm.off[g + 1];
      if (a < 0 || b < a || b > p.R) bad = true;
      else cnt = blocks_of(b - a, NT);
    }
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += v;
    }
    if (g < p.G) gm.prefix[g] = carry + incl - cnt;
    carry += __shfl_sync(kAll, incl, 31);
  }
  bad = __any_sync(kAll, bad);
  if (lane == 0) {
    gm.prefix[p.G] = carry;
    gm.total = bad ? 0 : carry;
    if (bad && p.status) atomicOr(p.status, kStBounds);
  }
}

// The tiles of one CTA (or team of CTAs): t, t + step, ...  Tiles are numbered
// by group, then output column tile, row blocks fastest (the CTAs that run
// together share weight tiles through L2).
template <bool GATED, int NW>
struct Walk {
  int t, step, total;
  int g = 0;
  __device__ __forceinline__ Walk(const GroupMap& gm, const GemmParams8& p, int first, int st)
      : t(first), step(st), total(gm.total * p.nt) {}
  __device__ __forceinline__ bool more() const { return t < total; }
  __device__ __forceinline__ void next() { t += step; }
  // The tile t; successive calls come with rising t.
  __device__ __forceinline__ Tile8 tile(const GroupMap& gm, const GemmParams8& p) {
    while (t >= gm.prefix[g + 1] * p.nt) ++g;
    const int rows = gm.off[g + 1] - gm.off[g];
    const int nb = gm.prefix[g + 1] - gm.prefix[g];
    int local = t - gm.prefix[g] * p.nt, b = 0, per = rows;
    if (nb > 1) {                              // equal blocks, in steps of 16 rows
      per = ((rows - 1) / nb + 16) / 16 * 16;
      b = local % nb;
      local /= nb;
    }
    Tile8 ti;
    ti.g = g;
    ti.n0 = local * (GATED ? 64 : 128) * NW;
    ti.row0 = gm.off[g] + b * per;
    ti.rows = min(per, rows - b * per);
    return ti;
  }
};

// Exponents q[0 .. n-1] (n <= 16) of an array [lo, hi) as they stand in memory,
// in words of four.  Any alignment: the aligned words that hold them are
// loaded and shifted, but for those that reach beyond the array's ends.
__device__ __forceinline__ void load_exps(const int8_t* q, int n, const int8_t* lo,
                                          const int8_t* hi, uint32_t (&w)[4]) {
  if (!ptx::words_inside(q, n, lo, hi)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = ptx::bytes_word(q + 4 * i, n - 4 * i);
    return;
  }
  const uintptr_t at = reinterpret_cast<uintptr_t>(q);
  const uint32_t* base = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
  const int off = (int)(at & 3);
  uint32_t v[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = 4 * i - off < n ? __ldcg(base + i) : 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(v[i], v[i + 1], 8 * off);
}

// Word i of n exponents -> E8M0 bytes.  -128 has no E8M0 counterpart (its byte
// would be the NaN scale).
__device__ __forceinline__ uint32_t scale_bytes(uint32_t w, int i, int n, bool* bad) {
  const int left = n - 4 * i;
  if (left < 4) w &= left > 0 ? (1u << (8 * left)) - 1u : 0u;
  *bad |= __vcmpeq4(w, 0x80808080u) != 0;
  return __vadd4(w, 0x7f7f7f7fu);
}

// Sixteen accumulator columns (rows of the group, from c0) of one weight row
// per lane -> outputs.
template <bool GATED>
__device__ __forceinline__ void store16(const GemmParams8& p, const Tile8& ti, int q, int lane,
                                        int c0, const uint32_t (&v)[16]) {
  const int left = ti.rows - c0;         // rows to store, the same in every lane
  if (GATED) {
    // lanes 0-15 finish the even rows of each pair, lanes 16-31 the odd ones
    const bool up = lane >= 16;
    const int n = ti.n0 + q * 16 + (lane & 15);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) +
                       (size_t)(ti.row0 + c0 + (up ? 1 : 0)) * p.N + n;
    const size_t step = 2 * (size_t)p.N;
    const int mine = n < p.N ? left - (up ? 1 : 0) : 0;
    float least = 0.f;
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const float got = __uint_as_float(__shfl_xor_sync(kAll, up ? v[j] : v[j + 1], 16));
      const float own = __uint_as_float(up ? v[j + 1] : v[j]);
      const float g = up ? got : own;
      const float a = silu_times_near<false>(g, up ? own : got);
      least = fminf(least, g);
      if (j < mine) *y = __float2bfloat16_rn(a);
      y += step;
    }
    // (looked at once for all rows; a branch for each gate takes 64 experts, 8192
    // rows, N = 2048, K = 6144 from 295 us to 306; none at all 293)
    if (__any_sync(kAll, least < kGateFar)) {
      y -= 8 * step;
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        const float got = __uint_as_float(__shfl_xor_sync(kAll, up ? v[j] : v[j + 1], 16));
        const float own = __uint_as_float(up ? v[j + 1] : v[j]);
        const float a = silu_times_wide<false>(up ? got : own, up ? own : got);
        if (j < mine) *y = __float2bfloat16_rn(a);
        y += step;
      }
    }
  } else {
    const int n = ti.n0 + q * 32 + lane;
    if (n >= p.N) return;
    const size_t at = (size_t)(ti.row0 + c0) * p.N + n;
    if (p.y_bf16) {
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + at;
      if (left >= 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j, y += p.N) *y = __float2bfloat16_rn(__uint_as_float(v[j]));
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j, y += p.N)
          if (j < left) *y = __float2bfloat16_rn(__uint_as_float(v[j]));
      }
    } else {
      float* y = static_cast<float*>(p.y) + at;
      if (left >= 16) {
#pragma unroll
        for (int j = 0; j < 16; ++j, y += p.N) *y = __uint_as_float(v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j, y += p.N)
          if (j < left) *y = __uint_as_float(v[j]);
      }
    }
  }
}

template <int NT, bool GATED, int NW>
__global__ void __launch_bounds__(kThreads, 1) gemm_fp8_kernel(const __grid_constant__ GemmParams8 p) {
  using C = Cfg<NT, NW>;
  constexpr int COLS_W = GATED ? 64 : 128;   // output columns of a weight tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  uint8_t* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* ring_x = ring + C::WST * C::W_BYTES;
  Shared8& ss = *reinterpret_cast<Shared8*>(ring + C::RING);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  ptx::pdl_launch_dependents();
  if (warp == 1) {
    ptx::tmem_alloc(&ss.tmem_base, C::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::WST; ++i) {
      ptx::mbar_init(&ss.full[i], 2);
      ptx::mbar_init(&ss.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ss.sf_full[i], 4);
      ptx::mbar_init(&ss.sf_empty[i], 1);
    }
    for (int i = 0; i < C::ACC; ++i) {
      ptx::mbar_init(&ss.acc_full[i], 1);
      ptx::mbar_init(&ss.acc_empty[i], kEpiWarps);
    }
    ptx::mbar_init(&ss.drain, 1);
    ptx::mbar_init(&ss.sf_bar, 4);
    ss.abort = 0;
    ss.bad = 0;
    ptx::fence_barrier_init();
    ptx::tma_prefetch_desc(&p.x);
    ptx::tma_prefetch_desc(&p.w1);
    if (GATED) ptx::tma_prefetch_desc(&p.w3);
  }
  ptx::pdl_wait();
  for (int i = threadIdx.x; i <= p.G; i += kThreads)
    ss.gm.off[i] = p.offsets ? p.offsets[i] : i ? p.R : 0;
  __syncthreads();
  if (warp == 2) build_groups<NT>(ss.gm, p, lane);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();

  const uint32_t tmem = ss.tmem_base;
  const uint32_t sf_base = tmem + C::ACC * NT;
  volatile int* abort = &ss.abort;
  // a cluster of `split` CTAs works on the same tile, each on its K-blocks
  const int rank = p.split > 1 ? (int)ptx::cluster_rank() : 0;
  const int first = blockIdx.x / p.split, step = gridDim.x / p.split;
  Walk<GATED, NW> walk(ss.gm, p, first, step);
  const int kb0 = (int)((long long)p.KB * rank / p.split);
  const int kb1 = (int)((long long)p.KB * (rank + 1) / p.split);
  // scale words cover K-blocks 4s .. 4s + 3
  const int s0 = kb0 / 4, s1 = kb1 > kb0 ? (kb1 + 3) / 4 : s0;

  if (warp == 0 || warp == kRowWarp) {
    const bool wside = warp == 0;
    if (ptx::elect_one()) {
      // Both producers walk the weights' stages.  The row producer's own stage
      // is free when the products of the K-block XST back are done, which that
      // K-block's weight stage tells; since XST <= WST that barrier cannot have
      // moved on by another phase.
      int stage = 0, xs = 0, wait_at = 0, lag = wside ? C::WST : C::XST;
      uint32_t phase = 0, wait_phase = 0, issued = 0, parity = 0;
      bool ok = true;
      for (; ok && walk.more(); walk.next()) {
        const Tile8 ti = walk.tile(ss.gm, p);
        const int wrow = ti.g * p.N + ti.n0;
        const int boxes = (mma_rows(ti.rows) + C::XBOX - 1) / C::XBOX;
        const int bytes = wside ? C::W_BYTES : boxes * C::XBOX * kBK;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (lag > 0) {
            --lag;
          } else {
            if (!ptx::mbar_wait(&ss.empty[wait_at], wait_phase, abort)) { ok = false; break; }
            if (++wait_at == C::WST) { wait_at = 0; wait_phase ^= 1u; }
          }
          uint64_t* bar = &ss.full[stage];
          ptx::mbar_arrive_expect_tx(bar, bytes);
          auto load = [&](void* dst, const CUtensorMap* m, int row) {
            ptx::tma_load_2d(dst, m, bar, kb * kBK, row);
          };
          if (!wside) {
            uint8_t* dst = ring_x + xs * C::X_BYTES;
            if (++xs == C::XST) xs = 0;
            for (int j = 0; j < boxes; ++j)
              load(dst + j * C::XBOX * kBK, &p.x, ti.row0 + j * C::XBOX);
          } else if (GATED) {
            uint8_t* dst = ring + stage * C::W_BYTES;
#pragma unroll
            for (int j = 0; j < 4 * NW; ++j) {
              load(dst + j * 4096, &p.w1, wrow + j * 16);
              load(dst + j * 4096 + 2048, &p.w3, wrow + j * 16);
            }
          } else {
#pragma unroll
            for (int w = 0; w < NW; ++w)
              load(ring + stage * C::W_BYTES + w * kWTile, &p.w1, wrow + w * 128);
          }
          issued |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == C::WST) { stage = 0; phase ^= 1u; }
        }
      }
      // loads in flight end before the CTA does
      for (int s = 0; s < C::WST; ++s)
        if (issued & (1u << s)) ffn::wait_drain(&ss.full[s], (parity >> s) & 1u, abort);
    }
  } else if (warp == 1) {
    if (ptx::elect_one()) {
      const uint32_t desc_w = ptx::desc_sw128_lo(ptx::smem_addr(ring));
      const uint32_t desc_x = ptx::desc_sw128_lo(ptx::smem_addr(ring_x));
      int ws = 0, xs = 0, buf = 0, slot = 0;
      uint32_t phase = 0, aphase = 0, sphase = 0;
      bool ok = true;
      for (; ok && walk.more(); walk.next()) {
        const Tile8 ti = walk.tile(ss.gm, p);
        const uint32_t idesc = ptx::idesc_mxf8(128, mma_rows(ti.rows));
        // the products of K-block kb with weight tile w, from a stage
        auto products = [&](int w, int acc, int kb, int wstage, int xstage) {
          const uint32_t da = desc_w + wstage * (C::W_BYTES >> 4) + w * (kWTile >> 4);
          const uint32_t db = desc_x + xstage * (C::X_BYTES >> 4);
          const uint32_t id = idesc | ptx::idesc_sf_byte(kb & 3, kb & 3);
          const uint32_t sf = sf_base + slot * C::SF_SLOT;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            ptx::mma_mxf8_ss(tmem + acc * NT, ptx::desc_sw128(da + 2 * k), ptx::desc_sw128(db + 2 * k),
                             id, sf + 4 * w, sf + 4 * NW, k > 0 ? 1u : kb > kb0);
        };
        auto next_acc = [&] {
          if (++buf == C::ACC) { buf = 0; aphase ^= 1u; }
        };
        if (!ptx::mbar_wait(&ss.acc_empty[buf], aphase ^ 1u, abort)) break;
        const int acc0 = buf;
        int lead = kb0;                  // K-blocks that the first weight tile is done with
        if (NW == 2) {
          // while the second accumulator is still being stored, the first weight
          // tile goes ahead: by the K-blocks that the ring and a scale slot hold
          next_acc();
          if (!ptx::mbar_wait(&ss.sf_full[slot], sphase, abort)) break;
          int ls = ws;
          uint32_t lphase = phase;
          const int most = min(kb1, C::WST < 4 ? C::WST : 4);
          while (ok && lead < most && !ptx::mbar_test(&ss.acc_empty[buf], aphase ^ 1u)) {
            ok = ptx::mbar_wait(&ss.full[ls], lphase, abort);
            ptx::tc_fence_after();
            if (ok) products(0, acc0, lead++, ls, ls);
            if (++ls == C::WST) { ls = 0; lphase ^= 1u; }
          }
          if (!ok || !ptx::mbar_wait(&ss.acc_empty[buf], aphase ^ 1u, abort)) break;
        }
        for (int kb = kb0; kb < kb1; ++kb) {
          if (kb == kb0 || (kb & 3) == 0) {
            if (!ptx::mbar_wait(&ss.sf_full[slot], sphase, abort)) { ok = false; break; }
          }
          if (!ptx::mbar_wait(&ss.full[ws], phase, abort)) { ok = false; break; }
          ptx::tc_fence_after();
          if (NW == 1 || kb >= lead) products(0, acc0, kb, ws, xs);
          if (NW == 2) {
            if (kb == kb1 - 1) ptx::mma_commit(&ss.acc_full[acc0]);
            products(1, buf, kb, ws, xs);
          }
          ptx::mma_commit(&ss.empty[ws]);
          if (++ws == C::WST) { ws = 0; phase ^= 1u; }
          if (++xs == C::XST) xs = 0;
          if ((kb & 3) == 3 || kb == kb1 - 1) {
            ptx::mma_commit(&ss.sf_empty[slot]);
            if (++slot == 2) { slot = 0; sphase ^= 1u; }
          }
        }
        if (!ok) break;
        ptx::mma_commit(&ss.acc_full[buf]);
        next_acc();
      }
      // nothing is in flight when tensor memory is freed
      ptx::mma_commit(&ss.drain);
      ffn::wait_drain(&ss.drain, 0, abort);
    }
  } else if (warp < kSfWarp0) {
    const int q = warp & 3;              // TMEM lane quarter of this warp
    const int half = (warp - 2) >> 2;    // its turn of 16 rows among the quarter's two warps
    int buf = 0, w = 0;
    uint32_t aphase = 0;
    while (walk.more()) {
      Tile8 ti = walk.tile(ss.gm, p);
      ti.n0 += w * COLS_W;
      if (__any_sync(kAll, !ptx::mbar_wait(&ss.acc_full[buf], aphase, abort))) break;
      ptx::tc_fence_after();
      const uint32_t acc = tmem + buf * NT + ((uint32_t)(q * 32) << 16);
      auto use = [&](int c, const uint32_t (&v)[16]) {
        if (NW == 1 && p.split > 1) {
          // this CTA's part of the tile, [row][weight row], in the ring (all its
          // loads and products are done, and a cluster has one tile)
          float* part = reinterpret_cast<float*>(ring) + (size_t)c * 128 + q * 32 + lane;
#pragma unroll
          for (int j = 0; j < 16; ++j) part[j * 128] = __uint_as_float(v[j]);
        } else {
          store16<GATED>(p, ti, q, lane, c, v);
        }
      };
      // sixteen columns are read while the sixteen before them are stored
      uint32_t a[16], b[16];
      int c = half * 16;
      if (c < ti.rows) ptx::tmem_ld_x16(acc + c, a);
      for (; c < ti.rows; c += 64) {
        ptx::tmem_wait_ld();
        if (c + 32 < ti.rows) ptx::tmem_ld_x16(acc + c + 32, b);
        use(c, a);
        if (c + 32 < ti.rows) {
          ptx::tmem_wait_ld();
          if (c + 64 < ti.rows) ptx::tmem_ld_x16(acc + c + 64, a);
          use(c + 32, b);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(&ss.acc_empty[buf]);
      if (++buf == C::ACC) { buf = 0; aphase ^= 1u; }
      if (++w == NW) { w = 0; walk.next(); }
    }
  } else {
    constexpr int RPT = (NT + 127) / 128;      // rows per thread
    constexpr int XC = (NT + 31) / 32;         // scale columns of the rows
    const int tid = threadIdx.x - kSfWarp0 * 32;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    ptx::WarpBarrier team_bar{&ss.sf_bar};
    int slot = 0, sbuf = 0;
    uint32_t sphase = 0;
    bool bad = false, ok = true;
    // chunk c: K-blocks 16 c .. 16 c + 15, scale sets 4 c .. 4 c + 3
    const int c0 = s0 / 4, c1 = (s1 + 3) / 4;
    uint32_t xw[RPT][4], ww[NW][4];
    auto load = [&](const Tile8& ti, int c) {
      const int n = min(16, p.KB - 16 * c);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int r = tid + 128 * i;
        if (r < ti.rows)
          load_exps(p.xe + (size_t)(ti.row0 + r) * p.KB + 16 * c, n, p.xe,
                    p.xe + (size_t)p.R * p.KB, xw[i]);
      }
      const int8_t* we = GATED && (lane & 16) ? p.w3e : p.w1e;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        // (a second weight tile may lie behind the last column: any scale will do)
        const int nb = min((ti.n0 + w * COLS_W) / 128, p.NB - 1);
        load_exps(we + ((size_t)ti.g * p.NB + nb) * p.KB + 16 * c, n, we,
                  we + (size_t)p.G * p.NB * p.KB, ww[w]);
      }
    };
    int c = c0;
    Tile8 ti{};
    if (walk.more()) {
      ti = walk.tile(ss.gm, p);
      load(ti, c);
    }
    while (ok && walk.more()) {
      const int n = min(16, p.KB - 16 * c);
      uint32_t wa[NW][4];
#pragma unroll
      for (int w = 0; w < NW; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) wa[w][i] = scale_bytes(ww[w][i], i, n, &bad);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int r = tid + 128 * i;
        if (r < ti.rows) {
#pragma unroll
          for (int j = 0; j < 4; ++j) ss.sf_rows[sbuf][j][r] = scale_bytes(xw[i][j], j, n, &bad);
        }
      }
      const int rows = ti.rows;
      const int beg = max(4 * c, s0), end = min(4 * c + 4, s1);
      const int cur = 4 * c;
      // the next chunk's exponents are on their way while this one is used
      if (++c == c1) {
        c = c0;
        walk.next();
        if (walk.more()) ti = walk.tile(ss.gm, p);
      }
      if (walk.more()) load(ti, c);
      if (!team_bar.sync(abort, lane)) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int s = cur + j;
        if (s < beg || s >= end) continue;
        uint32_t wx[8];
#pragma unroll
        for (int i = 0; i < XC; ++i) wx[i] = ss.sf_rows[sbuf][j][i * 32 + lane];
        if (__any_sync(kAll, !ptx::mbar_wait(&ss.sf_empty[slot], sphase ^ 1u, abort))) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t dst = sf_base + slot * C::SF_SLOT + lanes, dx = dst + 4 * NW;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const uint32_t w4[4] = {wa[w][j], wa[w][j], wa[w][j], wa[w][j]};
          ptx::tmem_st_x4(dst + 4 * w, w4);
        }
        // (words of rows behind the tile's last are whatever stood there)
        if (XC > 4 && rows > 128) ptx::tmem_st_x8(dx, wx);
        else if (XC > 1) ptx::tmem_st_x4(dx, wx);
        else ptx::tmem_st_x1(dx, wx[0]);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ss.sf_full[slot]);
        if (++slot == 2) { slot = 0; sphase ^= 1u; }
      }
      sbuf ^= 1;
    }
    if (bad) ss.bad = 1;
  }

  __syncthreads();
  if (NW == 1 && p.split > 1) {
    // partial tiles -> outputs: rank r finishes the rows r, r + split, ...
    ptx::cluster_sync();
    Walk<GATED, NW> own(ss.gm, p, first, step);
    if (own.more() && !*abort) {
      const Tile8 ti = own.tile(ss.gm, p);
      const uint32_t part = ptx::smem_addr(ring);
      // a thread finishes four neighbouring weight rows; the parts of all ranks
      // are on their way before the first is added
      constexpr int QUADS = GATED ? 16 : 32;     // of output columns in a row of the tile
      for (int i = threadIdx.x; i < ti.rows * QUADS; i += kThreads) {
        const int c = i / QUADS, f = (i % QUADS) * 4;
        if (c % p.split != rank || ti.n0 + f >= p.N) continue;
        const uint32_t at = part + (c * 128 + (GATED ? (f >> 4) * 32 + (f & 15) : f)) * 4;
        float4 v[8], w[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < p.split) {
            v[r] = ptx::ld_cluster_f32x4(at, r);
            if (GATED) w[r] = ptx::ld_cluster_f32x4(at + 64, r);
          }
        float4 s = v[0], u = w[0];
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < p.split) {
            s.x += v[r].x; s.y += v[r].y; s.z += v[r].z; s.w += v[r].w;
            if (GATED) { u.x += w[r].x; u.y += w[r].y; u.z += w[r].z; u.w += w[r].w; }
          }
        if (GATED) {
          s.x = silu_times_wide<false>(s.x, u.x); s.y = silu_times_wide<false>(s.y, u.y);
          s.z = silu_times_wide<false>(s.z, u.z); s.w = silu_times_wide<false>(s.w, u.w);
        }
        // (N is a multiple of 8: four columns are all there or not at all)
        const size_t out = (size_t)(ti.row0 + c) * p.N + ti.n0 + f;
        if (GATED || p.y_bf16)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + out) =
              make_uint2(ffn::pack_bf16(s.x, s.y), ffn::pack_bf16(s.z, s.w));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(p.y) + out) = s;
      }
    }
    ptx::cluster_sync();   // no CTA leaves while another reads its part
  }
  if (warp == 1) ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  if (threadIdx.x == 0 && p.status) {
    if (ss.abort) atomicOr(p.status, kStTimeout);
    if (ss.bad) atomicOr(p.status, kStBounds);
  }
}

template <int NT, bool GATED, int NW>
cudaError_t launch_nt(const GemmParams8& p, long long tiles, cudaStream_t st) {
  constexpr int smem = smem_bytes8<NT, NW>();
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_once(gemm_fp8_kernel<NT, GATED, NW>, smem, smem_set);
  if (e != cudaSuccess) return e;
  const long long want = tiles * p.split, sms = num_sms();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.split > 1 ? want : std::min(want, sms)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_fp8_kernel<NT, GATED, NW>, p);
}

template <int NT, int NW, bool GATED>
cudaError_t launch_any(GemmParams8& p, cudaStream_t st, const char** why, const Gemm8Args& a) {
  const uint32_t box = GATED ? 16 : 128;
  bool ok = make_tensor_map(&p.x, a.x, a.R, a.K, Cfg<NT, NW>::XBOX, kBK, 1, 128) &&
            make_tensor_map(&p.w1, a.W1, (uint64_t)a.G * a.N, a.K, box, kBK, 1, 128);
  p.w3 = p.w1;
  if (ok && GATED) ok = make_tensor_map(&p.w3, a.W3, (uint64_t)a.G * a.N, a.K, box, kBK, 1, 128);
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed for a product operand";
    return cudaErrorInvalidValue;
  }
  constexpr int COLS = (GATED ? 64 : 128) * NW;
  p.nt = (a.N + COLS - 1) / COLS;
  // row blocks: at most one per group with rows, and one per NT rows
  const long long blocks = std::min<long long>(a.R, (long long)a.R / NT + std::min(a.G, a.R));
  const long long tiles = blocks * p.nt;
  // Few tiles: split K over a cluster while that leaves every CTA an SM of its
  // own and two K-blocks, and takes at least nine K-blocks off each: joining
  // the parts costs about 2 us.  (Graph times: 20 groups of 58 rows, N = 32, K =
  // 4688 12.0 us split against 13.7; 13 groups of 6 rows, N = 8, K = 4192 gated
  // 8.4 against 11.7; one row, N = 6144, K = 2048 8.3 against 7.5, which is why
  // eight K-blocks are not enough.)
  p.split = 1;
  for (int s = 2; NW == 1 && s <= 8; s *= 2)
    if (tiles * s <= num_sms() && p.KB >= s * 2 && p.KB - p.KB / s >= 9) p.split = s;
  return launch_nt<NT, GATED, NW>(p, tiles, st);
}

// Rows per tile.  240 (two accumulators of that width fill tensor memory) read
// the weights for the most rows; narrower tiles leave shared memory to the
// weights' ring.  So: the narrowest that cuts a group into no more blocks than
// 240 would, for groups two standard deviations above the average; and narrower
// still while a quarter of the SMs have no tile.  (17 groups of 632 rows, N = 40,
// K = 528 gated: 10.0 us narrowed against 13.3; 73 groups of 297, N = 24, K =
// 144, with a tile for 146 of 148 SMs: 12.7 narrowed against 9.6.)
//
// Two weight tiles for the rows of a stage, where the tiles are many: halving
// their number must not leave SMs idle at the end, and the epilogue, which the
// next tile covers only in part, must be small beside the products.  At 160 rows
// three accumulators fit, so from 8 tiles an SM on (128 groups of 256 rows, N =
// 4096: 117 us against 136 at K = 512, 252 against 286 at K = 1408; gated 576
// against 675; 5 tiles an SM, 128 groups of 125 rows, N = 768, K = 1024: 37.1
// against 35.3).  At 240 rows only two fit, which 32 K-blocks make up for (one
// group of 8192 rows, N = 8192: 372 us against 400 at K = 6144, 133 against 125 at
// K = 2048); the gated epilogue is longer, and there 160 rows are faster (K = 6144:
// 724 against 766, and 765 with one weight tile).
template <bool GATED>
cudaError_t launch_rows(GemmParams8& p, cudaStream_t st, const char** why, const Gemm8Args& a) {
  // (sizes end 256 below 2^31, so that a tile's width can be added to them)
  const int groups = std::min(a.G, a.R), avg = (a.R - 1) / groups + 1;
  const int top = a.G > 1 ? avg + (int)(2.f * sqrtf((float)avg)) : avg;
  const int nb = (top + 239) / 240, need = (top - 1) / nb + 1;
  constexpr int widths[] = {32, 64, 96, 144, 160, 240};
  int w = 0;
  while (widths[w] < need) ++w;
  const long long cols = GATED ? (a.N + 63) / 64 : (a.N + 127) / 128;
  auto tiles = [&] { return (long long)groups * ((avg + widths[w] - 1) / widths[w]) * cols; };
  while (w > 0 && tiles() < num_sms() * 3 / 4) --w;
  const bool long_k = p.KB >= 32;
  if (widths[w] > 96 && (widths[w] < 240 || long_k) && tiles() >= (long_k ? 4 : 8) * num_sms()) {
    if constexpr (!GATED)
      if (widths[w] == 240) return launch_any<240, 2, GATED>(p, st, why, a);
    return launch_any<160, 2, GATED>(p, st, why, a);
  }
  switch (widths[w]) {
    case 32: return launch_any<32, 1, GATED>(p, st, why, a);
    case 64: return launch_any<64, 1, GATED>(p, st, why, a);
    case 96: return launch_any<96, 1, GATED>(p, st, why, a);
    case 144: return launch_any<144, 1, GATED>(p, st, why, a);
    case 160: return launch_any<160, 1, GATED>(p, st, why, a);
    default: return launch_any<240, 1, GATED>(p, st, why, a);
  }
}

}  // namespace

cudaError_t launch_gemm_fp8(const Gemm8Args& a, cudaStream_t st, const char** why) {
  GemmParams8 p{};
  p.xe = a.xe;
  p.w1e = a.W1e;
  p.w3e = a.W3e;
  p.offsets = a.offsets;
  p.y = a.y;
  p.y_bf16 = a.y_bf16;
  p.G = a.G; p.R = a.R; p.N = a.N; p.K = a.K;
  p.KB = (a.K + 127) / 128;
  p.NB = (a.N + 127) / 128;
  p.status = a.status;
  *why = "product launch";
  return a.W3 ? launch_rows<true>(p, st, why, a) : launch_rows<false>(p, st, why, a);
}

}  // namespace moe
