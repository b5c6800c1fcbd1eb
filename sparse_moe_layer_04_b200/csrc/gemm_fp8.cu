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
// CTA structure (320 threads, tiles taken round-robin):
//   warp 0      TMA producer: weight tile (128 x 128 codes) and row tile
//               (NT x 128 codes), 128-byte swizzled, into a ring of stages
//   warp 1      TMEM allocator and MMA issuer (one elected thread)
//   warps 2-5   epilogue: TMEM -> registers -> global; two accumulators, so
//               a tile's epilogue overlaps the next tile's products
//   warps 6-9   scale writers: the exponents of sixteen K-blocks at a time,
//               loaded a row per thread while the sixteen before them are in
//               use, exchanged through shared memory, and written as 32-bit
//               words of four E8M0 bytes into one of two TMEM slots; each of
//               the four warps fills its lane quarter with the same words, as
//               the tensor core expects them
// Gated tiles hold 64 output columns: the 128 weight rows alternate 16 of W1
// and 16 of W3, so every warp's lanes 0-15 hold gates and lanes 16-31 the ups
// of the same columns, which one shuffle per pair of rows brings together.
//
// Large groups run on pairs of CTAs (PAIR): one product of M = 256 weight rows,
// 128 from each CTA, whose row operand is split between the two, so a CTA
// stages half the rows per product.  Both CTAs' loads complete on the first
// one's barriers, it issues the products, and their completion is signalled
// to both; each CTA writes its own scales and stores its own output columns.
//
// Few tiles (one row through one matrix): a cluster of CTAs shares a tile,
// each with its own range of K-blocks, and adds the partial tiles through
// distributed shared memory in rank order, so results do not depend on timing.
#include <algorithm>

#include <cuda_bf16.h>

#include "ffn_common.cuh"
#include "sm100_scaled.cuh"

namespace moe {
namespace {

constexpr int kBK = 128;                 // K elements of a stage = one exponent
constexpr int kWTile = 128 * kBK;        // weight tile bytes
constexpr int kThreads = 320;
constexpr int kMaxStages = 11;
constexpr int kMaxG = 1024;
constexpr int kSfSlotCols = 12;          // 4 columns for the weights, 8 for the rows
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
  int nt;               // output column tiles of a group (PAIR: pairs of them)
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

template <int NT, bool PAIR>
struct Cfg {
  // rows of one TMA box of the row operand, and of a stage's share of it: a
  // tile loads only as many boxes as its rows need
  static constexpr int XROWS = PAIR ? NT / 2 : NT;
  static constexpr int XBOX = PAIR ? 24 : NT < 48 ? NT : 32;
  static constexpr int X_BYTES = XROWS * kBK;
  static constexpr int STAGE = kWTile + X_BYTES;
  static constexpr int STAGES = (200 * 1024) / STAGE < kMaxStages ? (200 * 1024) / STAGE : kMaxStages;
  static constexpr int SF_COLS = 2 * kSfSlotCols;
  static constexpr uint32_t TMEM_COLS = 2 * NT + SF_COLS <= 128   ? 128
                                        : 2 * NT + SF_COLS <= 256 ? 256
                                                                  : 512;
  static_assert(2 * NT + SF_COLS <= 512 && NT % 16 == 0 && NT <= 240, "tensor memory columns");
  static_assert(XROWS % XBOX == 0 && XBOX % 8 == 0 && X_BYTES % 1024 == 0, "row boxes");
};

struct Shared8 {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t sf_full[2], sf_empty[2];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint64_t sf_bar;             // barrier of the four scale warps
  uint32_t tmem_base;
  int abort;
  int bad;
  uint32_t sf_rows[2][4][256]; // scale words of sixteen K-blocks [set][row]
  GroupMap gm;
};

template <int NT, bool PAIR>
constexpr int smem_bytes8() {
  return 1024 + Cfg<NT, PAIR>::STAGES * Cfg<NT, PAIR>::STAGE + (int)sizeof(Shared8);
}

__device__ __forceinline__ int blocks_of(int rows, int nt) { return (rows + nt - 1) / nt; }

// Rows of the product's row operand: the tile's, in steps of 16.
__device__ __forceinline__ int mma_rows(int rows) { return max(16, (rows + 15) / 16 * 16); }

// One warp: checks the offsets and counts each group's row blocks.  Offsets
// that are not increasing within [0, R] give no tiles and raise kStBounds.
template <int NT>
__device__ void build_groups(GroupMap& gm, const GemmParams8& p, int lane) {
  int carry = 0;
  bool bad = false;
  for (int base = 0; base < p.G; base += 32) {
    const int g = base + lane;
    int cnt = 0;
    if (g < p.G) {
      const int a = p.offsets ? p.offsets[g] : 0;
      const int b = p.offsets ? p.offsets[g + 1] : p.R;
      gm.off[g] = a;
      if (g == p.G - 1) gm.off[p.G] = b;
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

// Tile t: groups in order, then output column tiles, row blocks fastest (the
// CTAs that run together share weight tiles through L2).
// `rank`: this CTA's half of a pair's columns.
template <int NT, bool GATED, bool PAIR>
__device__ __forceinline__ Tile8 tile_at(int t, const GroupMap& gm, const GemmParams8& p, int rank) {
  const int q = t / p.nt;
  int lo = 0, hi = p.G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (gm.prefix[mid] <= q) lo = mid; else hi = mid - 1;
  }
  const int rows = gm.off[lo + 1] - gm.off[lo];
  const int nb = blocks_of(rows, NT);
  const int local = t - gm.prefix[lo] * p.nt;
  const int per = (blocks_of(rows, nb) + 15) / 16 * 16;   // rows per block
  const int b = local % nb;
  Tile8 ti;
  ti.g = lo;
  ti.n0 = (PAIR ? local / nb * 2 + rank : local / nb) * (GATED ? 64 : 128);
  ti.row0 = gm.off[lo] + b * per;
  ti.rows = max(0, min(per, rows - b * per));
  return ti;
}

// Exponents q[0 .. n-1] (n <= 16) as they stand in memory, in words of four.
// Any alignment: the aligned words that hold them are loaded and shifted.
__device__ __forceinline__ void load_exps(const int8_t* q, int n, uint32_t (&w)[4]) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(q);
  const uint32_t* base = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
  const int off = (int)(at & 3);
  uint32_t v[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = 4 * i - off < n ? __ldg(base + i) : 0u;
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

// Sixteen accumulator columns (rows of the group) of one weight row per
// lane -> outputs.
template <bool GATED>
__device__ __forceinline__ void store16(const GemmParams8& p, const Tile8& ti, int q, int lane,
                                        int c0, const float (&v)[16]) {
  if (GATED) {
    // lanes 0-15 finish the even rows of each pair, lanes 16-31 the odd ones
    const bool up = lane >= 16;
    const int n = ti.n0 + q * 16 + (lane & 15);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y);
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const float got = __shfl_xor_sync(kAll, up ? v[j] : v[j + 1], 16);
      const float gate = up ? got : v[j];
      const float mul = up ? v[j + 1] : got;
      const int c = c0 + j + (up ? 1 : 0);
      if (c < ti.rows && n < p.N)
        y[(size_t)(ti.row0 + c) * p.N + n] = __float2bfloat16_rn(ffn::silu_times(gate, mul));
    }
  } else {
    const int n = ti.n0 + q * 32 + lane;
    if (n >= p.N) return;
    if (p.y_bf16) {
      __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y) + (size_t)(ti.row0 + c0) * p.N + n;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c0 + j < ti.rows) y[(size_t)j * p.N] = __float2bfloat16_rn(v[j]);
    } else {
      float* y = static_cast<float*>(p.y) + (size_t)(ti.row0 + c0) * p.N + n;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c0 + j < ti.rows) y[(size_t)j * p.N] = v[j];
    }
  }
}

template <int NT, bool GATED, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1) gemm_fp8_kernel(const __grid_constant__ GemmParams8 p) {
  using C = Cfg<NT, PAIR>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  uint8_t* ring = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  Shared8& ss = *reinterpret_cast<Shared8*>(ring + STAGES * C::STAGE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  ptx::pdl_launch_dependents();
  if (warp == 1) {
    if (PAIR) {
      ptx::tmem_alloc_pair(&ss.tmem_base, C::TMEM_COLS);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(&ss.tmem_base, C::TMEM_COLS);
      ptx::tmem_relinquish();
    }
  }
  if (threadIdx.x == 0) {
    // a pair's products wait on the first CTA's barriers, which both CTAs' scale
    // writers and epilogues arrive on
    for (int i = 0; i < STAGES; ++i) {
      ptx::mbar_init(&ss.full[i], 1);
      ptx::mbar_init(&ss.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ss.sf_full[i], PAIR ? 8 : 4);
      ptx::mbar_init(&ss.sf_empty[i], 1);
      ptx::mbar_init(&ss.acc_full[i], 1);
      ptx::mbar_init(&ss.acc_empty[i], PAIR ? 8 : 4);
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
  if (warp == 2) build_groups<NT>(ss.gm, p, lane);
  ptx::tc_fence_before();
  __syncthreads();
  if (PAIR) ptx::cluster_sync();   // the barriers of both CTAs are initialised
  ptx::tc_fence_after();

  const uint32_t tmem = ss.tmem_base;
  const uint32_t sf_base = tmem + 2 * NT;
  volatile int* abort = &ss.abort;
  // a cluster of `split` CTAs works on the same tiles, each on its K-blocks (or,
  // as a pair, each on its columns of all of them)
  const int rank = p.split > 1 || PAIR ? (int)ptx::cluster_rank() : 0;
  const int team = PAIR ? 2 : p.split;
  const int first = blockIdx.x / team, step = gridDim.x / team;
  const int total = ss.gm.total * p.nt;
  const int kb0 = PAIR ? 0 : (int)((long long)p.KB * rank / p.split);
  const int kb1 = PAIR ? p.KB : (int)((long long)p.KB * (rank + 1) / p.split);
  // scale words cover K-blocks 4s .. 4s + 3
  const int s0 = kb0 / 4, s1 = kb1 > kb0 ? (kb1 + 3) / 4 : s0;

  if (warp == 0) {
    if (ptx::elect_one()) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      bool ok = true;
      for (int t = first; ok && t < total; t += step) {
        const Tile8 ti = tile_at<NT, GATED, PAIR>(t, ss.gm, p, rank);
        const int wrow = ti.g * p.N + ti.n0;
        const int n = mma_rows(ti.rows);
        const int xn = PAIR ? n / 2 : n;           // rows this CTA stages
        const int xrow = ti.row0 + (PAIR ? rank * xn : 0);
        const int boxes = (xn + C::XBOX - 1) / C::XBOX;
        const int bytes = kWTile + boxes * C::XBOX * kBK;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!ptx::mbar_wait(&ss.empty[stage], phase ^ 1u, abort)) { ok = false; break; }
          uint8_t* sw = ring + stage * C::STAGE;
          uint64_t* bar = &ss.full[stage];
          if (PAIR) {
            const uint32_t lead = ptx::map_rank(bar, 0);
            if (rank == 0) ptx::mbar_arrive_expect_tx(bar, 2 * bytes);
            if (GATED) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                ptx::tma_load_2d_pair(sw + j * 4096, &p.w1, lead, kb * kBK, wrow + j * 16);
                ptx::tma_load_2d_pair(sw + j * 4096 + 2048, &p.w3, lead, kb * kBK, wrow + j * 16);
              }
            } else {
              ptx::tma_load_2d_pair(sw, &p.w1, lead, kb * kBK, wrow);
            }
            for (int j = 0; j < boxes; ++j)
              ptx::tma_load_2d_pair(sw + kWTile + j * C::XBOX * kBK, &p.x, lead, kb * kBK,
                                    xrow + j * C::XBOX);
          } else {
            ptx::mbar_arrive_expect_tx(bar, bytes);
            if (GATED) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                ptx::tma_load_2d(sw + j * 4096, &p.w1, bar, kb * kBK, wrow + j * 16);
                ptx::tma_load_2d(sw + j * 4096 + 2048, &p.w3, bar, kb * kBK, wrow + j * 16);
              }
            } else {
              ptx::tma_load_2d(sw, &p.w1, bar, kb * kBK, wrow);
            }
            for (int j = 0; j < boxes; ++j)
              ptx::tma_load_2d(sw + kWTile + j * C::XBOX * kBK, &p.x, bar, kb * kBK,
                               xrow + j * C::XBOX);
          }
          issued |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      // loads in flight end before the CTA does; a pair's second CTA sees its
      // loads' stages released (their products have read them)
      for (int s = 0; s < STAGES; ++s)
        if (issued & (1u << s)) {
          if (!PAIR || rank == 0) ffn::wait_drain(&ss.full[s], (parity >> s) & 1u, abort);
          else ffn::wait_drain(&ss.empty[s], (parity >> s) & 1u, abort);
        }
    }
  } else if (warp == 1) {
    if ((!PAIR || rank == 0) && ptx::elect_one()) {
      auto commit = [](uint64_t* bar) {
        if (PAIR) ptx::mma_commit_pair(bar); else ptx::mma_commit(bar);
      };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return PAIR ? ptx::mbar_wait_cluster(bar, parity, abort) : ptx::mbar_wait(bar, parity, abort);
      };
      int stage = 0, buf = 0, slot = 0;
      uint32_t phase = 0, aphase = 0, sphase = 0;
      bool ok = true;
      for (int t = first; ok && t < total; t += step) {
        const Tile8 ti = tile_at<NT, GATED, PAIR>(t, ss.gm, p, rank);
        const uint32_t idesc = ptx::idesc_mxf8(PAIR ? 256 : 128, mma_rows(ti.rows));
        if (!wait(&ss.acc_empty[buf], aphase ^ 1u)) break;
        const uint32_t acc = tmem + buf * NT;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (kb == kb0 || (kb & 3) == 0) {
            if (!wait(&ss.sf_full[slot], sphase)) { ok = false; break; }
          }
          if (!wait(&ss.full[stage], phase)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t sw = ptx::smem_addr(ring + stage * C::STAGE);
          const uint64_t da = ptx::smem_desc_sw128(sw);
          const uint64_t db = ptx::smem_desc_sw128(sw + kWTile);
          const uint32_t id = idesc | ptx::idesc_sf_byte(kb & 3, kb & 3);
          const uint32_t sfa = sf_base + slot * kSfSlotCols, sfb = sfa + 4;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (PAIR)
              ptx::mma_mxf8_ss_pair(acc, da + 2 * k, db + 2 * k, id, sfa, sfb, kb > kb0 || k > 0);
            else
              ptx::mma_mxf8_ss(acc, da + 2 * k, db + 2 * k, id, sfa, sfb, kb > kb0 || k > 0);
          }
          commit(&ss.empty[stage]);
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          if ((kb & 3) == 3 || kb == kb1 - 1) {
            commit(&ss.sf_empty[slot]);
            if (++slot == 2) { slot = 0; sphase ^= 1u; }
          }
        }
        if (!ok) break;
        commit(&ss.acc_full[buf]);
        if (++buf == 2) { buf = 0; aphase ^= 1u; }
      }
      // nothing is in flight when tensor memory is freed
      commit(&ss.drain);
      ffn::wait_drain(&ss.drain, 0, abort);
    }
  } else if (warp < 6) {
    const int q = warp & 3;              // TMEM lane quarter of this warp
    int buf = 0;
    uint32_t aphase = 0;
    for (int t = first; t < total; t += step) {
      const Tile8 ti = tile_at<NT, GATED, PAIR>(t, ss.gm, p, rank);
      if (__any_sync(kAll, !ptx::mbar_wait(&ss.acc_full[buf], aphase, abort))) break;
      ptx::tc_fence_after();
      const uint32_t acc = tmem + buf * NT + ((uint32_t)(q * 32) << 16);
      for (int c = 0; c < ti.rows; c += 16) {
        uint32_t r[16];
        ptx::tmem_ld_x16(acc + c, r);
        ptx::tmem_wait_ld();
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = kb1 > kb0 ? __uint_as_float(r[j]) : 0.f;
        if (p.split > 1) {
          // this CTA's part of the tile, [row][weight row], in the ring (all
          // its loads and products are done, and a cluster has one tile)
          float* part = reinterpret_cast<float*>(ring);
#pragma unroll
          for (int j = 0; j < 16; ++j) part[(c + j) * 128 + q * 32 + lane] = v[j];
        } else {
          store16<GATED>(p, ti, q, lane, c, v);
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) ptx::mbar_arrive_cluster(ptx::map_rank(&ss.acc_empty[buf], 0));
        else ptx::mbar_arrive(&ss.acc_empty[buf]);
      }
      if (++buf == 2) { buf = 0; aphase ^= 1u; }
    }
  } else {
    constexpr int RPT = (NT + 127) / 128;      // rows per thread
    constexpr int XC = (NT + 31) / 32;         // scale columns of the rows
    const int tid = threadIdx.x - 192;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    ptx::WarpBarrier team_bar{&ss.sf_bar};
    int slot = 0, sbuf = 0;
    uint32_t sphase = 0;
    bool bad = false, ok = true;
    // chunk c: K-blocks 16 c .. 16 c + 15, scale sets 4 c .. 4 c + 3
    const int c0 = s0 / 4, c1 = (s1 + 3) / 4;
    uint32_t xw[RPT][4], ww[4];
    auto load = [&](const Tile8& ti, int c) {
      const int n = min(16, p.KB - 16 * c);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const int r = tid + 128 * i;
        if (r < ti.rows) load_exps(p.xe + (size_t)(ti.row0 + r) * p.KB + 16 * c, n, xw[i]);
      }
      // (a pair's second tile may lie behind the last column: any scale will do)
      load_exps((GATED && (lane & 16) ? p.w3e : p.w1e) +
                    ((size_t)ti.g * p.NB + min(ti.n0 / 128, p.NB - 1)) * p.KB + 16 * c,
                n, ww);
    };
    int t = first, c = c0;
    Tile8 ti{};
    if (t < total) {
      ti = tile_at<NT, GATED, PAIR>(t, ss.gm, p, rank);
      load(ti, c);
    }
    while (ok && t < total) {
      const int n = min(16, p.KB - 16 * c);
      uint32_t wa[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) wa[i] = scale_bytes(ww[i], i, n, &bad);
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
        t += step;
        if (t < total) ti = tile_at<NT, GATED, PAIR>(t, ss.gm, p, rank);
      }
      if (t < total) load(ti, c);
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
        const uint32_t dst = sf_base + slot * kSfSlotCols + lanes;
        const uint32_t w4[4] = {wa[j], wa[j], wa[j], wa[j]};
        ptx::tmem_st_x4(dst, w4);
        // (words of rows behind the tile's last are whatever stood there)
        if (XC > 4 && rows > 128) ptx::tmem_st_x8(dst + 4, wx);
        else if (XC > 1) ptx::tmem_st_x4(dst + 4, wx);
        else ptx::tmem_st_x1(dst + 4, wx[0]);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) ptx::mbar_arrive_cluster(ptx::map_rank(&ss.sf_full[slot], 0));
          else ptx::mbar_arrive(&ss.sf_full[slot]);
        }
        if (++slot == 2) { slot = 0; sphase ^= 1u; }
      }
      sbuf ^= 1;
    }
    if (bad) ss.bad = 1;
  }

  __syncthreads();
  if (PAIR) ptx::cluster_sync();   // neither CTA leaves while the other uses its memory
  if (!PAIR && p.split > 1) {
    // partial tiles -> outputs: rank r finishes the rows r, r + split, ...
    ptx::cluster_sync();
    if (first < total && !*abort) {
      const Tile8 ti = tile_at<NT, GATED, PAIR>(first, ss.gm, p, rank);
      const uint32_t part = ptx::smem_addr(ring);
      if (GATED) {
        for (int i = threadIdx.x; i < ti.rows * 64; i += kThreads) {
          const int c = i >> 6, f = i & 63;
          if (c % p.split != rank) continue;
          const uint32_t at = part + (c * 128 + (f >> 4) * 32 + (f & 15)) * 4;
          float g = 0.f, u = 0.f;
          for (int r = 0; r < p.split; ++r) {
            g += ptx::ld_cluster_f32(at, r);
            u += ptx::ld_cluster_f32(at + 64, r);
          }
          if (ti.n0 + f < p.N)
            static_cast<__nv_bfloat16*>(p.y)[(size_t)(ti.row0 + c) * p.N + ti.n0 + f] =
                __float2bfloat16_rn(ffn::silu_times(g, u));
        }
      } else {
        for (int i = threadIdx.x; i < ti.rows * 128; i += kThreads) {
          const int c = i >> 7, f = i & 127;
          if (c % p.split != rank) continue;
          float v = 0.f;
          for (int r = 0; r < p.split; ++r) v += ptx::ld_cluster_f32(part + i * 4, r);
          const size_t at = (size_t)(ti.row0 + c) * p.N + ti.n0 + f;
          if (ti.n0 + f < p.N) {
            if (p.y_bf16) static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(v);
            else static_cast<float*>(p.y)[at] = v;
          }
        }
      }
    }
    ptx::cluster_sync();   // no CTA leaves while another reads its part
  }
  if (warp == 1) {
    if (PAIR) ptx::tmem_dealloc_pair(tmem, C::TMEM_COLS);
    else ptx::tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (threadIdx.x == 0 && p.status) {
    if (ss.abort) atomicOr(p.status, kStTimeout);
    if (ss.bad) atomicOr(p.status, kStBounds);
  }
}

template <int NT, bool GATED, bool PAIR>
cudaError_t launch_nt(const GemmParams8& p, long long tiles, cudaStream_t st) {
  constexpr int smem = smem_bytes8<NT, PAIR>();
  static std::atomic<uint64_t> smem_set{0};
  cudaError_t e = set_smem_once(gemm_fp8_kernel<NT, GATED, PAIR>, smem, smem_set);
  if (e != cudaSuccess) return e;
  const int team = PAIR ? 2 : p.split;
  const long long want = tiles * team, sms = num_sms() / team * team;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.split > 1 ? want : std::min(want, sms)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = team;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_fp8_kernel<NT, GATED, PAIR>, p);
}

template <int NT, bool PAIR>
cudaError_t launch_any(GemmParams8& p, bool gated, cudaStream_t st, const char** why,
                       const Gemm8Args& a) {
  const uint32_t box = gated ? 16 : 128;
  bool ok = make_tensor_map(&p.x, a.x, a.R, a.K, Cfg<NT, PAIR>::XBOX, kBK, 1, 128) &&
            make_tensor_map(&p.w1, a.W1, (uint64_t)a.G * a.N, a.K, box, kBK, 1, 128);
  p.w3 = p.w1;
  if (ok && gated) ok = make_tensor_map(&p.w3, a.W3, (uint64_t)a.G * a.N, a.K, box, kBK, 1, 128);
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed for a product operand";
    return cudaErrorInvalidValue;
  }
  p.nt = gated ? (a.N + 63) / 64 : (a.N + 127) / 128;
  if (PAIR) p.nt = (p.nt + 1) / 2;
  // row blocks: at most one per group with rows, and one per NT rows
  const long long blocks = std::min<long long>(a.R, (long long)a.R / NT + std::min(a.G, a.R));
  const long long tiles = blocks * p.nt;
  // Few tiles: split K over a cluster while that leaves every CTA an SM of its
  // own and at least two K-blocks.
  p.split = 1;
  if (!PAIR)
    while (p.split < 8 && tiles * p.split * 2 <= num_sms() && p.KB >= p.split * 4) p.split *= 2;
  return gated ? launch_nt<NT, true, PAIR>(p, tiles, st) : launch_nt<NT, false, PAIR>(p, tiles, st);
}

}  // namespace

cudaError_t launch_gemm_fp8(const Gemm8Args& a, cudaStream_t st, const char** why) {
  const bool gated = a.W3 != nullptr;
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
  // Rows per tile by the average group: small groups leave the weight stream
  // in charge, so the ring holds weights; large ones are bound by the products
  // and by what the SMs read from L2, which pairs of CTAs halve for the rows.
  const int avg = a.R / a.G;
  if (avg <= 16) return launch_any<32, false>(p, gated, st, why, a);
  if (avg <= 64) return launch_any<128, false>(p, gated, st, why, a);
  return launch_any<240, true>(p, gated, st, why, a);
}

}  // namespace moe
