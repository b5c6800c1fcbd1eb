// The whole layer for a few tokens (T <= 16) in two kernels.
//
// With few tokens the layer is its weight stream: each chosen expert's three
// matrices are read once and used for one or two tokens.  What can be lost is
// time in which the stream stands still, so the second kernel is persistent
// and one queue of tiles covers both expert products:
//
//   few_router_kernel   logits (fp32 FMAs), and in the block that finishes
//                       last the selection, the weights and the list of
//                       "slots": the shared experts, then the chosen experts
//                       in increasing order.  FP8: the hidden rows are also
//                       split into two E4M3 pieces here.
//   few_ffn_kernel      tiles claimed in order from a counter:
//     gate/up  (slot, up to 64 features): act = silu(W1 h) * (W3 h) for every
//              token, kept for the tokens that chose the expert
//     down     (slots, 128 output rows, part of K): y = W2 act of one slot, or
//              of a few in turn when the experts are narrow, weighted, a row
//              for each token that chose it; whoever completes the last unit of
//              128 output rows adds each token's rows, shared experts first, then
//              in the order of its choices
// Activations and results are held for (token, choice) pairs alone, ordered by
// slot and then by token; a slot's word of tokens says where its pairs start.
// The shared experts' gate/up tiles need no routing, so this kernel starts on
// them while the first one runs (programmatic dependent launch).
//
// The weights are the M = 128 operand of the tensor core, straight from
// memory by TMA, and the tokens the N operand: all T tokens against every
// chosen expert, since 16 columns cost no more than one.  A column depends on
// its own token alone, so what an expert computes for a token that did not
// choose it is dropped, whatever it is.
//
// Precision.  bf16 weights: hidden rows enter as they are; an activation
// enters as three bf16 pieces (its rounding, and twice what is left: all 24
// bits), in columns of their own that the epilogue adds in fp32.  FP8 weights:
// the codes enter as they are, with their block exponents as the tensor
// core's scales, and the other operand is a sum of E4M3 pieces, each holding 4
// bits of what the ones before it leave, with a scale 2^4 lower.  A bf16 value
// has 8 bits, so two pieces hold it, down to the second one's subnormal step:
// 2^-13 of the block's scale, which leaves at most 2^-21.8 of the block's
// largest value; four hold an activation to 2^-16 of itself.  The pieces cost
// columns, not weight bytes.
//
// The tensor core's bf16 form cuts off its running sum at each step of 16,
// which over K = 6144 adds up to 1.5e-5 of the result (measured).  K-blocks
// therefore take turns over as many accumulators as fit in tensor memory, 48
// K-blocks at a time, and the epilogue adds those in fp32.
#include <algorithm>
#include <climits>

#include <cuda_bf16.h>

#include "ffn_common.cuh"
#include "gate.cuh"
#include "route_order.cuh"
#include "sm100_scaled.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kRouterThreads = 512;
constexpr int kRouterWarps = kRouterThreads / 32;
constexpr int EPB = 2;                   // experts per router block
constexpr int kPiecesH = 2, kPiecesA = 4;   // E4M3 pieces of a hidden value, an activation
constexpr int kPiecesB = 3;                 // bf16 pieces of an activation
constexpr int kPieceMinExp = -115;       // the last piece's exponent stays an E8M0 value

// ---------------------------------------------------------------------------
// kernel 1: router, selection, slots
// ---------------------------------------------------------------------------
struct FewRoute {
  const uint16_t* h;
  const float *Wr, *bias;
  int T, D, E, k;
  float scale;
  float* scores;          // [T, E]
  uint32_t* order;        // [T, E] the keys' order
  int32_t* idx;           // [T, k]
  float* w;               // [T, k]
  int32_t* pair_of;       // [T, k] pair of each choice, -1 for none
  float* pair_w;          // [pairs] weight
  int32_t* slot_expert;   // [slots]
  uint32_t* slot_mask;    // [slots] bit t: token t chose it; its first pair from bit 16 on
  int32_t* nslots;        // chosen experts
  int32_t* counts;        // [E] pairs per expert
  int32_t* ticket;        // zero between calls
  int* status;
  int router_blocks;
  // FP8: pieces of the hidden rows [kPiecesH * T, D] and exponents [T, KB]
  uint8_t* hq;
  int8_t* hqe;
  int32_t* hq_ready;      // counts the blocks that wrote them
};

// Sums v[i] over the warp for all i: lane l ends with the sums of v[i] whose
// index is congruent to it, in v[0 .. N/32 - 1] (N >= 32), or the sum of
// v[l % N] in v[0] (N < 32).
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N], int lane) {
  int n = N;
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    if (n > 1) {
      // keep the half of the values whose index matches this lane's bit
      n >>= 1;
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        if (i < n) {
          const bool upper = lane & off;
          const float send = upper ? v[i] : v[i + n];
          const float keep = upper ? v[i + n] : v[i];
          v[i] = keep + __shfl_xor_sync(kAll, send, off);
        }
      }
    } else {
      v[0] += __shfl_xor_sync(kAll, v[0], off);
    }
  }
}

// fp32 score of a logit, as moe_route computes it.
__device__ __forceinline__ float score(float logit) {
  return __double2float_rn(1.0 / (1.0 + exp(-(double)logit)));
}

// The pieces of one block of 128 (or 32) values held by a warp: piece p's
// codes of each value, given the block's exponent.
__device__ __forceinline__ uint32_t piece_code(float& rest, float inv, float unit) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(rest * inv));
  const uint32_t code = r & 0xffu;
  // value of the code, exactly: E4M3 -> f16 -> f32
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(r));
  float val;
  asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(val) : "r"(h2));
  rest -= val * unit;
  return code;
}

__device__ __forceinline__ float pow2f(int e) {   // e in [-126, 127]
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Smallest e >= kPieceMinExp with top <= 448 * 2^e (0 for a block of zeros).
__device__ __forceinline__ int block_exp(float top) {
  const uint32_t u = __float_as_uint(top);
  if (u == 0) return 0;
  // 448 = 1.75 * 2^8: one exponent more when the fraction exceeds 0.75
  return max((int)((u + 0x1fffffu) >> 23) - 135, kPieceMinExp);
}

// Logits of EPB experts for every token, their scores and keys.
template <int TT>
__device__ __forceinline__ void router_block(const FewRoute& p, float* s_part) {
  const int e0 = blockIdx.x * EPB;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float acc[EPB * TT];
#pragma unroll
  for (int i = 0; i < EPB * TT; ++i) acc[i] = 0.f;
  for (int d = threadIdx.x * 4; d < p.D; d += kRouterThreads * 4) {
    float4 wv[EPB];
#pragma unroll
    for (int i = 0; i < EPB; ++i)
      wv[i] = e0 + i < p.E ? *reinterpret_cast<const float4*>(p.Wr + (size_t)(e0 + i) * p.D + d)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
    uint2 hv[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
      hv[t] = t < p.T ? *reinterpret_cast<const uint2*>(p.h + (size_t)t * p.D + d)
                      : make_uint2(0, 0);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float a = __uint_as_float(hv[t].x << 16), b = __uint_as_float(hv[t].x & 0xffff0000u);
      const float c = __uint_as_float(hv[t].y << 16), e = __uint_as_float(hv[t].y & 0xffff0000u);
#pragma unroll
      for (int i = 0; i < EPB; ++i) {
        float& s = acc[t * EPB + i];
        s = fmaf(a, wv[i].x, s);
        s = fmaf(b, wv[i].y, s);
        s = fmaf(c, wv[i].z, s);
        s = fmaf(e, wv[i].w, s);
      }
    }
  }
  constexpr int N = EPB * TT;
  warp_sums<N>(acc, lane);
  // index of the sum a lane holds: its bits choose halves from the top down
  constexpr int PER = N > 32 ? N / 32 : 1;
  int at = 0;
  {
    int n = N;
#pragma unroll
    for (int off = 16; off; off >>= 1)
      if (n > 1) {
        n >>= 1;
        if (lane & off) at += n;
      }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) s_part[warp * N + at + i] = acc[i];
  __syncthreads();
  bool bad = false;
  for (int i = threadIdx.x; i < N; i += kRouterThreads) {
    double v = 0.0;
    for (int q = 0; q < kRouterWarps; ++q) v += (double)s_part[q * N + i];
    const int t = i / EPB, e = e0 + i % EPB;
    if (t < p.T && e < p.E) {
      const float l = (float)v, sc = score(l), key = __fadd_rn(sc, p.bias[e]);
      bad = !isfinite(l) || !isfinite(key);
      p.scores[(size_t)t * p.E + e] = sc;
      p.order[(size_t)t * p.E + e] = key_order(key);
    }
  }
  if (bad && p.status) atomicOr(p.status, kStNonFinite);
}

// Shared memory of the selection: the experts' token masks and first pairs (E
// rounded up to 32 each), then the keys' order [T][E].
__host__ __device__ constexpr int select_words(int T, int E) { return 2 * ((E + 31) / 32 * 32) + T * E; }

// Selection for every token (a warp each), then the slots.  One block.
__device__ void select_and_list(const FewRoute& p, uint32_t* smem) {
  __shared__ int s_cnt[32], s_pairs[32];   // slots and pairs of 32 experts
  const int EP = (p.E + 31) / 32 * 32, groups = EP / 32;
  uint32_t* s_mask = smem;
  int* s_first = reinterpret_cast<int*>(smem + EP);
  uint32_t* s_ord = smem + 2 * EP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < EP; e += kRouterThreads) s_mask[e] = 0u;
  for (int i = threadIdx.x; i < p.T * p.E; i += kRouterThreads) s_ord[i] = __ldcg(p.order + i);
  __syncthreads();
  const int t = warp;
  int my_e = INT_MAX;
  float my_w = 0.f;
  if (t < p.T) {
    uint32_t* ord = s_ord + t * p.E;
    for (int j = 0; j < p.k; ++j) {
      uint32_t bu = 0u;
      int be = INT_MAX;
      for (int e = lane; e < p.E; e += 32)
        if (ord[e] > bu) {   // increasing e: ties keep the lower index
          bu = ord[e];
          be = e;
        }
      warp_best(bu, be);
      // no key is left when some were NaN: the slot stays empty
      if (bu && lane == (be & 31)) ord[be] = 0u;   // read again by this lane alone
      if (bu && lane == j) my_e = be;
    }
    // the scores of the chosen, a lane each, and their sum in slot order
    const float my_s = my_e != INT_MAX ? __ldcg(p.scores + (size_t)t * p.E + my_e) : 0.f;
    float sum = __shfl_sync(kAll, my_s, 0);
    for (int j = 1; j < p.k; ++j) sum = __fadd_rn(sum, __shfl_sync(kAll, my_s, j));
    if (lane < p.k) {
      p.idx[t * p.k + lane] = my_e;
      my_w = __fmul_rn(__fdiv_rn(my_s, sum), p.scale);
      p.w[t * p.k + lane] = my_w;
      if (my_e != INT_MAX) atomicOr(&s_mask[my_e], 1u << t);
    }
  }
  __syncthreads();
  for (int g = warp; g < groups; g += kRouterWarps) {
    const uint32_t m = s_mask[g * 32 + lane];
    const unsigned b = __ballot_sync(kAll, m != 0u);
    const int pairs = __reduce_add_sync(kAll, __popc(m));
    if (lane == 0) {
      s_cnt[g] = __popc(b);
      s_pairs[g] = pairs;
    }
  }
  __syncthreads();
  for (int g = warp; g < groups; g += kRouterWarps) {
    const int e = g * 32 + lane;
    const uint32_t m = s_mask[e];
    const unsigned b = __ballot_sync(kAll, m != 0u);
    int base = 0, first = 0;
    for (int q = 0; q < g; ++q) {
      base += s_cnt[q];
      first += s_pairs[q];
    }
    const int slot = base + __popc(b & ((1u << lane) - 1u));
    int upto = __popc(m);                // pairs of this group's experts up to this one
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, upto, o);
      if (lane >= o) upto += v;
    }
    first += upto - __popc(m);
    s_first[e] = first;
    if (m) {
      p.slot_expert[slot] = e;
      p.slot_mask[slot] = (uint32_t)first << 16 | m;
    }
    if (e < p.E) p.counts[e] = __popc(m);
    if (g == groups - 1 && lane == 31) *p.nslots = slot + (m != 0u);
  }
  __syncthreads();
  if (t < p.T && lane < p.k) {
    int pair = -1;
    if (my_e != INT_MAX) {
      pair = s_first[my_e] + __popc(s_mask[my_e] & ((1u << t) - 1u));
      p.pair_w[pair] = my_w;
    }
    p.pair_of[t * p.k + lane] = pair;
  }
}

// One warp: the pieces of 128 columns of a hidden row.
__device__ __forceinline__ void split_hidden(const FewRoute& p, int unit, int lane) {
  const int KB = (p.D + 127) / 128;
  const int t = unit / KB, kb = unit - t * KB;
  const int col = kb * 128 + lane * 4;
  uint2 raw = make_uint2(0, 0);
  if (col < p.D) raw = *reinterpret_cast<const uint2*>(p.h + (size_t)t * p.D + col);
  float v[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u),
                __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u)};
  float top = 0.f;
  bool odd[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    odd[i] = !isfinite(v[i]);
    if (odd[i]) v[i] = 0.f;
    top = fmaxf(top, fabsf(v[i]));
  }
  top = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(top)));
  const int e = block_exp(top);
  if (lane == 0) p.hqe[t * KB + kb] = (int8_t)e;
#pragma unroll
  for (int q = 0; q < kPiecesH; ++q) {
    const float inv = pow2f(4 * q - e), unit2 = pow2f(e - 4 * q);
    uint32_t c = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t code = piece_code(v[i], inv, unit2);
      c |= (odd[i] ? 0x7fu : code) << (8 * i);
    }
    if (col < p.D) *reinterpret_cast<uint32_t*>(p.hq + (size_t)(q * p.T + t) * p.D + col) = c;
  }
}

template <int TT>
__global__ void __launch_bounds__(kRouterThreads) few_router_kernel(const FewRoute p) {
  extern __shared__ uint32_t s_dyn[];
  ptx::pdl_wait();
  // From here on everything before this call is complete and visible, which
  // the next kernel relies on before its own wait: it must not be let go
  // earlier.
  ptx::pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((int)blockIdx.x >= p.router_blocks) {
    const int unit = ((int)blockIdx.x - p.router_blocks) * kRouterWarps + warp;
    if (unit < p.T * ((p.D + 127) / 128)) split_hidden(p, unit, lane);
    // the pieces become visible to the whole GPU and to TMA, then the count
    ptx::fence_proxy_async_global();
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) atomicAdd(p.hq_ready, 1);
    return;
  }
  router_block<TT>(p, reinterpret_cast<float*>(s_dyn));
  // the block that finishes last selects
  __shared__ int s_last;
  __syncthreads();
  if (threadIdx.x == 0) s_last = ptx::atom_add_acq_rel_gpu(p.ticket, 1) == p.router_blocks - 1;
  __syncthreads();
  if (!s_last) return;
  select_and_list(p, s_dyn);
  if (threadIdx.x == 0) *p.ticket = 0;   // for the next call
}

// ---------------------------------------------------------------------------
// kernel 2: both expert products and the merge
// ---------------------------------------------------------------------------
constexpr int kAStage = 128 * 128;       // 128 weight rows x 128 bytes of K
constexpr int kBStage = 8192;
constexpr int kAStages = 9, kBStages = 8;
static_assert(kBStages <= kAStages, "the weights' stages release the tokens'");
constexpr int kRing = kAStages * kAStage + kBStages * kBStage;
constexpr int kSfSlot = 32;              // scale columns of one slot: 4 weights, 4 x 4 tokens
constexpr uint32_t kTmemCols = 512;
// TMEM columns of one of the two accumulator sets; the scale slots follow.  The
// epilogue reads 16 columns from a piece's first one, at most 10 beyond the
// set, which are still columns of this CTA.
__host__ __device__ constexpr int acc_cols(bool fp8) { return fp8 ? 192 : 240; }
// Accumulators that a unit of kb K-blocks takes turns over, for a token operand
// of n rows: chains of four K-blocks (16 steps) as far as the set reaches; each
// one costs the epilogue a read.
__device__ __forceinline__ int acc_count(bool fp8, int n, int kb) {
  return min((kb + 3) / 4, acc_cols(fp8) / n);
}
// K-blocks that go into one set before the epilogue takes it (a multiple of the
// K-blocks of a stage and of a scale word).
constexpr int kSegment = 48;
constexpr int kQueue = 4;

struct alignas(64) FewFfn {
  CUtensorMap x;                         // hidden rows (bf16) or their pieces, box NX x 128 B
  CUtensorMap act_r, act_s;              // activations [pairs * pieces, F], box 16 x 128 B
  CUtensorMap w1_r, w3_r, w1_s, w3_s;    // [E * F, D], box 16 rows
  CUtensorMap w2_r, w2_s;                // [E * D, F], box 128 rows
  const int8_t *e1_r, *e3_r, *e2_r, *e1_s, *e3_s, *e2_s;
  int T, D, E, F, k, S, Fs;
  int NX, PA;            // token operand rows: gate/up, down
  // features per gate/up tile (64, 32 or 16) and K-blocks per stage of one,
  // of a chosen and of a shared expert
  int fpt_r, fpt_s, sub_r, sub_s;
  int parts;             // K parts of a down unit
  int nd;                // blocks of 128 output rows
  int ntr, nts;          // gate/up tiles per chosen / shared slot
  int max_slots;         // S + the most experts the call can choose
  int spu_r, spu_s;      // slots of a down unit: chosen, shared
  int ngs;               // shared groups of slots (units per output block and part)
  // routing (written by the first kernel)
  const int32_t *pair_of, *slot_expert, *nslots;
  const uint32_t* slot_mask;
  const float* pair_w;
  const int8_t* hqe;     // FP8: exponents of the hidden rows [T, KB]
  // activations: a slot's pairs by piece, [pieces][its pairs] rows from row pieces *
  // (its first pair) on; their exponents (FP8: one per 32 features, [pairs, 4 * KB])
  uint8_t *a_r, *a_s;
  int8_t *ae_r, *ae_s;
  float* rows;           // [part][S * T + pairs][D]: the shared experts' results, then the pairs'
  float* out;
  int32_t* claim;        // claim counter, exit ticket, blocks of pieces written, then
                         // per-slot counts, then per-output-block tickets; zero
                         // between calls
  int hq_blocks;         // FP8: blocks that write the pieces of the hidden rows
  int32_t* touched;
  int* status;
};

struct Unit {
  int down;              // 0 gate/up, 1 down, -1 end
  int slot;              // shared slots first
  int at;                // first feature, or output block
  int part;
  int expert;            // row of the weight arrays
  uint32_t mask;         // its tokens and first pair, as slot_mask; shared: slot * T
  int last;              // down units of several slots come one slot at a time
};
__device__ __forceinline__ uint32_t unit_tokens(const Unit& u) { return u.mask & 0xffffu; }
__device__ __forceinline__ int unit_first(const Unit& u) { return (int)(u.mask >> 16); }

struct FewShared {
  uint64_t full[kAStages], empty[kAStages];   // a stage's weights and tokens; its products done
  uint64_t sf_full[2], sf_empty[2];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t q_full[kQueue], q_empty[kQueue];
  uint64_t drain;
  uint64_t epi;          // barrier of the four epilogue warps
  Unit q[kQueue];
  uint32_t tmem_base;
  int abort, bad, last, exit_last;
  int act_done[4];       // gate/up tiles whose part each epilogue warp has stored
  float act[2][64 * 17]; // FP8: activations of a tile [feature][token], by turns
  int tab[kFewMaxT * 32];        // the tokens' choices: their row of a part, -1 for none
};

constexpr int few_smem() { return 1024 + kRing + (int)sizeof(FewShared); }

// The tile queue seen by one consuming warp.
struct QueueReader {
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ bool next(FewShared& ss, Unit& u, volatile int* abort, int lane) {
    if (__any_sync(kAll, !ptx::mbar_wait(&ss.q_full[slot], phase, abort))) return false;
    const volatile Unit& q = ss.q[slot];
    u.down = q.down; u.slot = q.slot; u.at = q.at; u.part = q.part; u.expert = q.expert; u.mask = q.mask; u.last = q.last;
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive_after_reads(&ss.q_empty[slot]);
    if (++slot == kQueue) { slot = 0; phase ^= 1u; }
    return u.down >= 0;
  }
};

// K-blocks [k0, k1) of a unit, of EB elements each.
template <int EB>
__device__ __forceinline__ void unit_k(const FewFfn& p, const Unit& u, int* k0, int* k1) {
  if (u.down) {
    const int kb = ((u.slot < p.S ? p.Fs : p.F) + EB - 1) / EB;
    *k0 = kb * u.part / p.parts;
    *k1 = kb * (u.part + 1) / p.parts;
  } else {
    *k0 = 0;
    *k1 = (p.D + EB - 1) / EB;
  }
}

__device__ __forceinline__ int32_t* slot_count(const FewFfn& p, int slot) { return p.claim + 3 + slot; }
__device__ __forceinline__ int32_t* out_ticket(const FewFfn& p, int d) {
  return p.claim + 3 + p.max_slots + d;
}
// Arrivals after which a slot's activations are complete: four epilogue warps a tile.
__device__ __forceinline__ int slot_target(const FewFfn& p, int slot) {
  return 4 * (slot < p.S ? p.nts : p.ntr);
}

// Waits, whole warp, until a slot's activations are stored; every lane acquires.
__device__ __forceinline__ bool slot_wait(const FewFfn& p, int slot, volatile int* abort) {
  // (most are ready; the others are looked at closely for a moment first)
  for (int i = 0; i < 64; ++i) {
    if (__all_sync(kAll, ptx::ld_acquire_gpu(slot_count(p, slot)) >= slot_target(p, slot)))
      return true;
    __nanosleep(20);
  }
  return !__any_sync(kAll, !ptx::counter_wait(slot_count(p, slot), slot_target(p, slot), abort));
}

// Waits, whole warp, until the hidden rows' pieces are written.  The blocks of
// the first kernel that write them are all running before this kernel starts.
__device__ __forceinline__ bool pieces_wait(const FewFfn& p, volatile int* abort) {
  return !__any_sync(kAll, !ptx::counter_wait(p.claim + 2, p.hq_blocks, abort));
}

// Up to four exponents q[0 .. n-1] (n >= 1): the aligned words that hold them
// (`inside`: these lie within the array; else the bytes), so that the loads can
// be under way long before the bytes are put together.
struct RawScales {
  uint32_t a, b;
  int shift;
  __device__ __forceinline__ void load(const int8_t* q, int n, bool inside) {
    if (inside) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(q);
      const uint32_t* base = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
      shift = 8 * (int)(at & 3);
      a = __ldcg(base);
      b = 4 - (int)(at & 3) < n ? __ldcg(base + 1) : 0u;
    } else {
      shift = 0;
      a = ptx::bytes_word(q, n);
      b = 0;
    }
  }
  // Four E8M0 bytes (exponents from n on count as 0); outside the weights' range
  // of [-117, 7] raises *bad.
  __device__ __forceinline__ uint32_t word(int n, bool check, bool* bad) const {
    uint32_t w = __funnelshift_r(a, b, shift);
    if (n < 4) w &= (1u << (8 * n)) - 1u;
    if (check) *bad |= (__vcmpgts4(w, 0x07070707u) | __vcmplts4(w, 0x8b8b8b8bu)) != 0;
    return __vadd4(w, 0x7f7f7f7fu);
  }
};

// out for 128 columns, from the rows: shared experts, then the token's choices in
// their order.  Four groups of 32 threads take every fourth
// token, a thread four columns; kMergeLoads loads are in flight before the
// first is added.
constexpr int kMergeLoads = 8;
__device__ __forceinline__ void merge_block(const FewFfn& p, const FewShared& ss, int at, int tid) {
  const int d = at * 128 + (tid & 31) * 4;
  if (d >= p.D) return;
  const size_t part_rows = (size_t)(p.S + p.k) * p.T;
  // this thread's terms: its tokens one after the other, each token's experts,
  // each expert's K parts
  const int n = (p.S + p.k) * p.parts;
  const int total = (p.T - (tid >> 5) + 3) / 4 * n;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  int lt = tid >> 5, lj = 0, lpart = 0;  // the term being loaded
  int t = lt, done = 0;                  // the token being added, its terms so far
  for (int i0 = 0; i0 < total; i0 += kMergeLoads) {
    float4 r[kMergeLoads];
#pragma unroll
    for (int i = 0; i < kMergeLoads; ++i) {
      r[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + i < total) {
        const int row = lj < p.S ? lj * p.T + lt : ss.tab[lt * p.k + lj - p.S];
        if (row >= 0)
          r[i] = __ldcg(reinterpret_cast<const float4*>(
              p.rows + (lpart * part_rows + row) * p.D + d));
        if (++lpart == p.parts) {
          lpart = 0;
          if (++lj == p.S + p.k) { lj = 0; lt += 4; }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kMergeLoads; ++i) {
      if (i0 + i < total) {
        o.x += r[i].x; o.y += r[i].y; o.z += r[i].z; o.w += r[i].w;
        if (++done == n) {
          *reinterpret_cast<float4*>(p.out + (size_t)t * p.D + d) = o;
          o = make_float4(0.f, 0.f, 0.f, 0.f);
          done = 0;
          t += 4;
        }
      }
    }
  }
}

template <bool FP8>
__global__ void __launch_bounds__(FP8 ? 384 : 256, 1) few_ffn_kernel(const __grid_constant__ FewFfn p) {
  constexpr int EB = FP8 ? 128 : 64;     // K elements of 128 bytes
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_addr(smem_raw);
  // the token ring follows the weight ring, so a product that reads 128 rows
  // of a smaller tile stays inside the rings
  uint8_t* ring_a = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* ring_b = ring_a + kAStages * kAStage;
  FewShared& ss = *reinterpret_cast<FewShared*>(ring_a + kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 2) {
    ptx::tmem_alloc(&ss.tmem_base, kTmemCols);
    ptx::tmem_relinquish();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kAStages; ++i) {
      ptx::mbar_init(&ss.full[i], 2);
      ptx::mbar_init(&ss.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ss.sf_full[i], 4);
      ptx::mbar_init(&ss.sf_empty[i], 1);
      ptx::mbar_init(&ss.acc_full[i], 1);
      ptx::mbar_init(&ss.acc_empty[i], 4);
    }
    for (int i = 0; i < kQueue; ++i) {
      ptx::mbar_init(&ss.q_full[i], 1);
      ptx::mbar_init(&ss.q_empty[i], 1 + 1 + 1 + 4 + (FP8 ? 4 : 0));
    }
    ptx::mbar_init(&ss.drain, 1);
    ptx::mbar_init(&ss.epi, 4);
    ss.abort = 0;
    ss.bad = 0;
    for (int i = 0; i < 4; ++i) ss.act_done[i] = 0;
    ptx::fence_barrier_init();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = ss.tmem_base;
  volatile int* abort = &ss.abort;
  const int shared_tiles = p.S * p.nts;

  if (warp == 0) {
    // ---------------- weight producer and tile claimer ----------------
    if (ptx::elect_one()) {
      const uint64_t policy = ptx::l2_policy_evict_first();
      int stage = 0, qs = 0, routed = -1;
      uint32_t phase = 0, qphase = 0, issued = 0, parity = 0;
      int tile = atomicAdd(p.claim, 1);
      for (;;) {
        const uint32_t all = (1u << p.T) - 1u;
        Unit u{0, 0, 0, 0, 0, all, 1};
        int slots = 1;                   // of a down unit
        if (tile < shared_tiles) {
          u.slot = tile / p.nts;
          u.at = (tile - u.slot * p.nts) * p.fpt_s;
          u.expert = u.slot;
          u.mask = (uint32_t)(u.slot * p.T) << 16 | all;
        } else {
          const bool fresh = routed < 0;
          if (fresh) ptx::pdl_wait();    // the list of chosen experts
          int r = tile - shared_tiles;
          // a gate/up tile's expert is read along with the list's length, which
          // says whether there is such a tile
          int s = min(r / p.ntr, p.max_slots - p.S - 1);
          int expert = __ldcg(p.slot_expert + s);
          uint32_t mask = __ldcg(p.slot_mask + s);
          if (fresh) routed = __ldcg(p.nslots);
          if (r < routed * p.ntr) {
            u.slot = p.S + s;
            u.at = (r - s * p.ntr) * p.fpt_r;
          } else {
            r -= routed * p.ntr;
            const int per = p.nd * p.parts, g = r / per;
            const int groups = p.ngs + (routed + p.spu_r - 1) / p.spu_r;
            r -= g * per;
            u.down = g < groups ? 1 : -1;
            u.part = r / p.nd;
            u.at = r - u.part * p.nd;
            if (g < p.ngs) {
              u.slot = g * p.spu_s;
              slots = min(p.spu_s, p.S - u.slot);
            } else {
              const int first = (g - p.ngs) * p.spu_r;
              u.slot = p.S + first;
              slots = min(p.spu_r, routed - first);
              if (u.down >= 0) {
                expert = __ldcg(p.slot_expert + first);
                mask = __ldcg(p.slot_mask + first);
              }
            }
            u.last = slots <= 1;
          }
          if (u.slot >= p.S) {
            u.expert = expert;
            u.mask = mask;
          } else {
            u.expert = u.slot;
            u.mask = (uint32_t)(u.slot * p.T) << 16 | all;
          }
        }
        if (!ptx::mbar_wait(&ss.q_empty[qs], qphase ^ 1u, abort)) break;
        ss.q[qs] = u;
        ptx::mbar_arrive(&ss.q_full[qs]);
        if (++qs == kQueue) { qs = 0; qphase ^= 1u; }
        if (u.down < 0) break;
        const int next = atomicAdd(p.claim, 1);   // its latency hides under this tile
        const bool sh = u.slot < p.S;
        int k0, k1;
        unit_k<EB>(p, u, &k0, &k1);
        bool ok = true;
        if (u.down) {
          const CUtensorMap* m = sh ? &p.w2_s : &p.w2_r;
          for (;;) {
            // the unit's next slot, if it has one
            Unit v = u;
            if (--slots > 0) {
              ++v.slot;
              v.last = slots <= 1;
              if (sh) {
                v.expert = v.slot;
                v.mask = (uint32_t)(v.slot * p.T) << 16 | all;
              } else {
                v.expert = __ldcg(p.slot_expert + v.slot - p.S);
                v.mask = __ldcg(p.slot_mask + v.slot - p.S);
              }
            }
            const int row = u.expert * p.D + u.at * 128;
            for (int kb = k0; kb < k1; ++kb) {
              if (!ptx::mbar_wait(&ss.empty[stage], phase ^ 1u, abort)) { ok = false; break; }
              ptx::mbar_arrive_expect_tx(&ss.full[stage], kAStage);
              ptx::tma_load_2d_hint(ring_a + stage * kAStage, m, &ss.full[stage], kb * EB, row, policy);
              issued |= 1u << stage;
              parity = (parity & ~(1u << stage)) | (phase << stage);
              if (++stage == kAStages) { stage = 0; phase ^= 1u; }
            }
            if (!ok || slots <= 0) break;
            u = v;
            if (!ptx::mbar_wait(&ss.q_empty[qs], qphase ^ 1u, abort)) { ok = false; break; }
            ss.q[qs] = u;
            ptx::mbar_arrive(&ss.q_full[qs]);
            if (++qs == kQueue) { qs = 0; qphase ^= 1u; }
          }
        } else {
          const CUtensorMap* m1 = sh ? &p.w1_s : &p.w1_r;
          const CUtensorMap* m3 = sh ? &p.w3_s : &p.w3_r;
          const int row = u.expert * (sh ? p.Fs : p.F) + u.at;
          const int boxes = (sh ? p.fpt_s : p.fpt_r) / 16, sub = sh ? p.sub_s : p.sub_r;
          for (int kb = k0; kb < k1; kb += sub) {
            if (!ptx::mbar_wait(&ss.empty[stage], phase ^ 1u, abort)) { ok = false; break; }
            const int n = min(sub, k1 - kb);
            ptx::mbar_arrive_expect_tx(&ss.full[stage], n * boxes * 4096);
            uint8_t* dst = ring_a + stage * kAStage;
            for (int i = 0; i < n; ++i)
              for (int j = 0; j < boxes; ++j, dst += 4096) {
                ptx::tma_load_2d_hint(dst, m1, &ss.full[stage], (kb + i) * EB, row + j * 16, policy);
                ptx::tma_load_2d_hint(dst + 2048, m3, &ss.full[stage], (kb + i) * EB, row + j * 16, policy);
              }
            issued |= 1u << stage;
            parity = (parity & ~(1u << stage)) | (phase << stage);
            if (++stage == kAStages) { stage = 0; phase ^= 1u; }
          }
        }
        if (!ok) break;
        tile = next;
      }
      for (int s = 0; s < kAStages; ++s)
        if (issued & (1u << s)) ffn::wait_drain(&ss.full[s], (parity >> s) & 1u, abort);
    }
  } else if (warp == 1) {
    // ---------------- token / activation producer ----------------
    QueueReader q;
    Unit u;
    // It walks the weights' stages.  Its own stage is free when the products of
    // the stage kBStages back are done, which that weight stage tells; since
    // kBStages <= kAStages that barrier cannot have moved on by another phase.
    bool waited = false, pieces = false;
    int stage = 0, own = 0, wait_at = 0, lag = kBStages;
    uint32_t phase = 0, wait_phase = 0, issued = 0, parity = 0;
    while (q.next(ss, u, abort, lane)) {
      const bool sh = u.slot < p.S;
      if (!waited && (u.down || !sh)) {
        ptx::pdl_wait();
        waited = true;
      }
      if (FP8 && !pieces) {
        if (!pieces_wait(p, abort)) break;
        ptx::fence_proxy_async_global();
        pieces = true;
      }
      if (u.down) {
        if (!slot_wait(p, u.slot, abort)) break;
        ptx::fence_proxy_async_global();
      }
      int k0, k1;
      unit_k<EB>(p, u, &k0, &k1);
      const CUtensorMap* m = u.down ? (sh ? &p.act_s : &p.act_r) : &p.x;
      // down: as many boxes of 16 rows as the slot's pieces fill (what else they
      // hold, and the stage behind them, are columns that nobody reads)
      constexpr int pieces_a = FP8 ? kPiecesA : kPiecesB;
      const int row = u.down ? unit_first(u) * pieces_a : 0;
      const int boxes = u.down ? (__popc(unit_tokens(u)) * pieces_a + 15) / 16 : 1;
      const int bytes = u.down ? boxes * 2048 : p.NX * 128;
      const int sub = u.down ? 1 : sh ? p.sub_s : p.sub_r;
      bool ok = true;
      if (ptx::elect_one()) {
        for (int kb = k0; kb < k1; kb += sub) {
          if (lag > 0) {
            --lag;
          } else {
            if (!ptx::mbar_wait(&ss.empty[wait_at], wait_phase, abort)) { ok = false; break; }
            if (++wait_at == kAStages) { wait_at = 0; wait_phase ^= 1u; }
          }
          const int n = min(sub, k1 - kb);
          ptx::mbar_arrive_expect_tx(&ss.full[stage], n * bytes);
          uint8_t* dst = ring_b + own * kBStage;
          if (u.down) {
            for (int i = 0; i < boxes; ++i)
              ptx::tma_load_2d(dst + i * 2048, m, &ss.full[stage], kb * EB, row + i * 16);
          } else {
            for (int i = 0; i < n; ++i)
              ptx::tma_load_2d(dst + i * bytes, m, &ss.full[stage], (kb + i) * EB, 0);
          }
          if (++own == kBStages) own = 0;
          issued |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kAStages) { stage = 0; phase ^= 1u; }
        }
      }
      if (__any_sync(kAll, !ok)) break;
    }
    if (issued)
      for (int s = 0; s < kAStages; ++s)
        if (issued & (1u << s)) ffn::wait_drain(&ss.full[s], (parity >> s) & 1u, abort);
  } else if (warp == 2) {
    // ---------------- MMA issuer ----------------
    QueueReader q;
    Unit u;
    int as = 0, bs = 0, buf = 0, slot = 0;
    uint32_t aph = 0, cph = 0, sph = 0;
    const uint32_t desc_a = ptx::desc_sw128_lo(ptx::smem_addr(ring_a));
    const uint32_t desc_b = ptx::desc_sw128_lo(ptx::smem_addr(ring_b));
    while (q.next(ss, u, abort, lane)) {
      int k0, k1;
      unit_k<EB>(p, u, &k0, &k1);
      const bool sh = u.slot < p.S;
      const int sub = u.down ? 1 : sh ? p.sub_s : p.sub_r;
      const int n = u.down ? p.PA : p.NX;
      const uint32_t idesc = FP8 ? ptx::idesc_mxf8(128, n) : ptx::idesc_bf16_f32(128, n);
      // sizes of a K-block within its stage, in the descriptors' units of 16 bytes
      const int a_step = (u.down ? kAStage : (sh ? p.fpt_s : p.fpt_r) * 2 * 128) >> 4;
      const int b_step = n * 128 >> 4;
      // down: the four steps of a K-block name the token word's bytes in turn
      const uint32_t id_step = u.down ? ptx::idesc_sf_byte(0, 1) : 0u;
      bool ok = true;
      for (int seg = k0; seg < k1 && ok; seg += kSegment) {
        const int seg_end = min(seg + kSegment, k1);
        if (ptx::elect_one()) {
          ok = ptx::mbar_wait(&ss.acc_empty[buf], cph ^ 1u, abort);
          const int nacc = acc_count(FP8, n, seg_end - seg);
          uint32_t acc = tmem + buf * acc_cols(FP8);
          const uint32_t acc_end = acc + nacc * n;
          uint32_t more = 0;             // 0 in the first turn over the accumulators
          int kk = seg;
          while (ok && kk < seg_end) {
            if (!ptx::mbar_wait(&ss.full[as], aph, abort)) { ok = false; break; }
            uint32_t da = desc_a + as * (kAStage >> 4), db = desc_b + bs * (kBStage >> 4);
            const int end = min(kk + sub, seg_end);
            for (; kk < end; ++kk, da += a_step, db += b_step) {
              if (FP8 && (kk == k0 || (kk & 3) == 0) &&
                  !ptx::mbar_wait(&ss.sf_full[slot], sph, abort)) { ok = false; break; }
              ptx::tc_fence_after();
              if (FP8) {
                const uint32_t sfa = tmem + 2 * acc_cols(FP8) + slot * kSfSlot;
                // gate/up: one word per row covers four K-blocks; down: one word
                // per row and K-block covers its four steps of 32
                const uint32_t sfb = sfa + 4 + (u.down ? (kk & 3) * 4 : 0);
                const uint32_t id = idesc | ptx::idesc_sf_byte(kk & 3, u.down ? 0 : kk & 3);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  ptx::mma_mxf8_ss(acc, ptx::desc_sw128(da + 2 * k), ptx::desc_sw128(db + 2 * k),
                                   id + k * id_step, sfa, sfb, k > 0 ? 1u : more);
                if ((kk & 3) == 3 || kk == k1 - 1) {
                  ptx::mma_commit(&ss.sf_empty[slot]);
                  if (++slot == 2) { slot = 0; sph ^= 1u; }
                }
              } else {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  ptx::mma_f16_ss(acc, ptx::desc_sw128(da + 2 * k), ptx::desc_sw128(db + 2 * k), idesc,
                                  k > 0 ? 1u : more);
              }
              acc += n;
              if (acc == acc_end) {
                acc -= nacc * n;
                more = 1;
              }
            }
            if (!ok) break;
            ptx::mma_commit(&ss.empty[as]);
            if (++as == kAStages) { as = 0; aph ^= 1u; }
            if (++bs == kBStages) bs = 0;
          }
          if (ok) ptx::mma_commit(&ss.acc_full[buf]);
        }
        if (++buf == 2) { buf = 0; cph ^= 1u; }
        ok = !__any_sync(kAll, !ok);
      }
      if (!ok) break;
    }
    // nothing of this CTA is in flight when its tensor memory is freed
    if (ptx::elect_one()) {
      ptx::mma_commit(&ss.drain);
      ffn::wait_drain(&ss.drain, 0, abort);
    }
  } else if (warp == 3) {
    // ---------------- hand-over of activations ----------------
    // Counts a slot's finished tiles for the whole GPU, so that the epilogue
    // does not wait for its stores to get there.  The epilogue warps may be up to
    // two tiles apart (the two accumulator sets), and those without rows in a
    // narrow tile run ahead, so a tile is finished when each of the four has
    // counted it, not when four counts have come in.
    QueueReader q;
    Unit u;
    int tiles = 0;
    const volatile int* done = ss.act_done;
    while (q.next(ss, u, abort, lane)) {
      if (u.down) continue;
      ++tiles;
      const long long t0 = clock64();
      bool ok = true;
      while (min(min(done[0], done[1]), min(done[2], done[3])) < tiles) {
        __nanosleep(20);
        if (*abort) { ok = false; break; }
        if (clock64() - t0 > ptx::kWaitBudgetCycles) {
          *abort = 1;
          ok = false;
          break;
        }
      }
      if (__any_sync(kAll, !ok)) break;
      if (lane == 0) {
        // what the four warps stored before they were counted is ordered before
        // this, for TMA too
        __threadfence();
        ptx::fence_proxy_async_global();
        atomicAdd(slot_count(p, u.slot), 4);
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------- epilogue ----------------
    const int qt = warp & 3;
    const uint32_t lanes = (uint32_t)(qt * 32) << 16;
    QueueReader q;
    Unit u;
    ptx::WarpBarrier epi{&ss.epi};
    bool waited = false;
    int buf = 0, turn = 0, tiles = 0;
    uint32_t cph = 0;
    // The ticket of a down unit is looked at with the next one, so that its round
    // trip passes under that one's products: lane 0 of the first warp holds
    // its number, and `last_at` is the output block it stands for (-1: none).
    int ticket = 0, last_at = -1, units = 0;
    // All four warps; after this unit's rows are stored, or at the end: merges the
    // block of the unit before if that was its last unit, then takes this unit's
    // ticket.  The barrier orders the four warps' stores before lane 0's ticket,
    // whose release makes them visible to the whole GPU.
    auto settle = [&](int at) {
      if (qt == 0 && lane == 0) {
        ss.last = last_at >= 0 && ticket == units - 1;
        if (ss.last) *out_ticket(p, last_at) = 0;
      }
      if (!epi.sync(abort, lane)) return false;
      const bool merge = *reinterpret_cast<volatile int*>(&ss.last);
      if (at >= 0 && qt == 0 && lane == 0) ticket = ptx::atom_add_acq_rel_gpu(out_ticket(p, at), 1);
      if (merge) {
        __threadfence();
        merge_block(p, ss, last_at, threadIdx.x - 128);
      }
      last_at = at;
      // the flag is read before it is written again
      return epi.sync(abort, lane);
    };
    while (q.next(ss, u, abort, lane)) {
      const bool sh = u.slot < p.S;
      if (!waited && (u.down || !sh)) {
        ptx::pdl_wait();
        waited = true;
        units = (p.ngs + (__ldcg(p.nslots) + p.spu_r - 1) / p.spu_r) * p.parts;
        // (read after a barrier of all four warps, in settle)
        for (int i = threadIdx.x - 128; i < p.T * p.k; i += 128) {
          const int pair = __ldcg(p.pair_of + i);
          ss.tab[i] = pair >= 0 ? p.S * p.T + pair : -1;
        }
      }
      const uint32_t mask = unit_tokens(u);
      const int first = unit_first(u), cnt = __popc(mask);
      // a down unit's weights: lane i has its pair's
      float wl = 1.f;
      if (u.down && !sh && lane < cnt) wl = __ldcg(p.pair_w + first + lane);
      int k0, k1;
      unit_k<EB>(p, u, &k0, &k1);
      // the columns, pieces and accumulators added: v[i] is this lane's weight row
      // and token i (gate/up), or the slot's pair i (down)
      const int pieces = u.down ? (FP8 ? kPiecesA : kPiecesB) : (FP8 ? kPiecesH : 1);
      const int per = u.down ? cnt : p.T;
      const int n = u.down ? p.PA : p.NX;
      const int fpt = sh ? p.fpt_s : p.fpt_r;
      const bool rows = u.down || qt * 16 < fpt;     // this warp's rows belong to the tile
      float v[16];
#pragma unroll
      for (int t = 0; t < 16; ++t) v[t] = 0.f;
      bool ok = true;
      for (int seg = k0; seg < k1; seg += kSegment) {
        if (__any_sync(kAll, !ptx::mbar_wait(&ss.acc_full[buf], cph, abort))) { ok = false; break; }
        ptx::tc_fence_after();
        const uint32_t acc = tmem + buf * acc_cols(FP8) + lanes;
        const int nacc = acc_count(FP8, n, min(kSegment, k1 - seg));
        // smallest piece first, a piece's accumulators one after the other, four
        // reads in flight
        const int reads = rows ? pieces * nacc : 0;
        int c = pieces - 1, a = 0;
        for (int i0 = 0; i0 < reads; i0 += 4) {
          uint32_t r[4][16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i0 + i < reads) ptx::tmem_ld_x16(acc + a * n + c * per, r[i]);
            if (++a == nacc) { a = 0; --c; }
          }
          ptx::tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i0 + i < reads) {
#pragma unroll
              for (int t = 0; t < 16; ++t) v[t] += __uint_as_float(r[i][t]);
            }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ss.acc_empty[buf]);
        if (++buf == 2) { buf = 0; cph ^= 1u; }
      }
      if (!ok) break;

      if (!u.down) {
        const int F = sh ? p.Fs : p.F;
        const bool up = lane >= 16;
        const int f = u.at + qt * 16 + (lane & 15);
        const size_t row0 = (size_t)first * (FP8 ? kPiecesA : kPiecesB);
        // lanes 0-15 finish the even tokens, lanes 16-31 the odd ones
        float act[8];
        auto gates = [&](auto&& silu) {
#pragma unroll
          for (int t = 0; t < 16; t += 2) {
            const float got = __shfl_xor_sync(kAll, up ? v[t] : v[t + 1], 16);
            act[t / 2] = silu(t + (up ? 1 : 0), up ? got : v[t], up ? v[t + 1] : got);
          }
        };
        float least = 0.f;               // of the gates that count
        gates([&](int tt, float g, float u) {
          if ((mask >> tt) & 1u) least = fminf(least, g);
          return silu_times_near<true>(g, u);
        });
        if (__any_sync(kAll, least < kGateFar))
          gates([](int, float g, float u) { return silu_times_wide<true>(g, u); });
#pragma unroll
        for (int t = 0; t < 16; t += 2) {
          const float a = f < F ? act[t / 2] : 0.f;
          const int tt = t + (up ? 1 : 0);
          if (FP8) {
            ss.act[turn][(qt * 16 + (lane & 15)) * 17 + tt] = a;
          } else if (rows && f < F && ((mask >> tt) & 1u)) {
            __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(sh ? p.a_s : p.a_r) +
                                 (row0 + __popc(mask & ((1u << tt) - 1u))) * F + f;
            float rest = a;
#pragma unroll
            for (int c = 0; c < kPiecesB; ++c) {
              const __nv_bfloat16 piece = __float2bfloat16_rn(rest);
              dst[(size_t)c * cnt * F] = piece;
              // an infinite piece is all there is
              rest = __hisinf(piece) ? 0.f : rest - __bfloat162float(piece);
            }
          }
        }
        if (FP8) {
          // 32 features of a token per warp and round: exponent, then the pieces
          if (!epi.sync(abort, lane)) break;
          int8_t* ae = sh ? p.ae_s : p.ae_r;
          const int stride = (F + 127) / 128 * 4;   // exponents of a row
          for (int i = qt; i < p.T * (fpt / 32); i += 4) {
            const int t = i % p.T, b = i / p.T;
            if (!((mask >> t) & 1u)) continue;
            const int at = __popc(mask & ((1u << t) - 1u));   // among the slot's pairs
            float a = ss.act[turn][(b * 32 + lane) * 17 + t];
            const bool odd = !isfinite(a);
            if (odd) a = 0.f;
            const float top = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(fabsf(a))));
            const int e = block_exp(top);
            const int fb = u.at + b * 32;
            if (fb >= F) continue;
            if (lane == 0)
              ae[(size_t)(first + at) * stride + fb / 32] = (int8_t)e;
            uint8_t* dst = (sh ? p.a_s : p.a_r) + (row0 + at) * F + fb + lane;
#pragma unroll
            for (int c = 0; c < kPiecesA; ++c) {
              const uint32_t code = piece_code(a, pow2f(4 * c - e), pow2f(e - 4 * c));
              if (fb + lane < F) dst[(size_t)c * cnt * F] = (uint8_t)(odd ? 0x7fu : code);
            }
          }
          // the next tile writes the other half; a warp that comes back to this
          // one has met all four at that tile's barrier
          turn ^= 1;
        }
        // this warp's part is stored, as far as this CTA can see
        ++tiles;
        __syncwarp();
        if (lane == 0) {
          __threadfence_block();
          *const_cast<volatile int*>(&ss.act_done[qt]) = tiles;
        }
      } else {
        const int d = u.at * 128 + qt * 32 + lane;
        const size_t row0 = (size_t)u.part * (p.S + p.k) * p.T + (sh ? 0 : p.S * p.T) + first;
        float* dst = p.rows + row0 * p.D + d;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          if (i >= cnt) break;           // (mostly one or two)
          const float c = __shfl_sync(kAll, wl, i);
          if (d < p.D) dst[(size_t)i * p.D] = c * v[i];
        }
        if (!u.last) continue;
        if (!settle(u.at)) break;
      }
    }
    if (last_at >= 0 && !*abort) settle(-1);
  } else if (FP8 && warp >= 8) {
    // ---------------- scale writers ----------------
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int KBD = (p.D + 127) / 128;
    QueueReader q;
    Unit u;
    bool pieces = false, bad = false;
    int slot = 0;
    uint32_t sph = 0;
    while (q.next(ss, u, abort, lane)) {
      if (!pieces) {
        if (!pieces_wait(p, abort)) break;
        pieces = true;
      }
      const bool sh = u.slot < p.S;
      const int F = sh ? p.Fs : p.F, KBF = (F + 127) / 128;
      if (u.down && !slot_wait(p, u.slot, abort)) break;
      int k0, k1;
      unit_k<EB>(p, u, &k0, &k1);
      // the weights' exponents: the array, and this unit's row of blocks in it
      const int8_t* we0 = u.down          ? (sh ? p.e2_s : p.e2_r)
                          : (lane & 16) ? (sh ? p.e3_s : p.e3_r)
                                        : (sh ? p.e1_s : p.e1_r);
      const int8_t* we_end = we0 + (size_t)(sh ? p.S : p.E) * KBF * KBD;
      const int KB = u.down ? KBF : KBD;
      const int8_t* we = we0 + (u.down ? (size_t)u.expert * KBD + u.at
                                       : (size_t)u.expert * KBF + u.at / 128) * KB;
      const bool inside = ptx::words_inside(we, KB, we0, we_end);
      const int8_t* ae = (sh ? p.ae_s : p.ae_r) + (size_t)unit_first(u) * (KBF * 4);
      // the piece and token (gate/up) or pair (down) of this lane's two rows of the
      // token operand
      // (row + 1/2) / per is at least 1/32 away from every whole number
      const int per = u.down ? __popc(unit_tokens(u)) : p.T;
      const float inv = __fdividef(1.0f, (float)per);
      const int row_c[2] = {(int)((lane + 0.5f) * inv), (int)((lane + 32.5f) * inv)};
      const int row_t[2] = {lane - row_c[0] * per, 32 + lane - row_c[1] * per};
      // Token words: gate/up, one per row (the bytes are K-blocks); down, one per
      // row and K-block (the bytes are its steps of 32, and a row's exponents
      // start on four bytes).  A set's words are loaded while the one before it
      // is written.
      const int8_t* xq[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        xq[j] = row_c[j] >= (u.down ? kPiecesA : kPiecesH) ? nullptr
                : u.down ? ae + (size_t)row_t[j] * (KBF * 4)
                         : p.hqe + (size_t)row_t[j] * KBD;
      const int fe = (F + 31) / 32;      // exponents of an activation row
      RawScales ra, rx[2];
      uint32_t rd[4][2];
      auto load = [&](int s) {
        ra.load(we + 4 * s, KB - 4 * s, inside);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (!xq[j]) continue;
          if (!u.down) {
            // (in the workspace, with room behind them)
            rx[j].load(xq[j] + 4 * s, KBD - 4 * s, true);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (4 * s + i < KBF)
                rd[i][j] = __ldcg(reinterpret_cast<const uint32_t*>(xq[j]) + 4 * s + i);
          }
        }
      };
      bool ok = true;
      load(k0 / 4);
      for (int s = k0 / 4; s * 4 < k1; ++s) {
        uint32_t wa[4], wx[4][2];
        wa[0] = wa[1] = wa[2] = wa[3] = ra.word(KB - 4 * s, true, &bad);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t lower = 0x04040404u * row_c[j];   // a piece's scale is 2^-4 of the one before
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            wx[i][j] = 0x7f7f7f7fu;      // rows of no token: any valid scale
            if (!xq[j]) continue;
            if (!u.down) {
              if (i == 0) wx[i][j] = __vsub4(rx[j].word(KBD - 4 * s, false, &bad), lower);
            } else if (4 * s + i < KBF) {
              // exponents past the last feature count as 0 (their codes are zero)
              const int n = fe - 4 * (4 * s + i);
              uint32_t w = rd[i][j];
              if (n < 4) w &= (1u << (8 * n)) - 1u;
              wx[i][j] = __vsub4(__vadd4(w, 0x7f7f7f7fu), lower);
            }
          }
        }
        if ((s + 1) * 4 < k1) load(s + 1);
        if (__any_sync(kAll, !ptx::mbar_wait(&ss.sf_empty[slot], sph ^ 1u, abort))) { ok = false; break; }
        ptx::tc_fence_after();
        const uint32_t dst = tmem + 2 * acc_cols(FP8) + slot * kSfSlot + lanes;
        ptx::tmem_st_x4(dst, wa);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i == 0 || u.down) ptx::tmem_st_x2(dst + 4 + 4 * i, wx[i][0], wx[i][1]);
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ss.sf_full[slot]);
        if (++slot == 2) { slot = 0; sph ^= 1u; }
      }
      if (!ok) break;
    }
    if (bad) ss.bad = 1;
  }

  __syncthreads();
  if (warp == 2) ptx::tmem_dealloc(tmem, kTmemCols);
  ptx::pdl_launch_dependents();
  if (threadIdx.x == 0) {
    if (p.status) {
      if (ss.abort) atomicOr(p.status, kStTimeout);
      if (ss.bad) atomicOr(p.status, kStBounds);
    }
    // the last CTA leaves the claim counter and the slot counts zero
    __threadfence();
    ss.exit_last = atomicAdd(p.claim + 1, 1) == (int)gridDim.x - 1;
  }
  __syncthreads();
  if (ss.exit_last) {
    __threadfence();
    // no expert at all (no token has a key that is a number): nothing was merged
    ptx::pdl_wait();
    if (p.S == 0 && __ldcg(p.nslots) == 0)
      for (int i = threadIdx.x; i < p.T * p.D; i += blockDim.x) p.out[i] = 0.f;
    for (int i = threadIdx.x; i < p.max_slots; i += blockDim.x) *slot_count(p, i) = 0;
    if (threadIdx.x == 0) {
      *p.touched = __ldcg(p.nslots);
      p.claim[0] = p.claim[1] = p.claim[2] = 0;
    }
  }
}

template <int TT>
cudaError_t launch_few_router(FewRoute& r, int hq_blocks, cudaStream_t st) {
  r.router_blocks = (r.E + EPB - 1) / EPB;
  const int part = kRouterWarps * EPB * TT * 4;
  const int keys = select_words(r.T, r.E) * 4;
  static std::atomic<uint64_t> smem_set{0};
  const cudaError_t e = set_smem_once(few_router_kernel<TT>,
                                      std::max(part, select_words(kFewMaxT, 1024) * 4), smem_set);
  if (e != cudaSuccess) return e;
  return launch_pdl(few_router_kernel<TT>, dim3(r.router_blocks + hq_blocks), dim3(kRouterThreads),
                    (size_t)std::max(part, keys), st, r);
}

}  // namespace

// How a call is cut into tiles.
FewPlan few_plan(const moe_dims_t& d, bool fp8) {
  FewPlan L{};
  auto round16 = [](int n) { return (n + 15) / 16 * 16; };
  L.pieces_h = fp8 ? kPiecesH : 1;
  L.pieces_a = fp8 ? kPiecesA : kPiecesB;
  L.NX = round16(L.pieces_h * d.T);
  L.PA = round16(L.pieces_a * d.T);
  const int most = std::min(d.E, d.T * d.k);     // chosen experts at most
  L.max_slots = d.S + most;
  const int Fs = d.S > 0 ? d.Fs : 0;
  // Features per gate/up tile: 64 fill the 128 weight rows of a product.  When
  // that gives tiles to fewer than three quarters of the SMs, 32 (and with bf16
  // weights 16) spread the weight stream over more of them; the rows they leave
  // unused cost tensor time, which is why tiles are not cut any further.  (One
  // chosen expert of 2048 x 6144: 36 us with 16 features a tile, 55 with 64; 14
  // tokens, 55 experts of 192 x 104, up to 126 tiles of 64: 21 us as they are,
  // 25 in narrower ones.)  The shared experts' tiles run while the routing is
  // still being made and are to keep every SM busy by themselves, unless they
  // are small (one token, 1.6 MB tiles: 114 us cut into quarters, 116 whole).
  const int least = fp8 ? 32 : 16;
  auto tiles = [](int experts, int F, int fpt) { return (long long)experts * ((F + fpt - 1) / fpt); };
  L.fpt_s = L.fpt_r = 64;
  const int few = kSplitTargetBlocks * 3 / 4;
  auto bytes = [&](int fpt) { return (long long)fpt * 2 * d.D * (fp8 ? 1 : 2); };
  while (L.fpt_s > least && tiles(d.S, Fs, L.fpt_s) < few && bytes(L.fpt_s) > 400 << 10) L.fpt_s /= 2;
  while (L.fpt_r > least && tiles(d.S, Fs, L.fpt_s) + tiles(most, d.F, L.fpt_r) < few) L.fpt_r /= 2;
  // K-blocks per stage: the stage stays 16 KB of weights, within the token stage
  auto sub = [&](int fpt) {
    int n = 64 / fpt;
    while (n > 1 && n * L.NX * 128 > kBStage) n /= 2;
    return n;
  };
  L.sub_r = sub(L.fpt_r);
  L.sub_s = sub(L.fpt_s);
  L.nd = (d.D + 127) / 128;
  const int eb = fp8 ? 128 : 64;
  const int kb = std::min((d.F + eb - 1) / eb, d.S > 0 ? (Fs + eb - 1) / eb : 1 << 30);
  // K parts of a down unit, each with rows to write and to add: only while
  // all of them have an SM and at least eight K-blocks.  (One chosen expert, 48
  // output blocks: 36 us in two parts, 39 in one, 43 in four; one token through
  // nine experts, 432 units: 114 us in one, two or four parts.)
  L.parts = 1;
  while (L.parts < 8 && (long long)L.nd * L.parts * L.max_slots * 2 <= kSplitTargetBlocks &&
         kb >= 16 * L.parts)
    L.parts *= 2;
  // Slots of a down unit: narrow experts are taken together until a unit has 16
  // K-blocks, as long as there are two units per SM (a unit's ticket costs
  // its epilogue 1 us).
  auto together = [&](int slots, int kbs) {
    int n = 1;
    while (L.parts == 1 && n * kbs < 16 &&
           (long long)L.nd * ((slots + 2 * n - 1) / (2 * n)) >= 2 * kSplitTargetBlocks)
      n *= 2;
    return n;
  };
  L.spu_r = together(most, (d.F + eb - 1) / eb);
  L.spu_s = together(d.S, (Fs + eb - 1) / eb);
  return L;
}

cudaError_t launch_few(const FewArgs& a, cudaStream_t st, const char** why) {
  const moe_dims_t& d = a.d;
  const bool fp8 = a.w8 != nullptr;
  const FewPlan L = few_plan(d, fp8);
  const int Fs = d.S > 0 ? d.Fs : 0;

  FewRoute r{};
  r.h = a.h; r.Wr = a.Wr; r.bias = a.bias;
  r.T = d.T; r.D = d.D; r.E = d.E; r.k = d.k; r.scale = d.scale;
  r.scores = a.scores;
  r.order = a.order;
  r.idx = a.idx; r.w = a.w;
  r.pair_of = a.pair_of; r.pair_w = a.pair_w; r.slot_expert = a.slot_expert; r.slot_mask = a.slot_mask;
  r.nslots = a.nslots; r.counts = a.counts;
  r.ticket = a.ticket;
  r.status = a.status;
  r.hq = a.hq; r.hqe = a.hqe;
  const int units = fp8 ? d.T * ((d.D + 127) / 128) : 0;
  const int hq_blocks = (units + kRouterWarps - 1) / kRouterWarps;
  r.hq_ready = a.claim + 2;

  FewFfn f{};
  const int es = fp8 ? 1 : 2, eb = 128 / es;
  const void *W1 = fp8 ? (const void*)a.w8->W1 : a.W1, *W3 = fp8 ? (const void*)a.w8->W3 : a.W3;
  const void *W2 = fp8 ? (const void*)a.w8->W2 : a.W2;
  const void *S1 = fp8 ? (const void*)a.w8->Ws1 : a.Ws1, *S3 = fp8 ? (const void*)a.w8->Ws3 : a.Ws3;
  const void *S2 = fp8 ? (const void*)a.w8->Ws2 : a.Ws2;
  auto map = [&](CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box) {
    return make_tensor_map(m, base, rows, cols, box, eb, es, 128);
  };
  const uint64_t pairs = (uint64_t)d.T * d.k;
  bool ok = (fp8 ? map(&f.x, a.hq, L.pieces_h * d.T, d.D, L.NX) : map(&f.x, a.h, d.T, d.D, L.NX)) &&
            map(&f.act_r, a.a_r, pairs * L.pieces_a, d.F, 16) &&
            map(&f.w1_r, W1, (uint64_t)d.E * d.F, d.D, 16) &&
            map(&f.w3_r, W3, (uint64_t)d.E * d.F, d.D, 16) &&
            map(&f.w2_r, W2, (uint64_t)d.E * d.D, d.F, 128);
  f.act_s = f.act_r; f.w1_s = f.w1_r; f.w3_s = f.w3_r; f.w2_s = f.w2_r;
  if (ok && d.S > 0)
    ok = map(&f.act_s, a.a_s, (uint64_t)d.S * d.T * L.pieces_a, Fs, 16) &&
         map(&f.w1_s, S1, (uint64_t)d.S * Fs, d.D, 16) &&
         map(&f.w3_s, S3, (uint64_t)d.S * Fs, d.D, 16) &&
         map(&f.w2_s, S2, (uint64_t)d.S * d.D, Fs, 128);
  if (!ok) {
    *why = "cuTensorMapEncodeTiled failed for an expert operand";
    return cudaErrorInvalidValue;
  }
  if (fp8) {
    f.e1_r = a.w8->W1e; f.e3_r = a.w8->W3e; f.e2_r = a.w8->W2e;
    f.e1_s = a.w8->Ws1e; f.e3_s = a.w8->Ws3e; f.e2_s = a.w8->Ws2e;
  }
  f.T = d.T; f.D = d.D; f.E = d.E; f.F = d.F; f.k = d.k; f.S = d.S; f.Fs = Fs;
  f.NX = L.NX; f.PA = L.PA;
  f.fpt_r = L.fpt_r; f.fpt_s = L.fpt_s; f.sub_r = L.sub_r; f.sub_s = L.sub_s;
  f.parts = L.parts; f.nd = L.nd;
  f.ntr = (d.F + L.fpt_r - 1) / L.fpt_r;
  f.nts = (Fs + L.fpt_s - 1) / L.fpt_s;
  f.max_slots = L.max_slots;
  f.spu_r = L.spu_r; f.spu_s = L.spu_s;
  f.ngs = (d.S + L.spu_s - 1) / L.spu_s;
  f.pair_of = a.pair_of; f.slot_expert = a.slot_expert; f.nslots = a.nslots;
  f.slot_mask = a.slot_mask;
  f.pair_w = a.pair_w;
  f.hqe = a.hqe;
  f.a_r = a.a_r; f.a_s = a.a_s; f.ae_r = a.ae_r; f.ae_s = a.ae_s;
  f.rows = a.rows;
  f.out = a.out;
  f.claim = a.claim;
  f.hq_blocks = hq_blocks;
  f.touched = a.touched;
  f.status = a.status;

  *why = "router launch";
  cudaError_t e = d.T <= 1   ? launch_few_router<1>(r, hq_blocks, st)
                  : d.T <= 2 ? launch_few_router<2>(r, hq_blocks, st)
                  : d.T <= 4 ? launch_few_router<4>(r, hq_blocks, st)
                  : d.T <= 8 ? launch_few_router<8>(r, hq_blocks, st)
                             : launch_few_router<16>(r, hq_blocks, st);
  if (e != cudaSuccess) return e;
  *why = "expert launch";
  static std::atomic<uint64_t> set16{0}, set8{0};
  e = fp8 ? set_smem_once(few_ffn_kernel<true>, few_smem(), set8)
          : set_smem_once(few_ffn_kernel<false>, few_smem(), set16);
  if (e != cudaSuccess) return e;
  const long long gu = (long long)d.S * f.nts + (long long)(L.max_slots - d.S) * f.ntr;
  const long long dn = (long long)L.max_slots * L.nd * L.parts;
  const int grid = (int)std::min<long long>(num_sms(), gu + dn);
  return fp8 ? launch_pdl(few_ffn_kernel<true>, dim3(grid), dim3(384), few_smem(), st, f)
             : launch_pdl(few_ffn_kernel<false>, dim3(grid), dim3(256), few_smem(), st, f);
}

}  // namespace moe
