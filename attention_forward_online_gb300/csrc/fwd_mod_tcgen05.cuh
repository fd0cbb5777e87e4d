// fwd_mod_tcgen05.cuh - attention forward with modified scores (a tanh cap,
// a distance slope or a learned bias by distance bucket), any interval mask
// (mask plan) and shared key/value heads, on the tcgen05 tensor cores.
// Built for sm_103a; bf16 or fp16, d = 64 or 128.
//
// The online softmax of the library's other forward kernels: per key tile the
// row max m, l = l alpha + rowsum(2^(x - m)), O rescaled by alpha = 2^(m_old - m),
// O / l once at the end and LSE = m + log l; x is the modified score in base-2
// units (mod_common.cuh).  A row that sees no key keeps (m, l) = (-inf, 0) and
// gets O = 0, LSE = -inf.
//
// CTA layout (512 threads, one CTA per SM): two 128-row query tiles of one
// (b, h), whose key tiles stream once for both through a TMA ring.  Warps 0-3
// and 4-7 softmax of tile 0 and 1, one query row a thread; 8-11 rescale O in
// tensor memory; 12 TMA producer; 13 issues the MMAs, S0, PV0, S1, PV1 in
// turn, so that one tile's product runs under the other tile's softmax.
// Tensor memory: S0 at 0, S1 at 128 (P in 16 bits over their first 64
// columns), O0 at 256, O1 at 256 + d.
//
// Each tile has its own range of key tiles from the plan, [a_t, b_t) within
// the pair's range; a tile outside its range takes no part in a step.
// Key tiles that reach past the keys either tile sees get those rows of V
// set to zero in shared memory by the correction warps before the product
// (0 * NaN is NaN: what lies behind a sequence's last key must not reach O).
//
// O leaves through the query tile's place in shared memory and TMA stores.
//
// P is rounded to 16 bits, the width of the MMA's operand, before P V; its sum and
// everything else stay in fp32.  O is then off by about 1.4 times the rounding of
// a right result (bf16, against 64 bits: 0.0023 to 0.0024 of its size, 0.0017).
//
// What bounds it: the softmax between a score tile's two products, by issue
// and latency (two tiles a CTA hide each other's products, not all of each
// other's softmax).  Per 128 x 128 tile the products take 512 cycles each at
// d = 128, the exponentials 512 of the multifunction unit; a cap adds 4 to 5
// packed operations a pair of scores where the polynomial serves, else an
// exponential and a quarter of a reciprocal a score; one-sided slopes add a
// 16-element MMA step and nothing per score; a learned bias one packed FMA's
// operand from shared memory within its range and a constant beyond.
//
// Measured (bf16, causal unless noted; GPU time of the mask plan and this kernel
// replayed as a graph, scores of standard deviation 2; "of measured" is the dense
// bf16 matrix rate of this GPU type, 1940 TFLOP/s):
//   B1 H32 kv8 8192 d128 cap 50       446 to 452 us, 1220 TFLOP/s, 63 % of measured
//   B4 H16 2048 d128 plain / cap / slopes / both   74 / 98 / 82 / 133 us
//   B4 H16 2048 d64  plain / cap / slopes / both   61 / 86 / 67 / 114 us
//   the last without a mask, plain                 95 us
//   B4 H16 1501 d64 fp16 learned bias  53 us;  B1 H16 4096 d128, no mask, 112 us
// A unit of 256 rows costs 3 us before its first score and 2 us after its last
// besides (about 5 steps of such a pair of tiles in all at d = 64).
#pragma once

#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>

#include "mod_common.cuh"
#include "mod_internal.h"
#include "sm100_ptx.cuh"
#include "softmax_tile.cuh"
#include "tc_attn_mma.cuh"

namespace osattn {
namespace fwdmod {

constexpr int BM = 128;
constexpr int BN = 128;
constexpr int kQTiles = 2;
constexpr int kThreads = 512;
constexpr int kCorrWarp0 = 8, kProducerWarp = 12, kMmaWarp = 13;
constexpr uint32_t kTmemCols = 512;
constexpr float kLn2 = 0.6931471805599453f;

enum : uint32_t {
  kSiteEmpty = 41,
  kSiteQ = 42,
  kSiteKV = 43,
  kSiteP = 44,
  kSiteS = 45,
  kSiteAlpha = 46,
  kSiteO = 48,
  kSiteZero = 49,
  kSiteStage = 50,
  kSiteTable = 51
};

template <int HD, int MODE>
struct Cfg {
  static constexpr int kTileBytes = BN * HD * 2;
  static constexpr int kQBytes = BM * HD * 2;
  // Table of learned biases: ranges up to kSmallRel leave all five stages at d =
  // 128; wider ones (kModRelWide) take one (32 KB; a step with four stages
  // waits for its loads, 20 % slower).  At d = 64 the twelfth stage of 16 KB
  // makes room for any range.
  // (kRangeBytes: the least and greatest that each filling warp wrote.)
  static constexpr int kRangeBytes = 12 * 8;
  static constexpr int kTableBytes =
      mode_rel(MODE) ? kRangeBytes + (rel_entries(HD == 64 || MODE == kModRelWide ? kMaxRelRange : kSmallRel) * 4 + 15) / 16 * 16
                     : (MODE == kModSlopes ? kSlopeRowsBytes + kSlopeQBytes : 0);
  static constexpr int kStages = HD == 128 ? (MODE == kModRelWide ? 4 : 5) : (mode_rel(MODE) ? 11 : 12);
  static constexpr int kIters = HD == 128 ? 4 : 8;  // > kStages / 2 + 1
  static constexpr int kTileRegion = kQTiles * kQBytes + kStages * kTileBytes;
  static constexpr uint32_t kOCol0 = 256;
};

struct __align__(16) Bars {
  uint64_t q_full[kQTiles];
  uint64_t kv_full[8];    // [i % kIters]: V_{i-1} and K_i landed
  uint64_t kv_empty[8];   // [i % kIters]: the MMAs of iteration i are done
  uint64_t s_full[kQTiles];
  uint64_t alpha_full[kQTiles];  // 128 arrivals
  uint64_t p_full[kQTiles];      // softmax and correction, 256 arrivals
  uint64_t o_full[kQTiles];
  uint64_t staged[kQTiles];      // O_t is in shared memory, 128 arrivals
  uint64_t table;                // the learned biases are in shared memory, 384 arrivals
  uint64_t mma_drain;
  uint32_t tmem_base;
  int abort_flag;
  uint16_t alpha[kQTiles][BM];  // alpha_bits
};

template <int HD, int MODE>
constexpr int smem_bytes() {
  return Cfg<HD, MODE>::kTileRegion + Cfg<HD, MODE>::kTableBytes + static_cast<int>(sizeof(Bars));
}

struct Params {
  float* LSE;
  PlanView plan;
  int H, group, Nq, Nkv, BH;  // group: query heads per key/value head
  int num_q_blocks, n_tiles;  // 256-row units and 128-row tiles per (b, h)
  int group_heads;
  float scale, scale_log2;  // |scale|, |scale| * log2(e) (positive_scale)
  uint32_t neg_q;           // kIdescNegA if the scale is negative
  CapArgs cap;
  const float* slopes;
  RelArgs rel;
  int q_offset;
  unsigned int* status;
  uint64_t wait_limit_ns;
};

// One query tile's part of a CTA's stream of key tiles.
struct Range {
  int a, n;  // first step and number of steps it takes part in
};

template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kF16) return pack_f16x2(lo, hi);
  else return pack_bf16x2(lo, hi);
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > limit_ns) return;
  }
}

// The head's learned biases, written by the softmax and correction warps while
// the first loads and products run.
template <int HD, bool kF16, int MODE>
__device__ __forceinline__ bool fill_table(const Params& p, Bars* bars, float* bias, int h, const WaitCtl& wc) {
  float lo, hi;
  float2* range = reinterpret_cast<float2*>(bias) - 12;
  rel_fill<kF16>(bias, p.rel, p.H, h, threadIdx.x, kProducerWarp * 32, lo, hi);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
  }
  if ((threadIdx.x & 31) == 0) range[threadIdx.x >> 5] = make_float2(lo, hi);
  mbar_arrive(&bars->table);
  return __all_sync(0xffffffffu, mbar_wait(&bars->table, 0u, wc, kSiteTable));
}

// ------------------------------------------------------------------ softmax
template <int HD, bool kF16, int MODE>
__device__ __forceinline__ void softmax_role(const CUtensorMap* tmO, const Params& p, Bars* bars,
                                             float* bias, uint8_t* sQt, uint32_t tmem, int t, int b, int h,
                                             float slope, int q0, Range rg, const PlanTile& tile, int kt0,
                                             WaitCtl wc) {
  using C = Cfg<HD, MODE>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const int qi = q0 + row;
  const int2 see = plan_row(p.plan, b, p.Nq, qi, p.Nkv);
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t s_addr = lane_base + static_cast<uint32_t>(t * BN);
  [[maybe_unused]] const int p0 = q0 + p.q_offset, pos = p0 + row;
  TileScore<kF16, MODE> ts;
  ts.c = p.scale_log2;
  ts.off = 0.f;
  ts.cap = &p.cap;
  [[maybe_unused]] bool linear = false;
  if constexpr (mode_slopes(MODE)) {
    ts.slope2 = slope * kModLog2e;
    linear = MODE == kModSlopes && slope_linear(slope, p.scale);
  }
  float m = -INFINITY, l = 0.f;
  bool ok = true;
  if constexpr (mode_rel(MODE)) {
    ok = fill_table<HD, kF16, MODE>(p, bars, bias, h, wc);
    if (!ok) return;
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll
    for (int w = 0; w < 12; ++w) {
      const float2 r = reinterpret_cast<const float2*>(bias)[w - 12];
      lo = fminf(lo, r.x);
      hi = fmaxf(hi, r.y);
    }
    ts.strip_lo = lo;
    ts.strip_close = hi - lo <= ts.kSpread;
    ts.far_lo = bias[0];
    ts.far_hi = bias[rel_entries(p.rel.range) - 1];
  }

  for (int j = 0; j < rg.n; ++j) {
    ok = mbar_wait(&bars->s_full[t], static_cast<uint32_t>(j) & 1u, wc, kSiteS);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    tc_fence_after_sync();
    const int k0 = (kt0 + rg.a + j) * BN;
    const bool masked = !(tile.lo_max <= k0 && tile.hi_min >= k0 + BN);
    const int lo = see.x - k0, hi = see.y - k0;
    auto bits_of = [&](int ch) { return bit_range(lo - 32 * ch, hi - 32 * ch); };
    if constexpr (mode_slopes(MODE)) {
      const int d0 = k0 - pos;  // distance of the tile's first key
      const int side = linear ? slope_side(k0, p0, tile.left) : 0;
      ts.both_sides = side == 0;
      ts.d0 = static_cast<float>(d0);
      ts.off = side == 0 ? 0.f : (side > 0 ? ts.slope2 : -ts.slope2) * ts.d0;
    }
    if constexpr (mode_rel(MODE)) {
      const int R = p.rel.range;
      const int first = k0 - p0;  // distances of the whole tile: first - 127 .. first + 127
      const bool far = first + BN - 1 <= -R || first - (BM - 1) >= R;
      ts.strip = far ? nullptr : bias + (k0 - pos + R + kRelPad);
      ts.off = far ? (first <= 0 ? ts.far_lo : ts.far_hi) : 0.f;
      // a chunk of this warp's 32 rows has distances x + first - 32 quarter - 31 .. + 31
      ts.near_lo = -R - 31 - first + 32 * quarter;
      ts.near_hi = R + 31 - first + 32 * quarter;
    }
    auto publish = [&](uint16_t alpha) {
      bars->alpha[t][row] = alpha;
      mbar_arrive(&bars->alpha_full[t]);
    };
    TileMask mk;
    if (masked) {
      mk.classify(bits_of);
      ts.template tile<true, true, false>(s_addr, mk, bits_of, ts.by_place(), m, l, publish);
    } else {
      ts.template tile<false, true, false>(s_addr, mk, bits_of, ts.by_place(), m, l, publish);
    }
    tmem_st_wait();
    tc_fence_before_sync();
    mbar_arrive(&bars->p_full[t]);
  }

  if (ok && rg.n > 0) {
    ok = mbar_wait(&bars->o_full[t], 0u, wc, kSiteO);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) tc_fence_after_sync();
  }
  if (!ok || q0 >= p.Nq) return;
  // a row that saw nothing gets zeros even if its tile's products hold NaN
  const bool empty = l == 0.f;
  const float inv_l = empty ? 0.f : 1.f / l;
  const uint64_t inv2 = f2_pack(inv_l, inv_l);
  const uint32_t o_addr = lane_base + C::kOCol0 + static_cast<uint32_t>(t * HD);
#pragma unroll
  for (int ch = 0; ch < HD / 32; ++ch) {
    uint32_t orr[32];
    if (rg.n > 0) {
      tmem_ld_32x32b_x32(o_addr + ch * 32, orr);
      tmem_ld_wait();
      reg_fence32(orr);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) orr[e] = 0u;
    }
    uint32_t packed[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float a0, a1;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(orr[2 * e]), __uint_as_float(orr[2 * e + 1])), inv2),
                a0, a1);
      packed[e] = empty ? 0u : pack2<kF16>(a0, a1);
    }
    stage_row32(sQt, row, ch * 32, packed);  // over Q_t, whose last reader is done
  }
  if (qi < p.Nq)
    p.LSE[(static_cast<long long>(b) * p.H + h) * p.Nq + qi] = empty ? -INFINITY : (m + log2f(l)) * kLn2;
  fence_proxy_async();
  mbar_arrive(&bars->staged[t]);
  if (quarter == 0) {
    ok = mbar_wait(&bars->staged[t], 0u, wc, kSiteStage);
    if (ok && lane == 0) {
#pragma unroll
      for (int cb = 0; cb < HD / 64; ++cb) tma_store_4d(tmO, sQt + cb * BM * 128, cb * 64, q0, h, b);
      tma_store_drain();
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------------ correction
template <int HD, int MODE>
__device__ __forceinline__ void correction_tile(Bars* bars, uint32_t lane_base, int row, int t,
                                                int j, bool& ok, WaitCtl wc) {
  using C = Cfg<HD, MODE>;
  // alpha_full(j) follows s_full(j), and with it PV_t(j - 1), issued before S_t(j).
  ok = mbar_wait(&bars->alpha_full[t], static_cast<uint32_t>(j) & 1u, wc, kSiteAlpha);
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) return;
  const float alpha = alpha_of(bars->alpha[t][row]);
  if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
    tc_fence_after_sync();
    const uint64_t a2 = f2_pack(alpha, alpha);
    const uint32_t o_addr = lane_base + C::kOCol0 + static_cast<uint32_t>(t * HD);
#pragma unroll
    for (int ch = 0; ch < HD / 32; ++ch) {
      uint32_t orr[32];
      tmem_ld_32x32b_x32(o_addr + ch * 32, orr);
      tmem_ld_wait();
      reg_fence32(orr);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float a0, a1;
        f2_unpack(f2_mul(f2_pack(__uint_as_float(orr[2 * e]), __uint_as_float(orr[2 * e + 1])), a2),
                  a0, a1);
        orr[2 * e] = __float_as_uint(a0);
        orr[2 * e + 1] = __float_as_uint(a1);
      }
      tmem_st_32x32b_x32(o_addr + ch * 32, orr);
    }
    tmem_st_wait();
  }
  tc_fence_before_sync();
  mbar_arrive(&bars->p_full[t]);
}

// lo, hi: the keys that a row of either tile sees lie in [lo, hi).
template <int HD, int MODE>
__device__ __forceinline__ void correction_role(Bars* bars, uint8_t* sKV, uint32_t tmem, Range r0,
                                                Range r1, int n, int kt0, int lo, int hi, int Nkv,
                                                WaitCtl wc) {
  using C = Cfg<HD, MODE>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  bool ok = true;
  for (int j = 0; ok && j < n; ++j) {
    const int k0 = (kt0 + j) * BN;
    if (k0 < lo || min(k0 + BN, Nkv) > hi) {
      // keys of this tile that nobody sees: zero their rows of V_j, which
      // iteration j + 1 reads after p_full(j).  (Keys past Nkv are zeros
      // already, filled in by the load.)
      ok = mbar_wait(&bars->kv_full[(j + 1) % C::kIters],
                     static_cast<uint32_t>((j + 1) / C::kIters) & 1u, wc, kSiteZero);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (k0 + row < lo || k0 + row >= hi) {
        uint8_t* v = sKV + ((2 * j + 1) % C::kStages) * C::kTileBytes + row * 128;
#pragma unroll
        for (int cb = 0; cb < HD / 64; ++cb)
#pragma unroll
          for (int x = 0; x < 8; ++x)
            *reinterpret_cast<uint4*>(v + cb * BN * 128 + x * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async();
    }
    const int j0 = j - r0.a, j1 = j - r1.a;
    if (j0 >= 0 && j0 < r0.n) correction_tile<HD, MODE>(bars, lane_base, row, 0, j0, ok, wc);
    if (ok && j1 >= 0 && j1 < r1.n) correction_tile<HD, MODE>(bars, lane_base, row, 1, j1, ok, wc);
  }
}

// ------------------------------------------------------------------ producer
template <int HD, int MODE>
__device__ __forceinline__ void producer_role(const CUtensorMap* tmQ, const CUtensorMap* tmK,
                                              const CUtensorMap* tmV, Bars* bars, uint8_t* sQ,
                                              uint8_t* sKV, int b, int h, int hk, int q0, Range r0,
                                              Range r1, int n, int kt0, WaitCtl wc) {
  using C = Cfg<HD, MODE>;
  if (r0.n > 0) {
    mbar_arrive_expect_tx(&bars->q_full[0], C::kQBytes);
#pragma unroll
    for (int cb = 0; cb < HD / 64; ++cb)
      tma_load_4d(sQ + cb * BM * 128, tmQ, &bars->q_full[0], cb * 64, q0, h, b);
  }
  if (r1.n > 0) {
    mbar_arrive_expect_tx(&bars->q_full[1], C::kQBytes);
#pragma unroll
    for (int cb = 0; cb < HD / 64; ++cb)
      tma_load_4d(sQ + C::kQBytes + cb * BM * 128, tmQ, &bars->q_full[1], cb * 64, q0 + BM, h, b);
  }
  // Load u goes to stage u % kStages: K_j for u = 2j, V_j for u = 2j + 1.
  // MMA iteration i reads loads 2i - 1 and 2i; both signal kv_full[i % kIters].
  const int total = 2 * n;
  int u = 0, armed = 0;
  for (; u < total; ++u) {
    const int s = u % C::kStages;
    if (u >= C::kStages) {
      const int r = (u - C::kStages + 1) >> 1;  // iteration that read load u - kStages
      if (!mbar_wait(&bars->kv_empty[r % C::kIters], static_cast<uint32_t>(r / C::kIters) & 1u, wc,
                     kSiteEmpty))
        break;
    }
    const int i = (u + 1) >> 1;  // iteration that reads load u
    uint64_t* full = &bars->kv_full[i % C::kIters];
    if (u == 0 || (u & 1)) {  // first load of iteration i
      mbar_arrive_expect_tx(full, ((i < n) ? C::kTileBytes : 0) + ((i >= 1) ? C::kTileBytes : 0));
      armed = i + 1;
    }
    uint8_t* dst = sKV + s * C::kTileBytes;
    const CUtensorMap* map = (u & 1) ? tmV : tmK;
#pragma unroll
    for (int cb = 0; cb < HD / 64; ++cb)
      tma_load_4d(dst + cb * BN * 128, map, full, cb * 64, (kt0 + (u >> 1)) * BN, hk, b);
  }
  // Let every load this thread issued land before the CTA can exit.
  if (r0.n > 0) drain_wait(&bars->q_full[0], 0, wc.limit_ns);
  if (r1.n > 0) drain_wait(&bars->q_full[1], 0, wc.limit_ns);
  for (int i = (armed > C::kIters ? armed - C::kIters : 0); i < armed; ++i)
    drain_wait(&bars->kv_full[i % C::kIters], static_cast<uint32_t>(i / C::kIters) & 1u,
               wc.limit_ns);
}

// ------------------------------------------------------------------ MMA issuer
// Warp-wide: one elected lane issues (mma_ss_k).
// slope_tiles: the slope operands (mode slopes, 0 if this head's slope is not
// used that way); p0: position of the first row, left0, left1: PlanTile::left;
// neg_q: kIdescNegA for a negative scale.
template <int HD, bool kF16, int MODE>
__device__ __forceinline__ void mma_role(Bars* bars, uint32_t tmem, uint8_t* sQ, uint8_t* sKV,
                                         Range r0, Range r1, int n, int kt0, uint32_t slope_tiles, int p0,
                                         bool left0, bool left1, uint32_t neg_q, WaitCtl wc) {
  using C = Cfg<HD, MODE>;
  const uint64_t q_desc0 = sdesc_sw128(smem_u32(sQ), 16, 1024);
  const uint64_t q_desc1 = q_desc0 + static_cast<uint64_t>(C::kQBytes >> 4);
  const uint64_t k_desc = sdesc_sw128(smem_u32(sKV), 16, 1024);        // stage 0, K-major
  const uint64_t v_desc = sdesc_sw128(smem_u32(sKV), BN * 128, 1024);  // stage 0, MN-major
  constexpr uint64_t kStageStep = static_cast<uint64_t>(C::kTileBytes >> 4);
  const uint32_t s_col0 = tmem, s_col1 = tmem + BN;
  const uint32_t o_col0 = tmem + C::kOCol0, o_col1 = tmem + C::kOCol0 + HD;
  const uint32_t s_id = idesc_f16_f32(128, 128, 0, kF16) | neg_q;
  // the slope's share of a score tile: one more step of 16 inner elements
  [[maybe_unused]] auto add_slope = [&](uint32_t s_col, int j, int pt, bool left) {
    if (slope_tiles == 0) return;
    const int side = slope_side((kt0 + j) * BN, pt, left);
    if (side == 0) return;
    mma_ss_k<1, true>(s_col, slope_q_desc(slope_tiles + kSlopeRowsBytes), slope_rows_desc(slope_tiles),
                      idesc_f16_f32(128, 128, 0, kF16) | (side < 0 ? kIdescNegA : 0u));
  };
  bool ok = true;

  for (int j = 0; ok && j <= n; ++j) {
    const uint32_t vs = j > 0 ? static_cast<uint32_t>((2 * j - 1) % C::kStages) : 0u;
    const uint32_t ks = static_cast<uint32_t>((2 * j) % C::kStages);
    ok = warp_wait(&bars->kv_full[j % C::kIters], static_cast<uint32_t>(j / C::kIters) & 1u, wc,
                   kSiteKV);
    if (ok && j == 0) {
      if (r0.n > 0) ok = warp_wait(&bars->q_full[0], 0, wc, kSiteQ);
      if (ok && r1.n > 0) ok = warp_wait(&bars->q_full[1], 0, wc, kSiteQ);
    }
    if (!ok) break;
    tc_fence_after_sync();
    // i0, i1: this step's place in each tile's own range
    const int i0 = j - r0.a, i1 = j - r1.a;
    if (i0 > 0 && i0 <= r0.n) {
      ok = warp_wait(&bars->p_full[0], static_cast<uint32_t>(i0 - 1) & 1u, wc, kSiteP);
      if (!ok) break;
      tc_fence_after_sync();
      mma_tmem_a_128<HD, kF16, true>(o_col0, s_col0, v_desc + vs * kStageStep, i0 > 1);
      if (i0 == r0.n) mma_commit<true>(&bars->o_full[0]);
    }
    if (i0 >= 0 && i0 < r0.n) {
      mma_abt_id<HD>(s_col0, q_desc0, k_desc + ks * kStageStep, s_id);
      if constexpr (MODE == kModSlopes) add_slope(s_col0, j, p0, left0);
      mma_commit<true>(&bars->s_full[0]);
    }
    if (i1 > 0 && i1 <= r1.n) {
      ok = warp_wait(&bars->p_full[1], static_cast<uint32_t>(i1 - 1) & 1u, wc, kSiteP);
      if (!ok) break;
      tc_fence_after_sync();
      mma_tmem_a_128<HD, kF16, true>(o_col1, s_col1, v_desc + vs * kStageStep, i1 > 1);
      if (i1 == r1.n) mma_commit<true>(&bars->o_full[1]);
    }
    if (i1 >= 0 && i1 < r1.n) {
      mma_abt_id<HD>(s_col1, q_desc1, k_desc + ks * kStageStep, s_id);
      if constexpr (MODE == kModSlopes) add_slope(s_col1, j, p0 + BM, left1);
      mma_commit<true>(&bars->s_full[1]);
    }
    mma_commit<true>(&bars->kv_empty[j % C::kIters]);
  }
  mma_commit<true>(&bars->mma_drain);
  drain_wait(&bars->mma_drain, 0, wc.limit_ns);
  __syncwarp();
}

template <int HD, bool kF16, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    fwd_mod_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmO,
                   const Params p) {
  using C = Cfg<HD, MODE>;
  // No static shared memory: the dynamic part starts on the alignment that
  // swizzled tiles need.  (Rounding up at run time would take another 1 KB.)
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicExch(p.status, 3u /* OSATTN_ERR_CUDA */);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + kQTiles * C::kQBytes;
  float* bias = reinterpret_cast<float*>(smem + C::kTileRegion + (mode_rel(MODE) ? C::kRangeBytes : 0));
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kTileRegion + C::kTableBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Work unit: 256 query rows of one (b, h).  Within groups of group_heads
  // heads, whose K and V fit in L2 together, the last rows first: under a
  // causal mask those are the longest units.
  const int nqb = p.num_q_blocks, unit = blockIdx.x;
  const int g0 = (unit / (p.group_heads * nqb)) * p.group_heads;
  const int gsize = min(p.group_heads, p.BH - g0);
  const int rank = unit - g0 * nqb;
  const int bh = g0 + rank % gsize;
  const int qb = nqb - 1 - rank / gsize;
  const int b = bh / p.H, h = bh % p.H;
  float slope = 0.f;
  if constexpr (mode_slopes(MODE)) slope = __ldg(p.slopes + h);
  const int q0 = qb * (kQTiles * BM);
  const int t0 = qb * kQTiles;
  // (on their way during the set-up)
  const int4 entry0 = plan_load(p.plan, b, p.n_tiles, t0, p.Nkv);
  const int4 entry1 = t0 + 1 < p.n_tiles ? plan_load(p.plan, b, p.n_tiles, t0 + 1, p.Nkv) : make_int4(0, 0, 0, 0);

  if (threadIdx.x == 0) {
    for (int t = 0; t < kQTiles; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->alpha_full[t], 128);
      mbar_init(&bars->p_full[t], 256);
      mbar_init(&bars->o_full[t], 1);
      mbar_init(&bars->staged[t], 128);
    }
    for (int i = 0; i < C::kIters; ++i) {
      mbar_init(&bars->kv_full[i], 1);
      mbar_init(&bars->kv_empty[i], 1);
    }
    mbar_init(&bars->table, kProducerWarp * 32);
    mbar_init(&bars->mma_drain, 1);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kProducerWarp && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  if constexpr (MODE == kModSlopes) {
    uint8_t* at = reinterpret_cast<uint8_t*>(bias);
    if (threadIdx.x < BN) slope_fill_k<kF16>(at, threadIdx.x);
    if (threadIdx.x < 8) slope_fill_q<kF16>(at + kSlopeRowsBytes, threadIdx.x, slope, p.scale);
    fence_proxy_async();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{&bars->abort_flag, p.status, p.status + 1, p.wait_limit_ns};
  const PlanTile pt0 = plan_entry(entry0), pt1 = plan_entry(entry1);
  const bool any0 = pt0.lo < pt0.hi, any1 = pt1.lo < pt1.hi;
  int lo = 0, hi = 0;  // keys that either tile sees
  if (any0) lo = pt0.lo, hi = pt0.hi;
  if (any1) {
    lo = any0 ? min(lo, pt1.lo) : pt1.lo;
    hi = max(hi, pt1.hi);
  }
  const int kt0 = lo / BN;
  const int n = (hi + BN - 1) / BN - kt0;  // 0 when no row sees a key (lo = hi = 0)
  Range r0{0, 0}, r1{0, 0};
  if (any0) r0 = Range{pt0.lo / BN - kt0, (pt0.hi + BN - 1) / BN - pt0.lo / BN};
  if (any1) r1 = Range{pt1.lo / BN - kt0, (pt1.hi + BN - 1) / BN - pt1.lo / BN};

  // 256 x 184 + 128 x 88 + 128 x 56 = 512 x 128 registers
  if (warp < kCorrWarp0) {
    regs_inc<184>();
    const int t = warp >> 2;
    softmax_role<HD, kF16, MODE>(&tmO, p, bars, bias, sQ + t * C::kQBytes, tmem, t, b, h, slope, q0 + t * BM,
                                 t ? r1 : r0, t ? pt1 : pt0, kt0, wc);
  } else if (warp < kProducerWarp) {
    regs_dec<88>();
    if constexpr (mode_rel(MODE)) fill_table<HD, kF16, MODE>(p, bars, bias, h, wc);
    correction_role<HD, MODE>(bars, sKV, tmem, r0, r1, n, kt0, lo, hi, p.Nkv, wc);
  } else {
    regs_dec<56>();
    if (warp == kProducerWarp && lane == 0 && n > 0)
      producer_role<HD, MODE>(&tmQ, &tmK, &tmV, bars, sQ, sKV, b, h, h / p.group, q0, r0, r1, n, kt0, wc);
    else if (warp == kMmaWarp && n > 0) {
      uint32_t slope_tiles = 0;
      if constexpr (MODE == kModSlopes)
        if (slope_linear(slope, p.scale)) slope_tiles = smem_u32(bias);
      mma_role<HD, kF16, MODE>(bars, tmem, sQ, sKV, r0, r1, n, kt0, slope_tiles, q0 + p.q_offset, pt0.left,
                               pt1.left, p.neg_q, wc);
    }
  }

  __syncwarp();
  tmem_st_wait();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// The setmaxnreg split hands out exactly 512 x 128 registers; a build with
// another launch count would wait forever in setmaxnreg.inc and is refused.
constexpr int kLaunchRegs = 128;

template <int HD, bool kF16, int MODE>
cudaError_t set_attrs() {
  static_assert(smem_bytes<HD, MODE>() <= 232448, "shared memory per CTA");
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, fwd_mod_kernel<HD, kF16, MODE>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(fwd_mod_kernel<HD, kF16, MODE>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<HD, MODE>());
}

template <int HD, bool kF16>
cudaError_t prepare() {
  cudaError_t e;
  if ((e = set_attrs<HD, kF16, kModPlain>()) != cudaSuccess) return e;
  if ((e = set_attrs<HD, kF16, kModCap>()) != cudaSuccess) return e;
  if ((e = set_attrs<HD, kF16, kModSlopes>()) != cudaSuccess) return e;
  if ((e = set_attrs<HD, kF16, kModCapSlopes>()) != cudaSuccess) return e;
  if constexpr (HD == 128)
    if ((e = set_attrs<HD, kF16, kModRelWide>()) != cudaSuccess) return e;
  return set_attrs<HD, kF16, kModRel>();
}

template <int HD, bool kF16, int MODE>
cudaError_t launch_mode(unsigned grid, cudaStream_t s, const CUtensorMap& q, const CUtensorMap& k,
                        const CUtensorMap& v, const CUtensorMap& o, const Params& p) {
  fwd_mod_kernel<HD, kF16, MODE><<<grid, kThreads, smem_bytes<HD, MODE>(), s>>>(q, k, v, o, p);
  return cudaGetLastError();
}

template <int HD, bool kF16>
cudaError_t launch(const ModArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   const CUtensorMap& o) {
  Params p;
  p.LSE = a.LSE;
  p.n_tiles = (a.Nq + BM - 1) / BM;
  p.plan.tiles = static_cast<const int4*>(a.plan);
  p.plan.rows = a.plan ? reinterpret_cast<const int2*>(p.plan.tiles + static_cast<long long>(a.B) * p.n_tiles)
                       : nullptr;
  p.H = a.H;
  p.group = a.H / a.Hkv;
  p.Nq = a.Nq;
  p.Nkv = a.Nkv;
  p.BH = a.B * a.H;
  p.num_q_blocks = (a.Nq + kQTiles * BM - 1) / (kQTiles * BM);
  {
    // query heads whose K and V together take about 32 MB of L2
    const long long kv_head = 2ll * a.Nkv * a.d * 2;
    const long long gh = (32ll << 20) / kv_head * p.group;
    p.group_heads = static_cast<int>(gh < 1 ? 1 : (gh > p.BH ? p.BH : gh));
  }
  p.scale = positive_scale(a.scale);
  p.scale_log2 = p.scale * kModLog2e;
  p.neg_q = a.scale < 0.f ? kIdescNegA : 0u;
  p.cap = make_cap(p.scale, a.softcap, kF16);
  p.slopes = a.slopes;
  p.rel = a.rel;
  p.q_offset = a.q_offset;
  p.status = a.status;
  p.wait_limit_ns = a.wait_limit_ns;
  const long long units = static_cast<long long>(p.num_q_blocks) * p.BH;
  if (units > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned g = static_cast<unsigned>(units);
  switch (mod_score_mode(a)) {
    case kModCap: return launch_mode<HD, kF16, kModCap>(g, a.stream, q, k, v, o, p);
    case kModSlopes: return launch_mode<HD, kF16, kModSlopes>(g, a.stream, q, k, v, o, p);
    case kModCapSlopes: return launch_mode<HD, kF16, kModCapSlopes>(g, a.stream, q, k, v, o, p);
    case kModRel:
      if constexpr (HD == 128)
        if (a.rel.range > kSmallRel) return launch_mode<HD, kF16, kModRelWide>(g, a.stream, q, k, v, o, p);
      return launch_mode<HD, kF16, kModRel>(g, a.stream, q, k, v, o, p);
    default: return launch_mode<HD, kF16, kModPlain>(g, a.stream, q, k, v, o, p);
  }
}

}  // namespace fwdmod
}  // namespace osattn
