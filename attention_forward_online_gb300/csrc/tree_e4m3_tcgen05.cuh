// tree_e4m3_tcgen05.cuh - attention of drafted tokens over a paged cache of e4m3
// values with a scale for each block of tokens and head, on the tcgen05 tensor
// cores.  Built for sm_103a; queries in bf16 or fp16, d = 64 or 128.
//
// The pages are operands as they lie in memory (kind::f8f6f4): nothing is widened on
// the way, so a key tile costs shared memory only its own 128 d bytes.  Both products
// have the cache as A, with 128 rows, and the few query rows as B:
//   S^T = K Q^T  [128 keys x rows]     A: the K tile, K-major
//   O^T += V^T P^T  [d x rows]         A: the V tile read along its rows, MN-major
// So a thread of the softmax holds one key and all rows: a decode step of 4 or 8 rows
// keeps 128 threads busy, scales are one value a thread, and what a mask hides is
// known from one key.
//
// Precision.  Q and P keep theirs by being several 8-bit operands side by side, as
// columns of one product:
//   q 2^k = q0 + q1 / 16 (+ q2 / 256 for fp16) in e4m3, 2^k bringing a row to
//     [128, 256): 8 (11) bits are 4 + 4 (+ 3), so all are kept, down to 2^-21 of the
//     row's greatest element
//   w = p s_v, rounded to fp16, = w0 + w1 / 8 + w2 / 128 in e5m2: 3 + 4 + 4 bits with the signs
//     of the remainders, so fp16's 11 are kept, down to 2^-34 of the row's greatest weight
//     (unscaled terms would stop at 2^-27, e4m3 ones at 2^-22 or, scaled, 2^-26)
// The products of a term have accumulators of their own, added up in fp32 when they
// are read.  (Measured: the tensor cores add e4m3 products to 2^-21.5 of the sum of
// magnitudes of 128; terms 2^-25 below the greatest of an addition are lost.)
// The scale of a V block goes into the exponent, p s_v = 2^(x + log2 s_v - m), with m
// the running max of that sum: blocks of any scales meet in one accumulator.  l takes
// p, which is the weight over s_v, times 2^-20 (see kSumUnit).
//
// As for 16-bit pages, one CTA per SM is persistent over its share of the list of key
// tiles of all (sequence, key head, row tile) units (tree_walk.cuh); partials are
// joined by a dependent kernel in CTA order.  Even and odd key tiles go to two
// softmax warpgroups with their own accumulators and states, merged at the segment's
// end.  m moves only when a row's weight would pass 2^5.8 of it: one vote a tile, whose
// outcome is awaited after the weights have been formed.  A
// segment's tiles are taken from its end: near keys tend to weigh most, with distance
// slopes always, and m then moves in the first tiles alone.
//
// This is the form for up to 16 query rows a key head, a decode step above all; what it
// shares with tree_e4m3_wide.cuh is here too.  It is bound by HBM once a batch's caches are
// large, before that by the chain of two launches, page numbers, tiles and the join.
// Measured (bf16, blocks of 64, GPU time of both kernels replayed as a graph; "of measured":
// of this GPU type's copy rate, 6.78 TB/s):
//   B64 H32 kv8 T1 ctx 4096 .. 8192 d128, a token's heads side by side  137 to 140 us,
//     5.8 TB/s, 86 % of measured (the same over 16-bit pages: 258 to 267 us)
//   B64 H32 kv8 T1 ctx 4000 d128  96 us; T4 (16 rows) 112 us
//   B8 H32 kv8 ctx 6000 d128  4 rows 29 us, 16 rows 36.5 us
//   B1 H32 kv8 T1 d128  ctx 700 14.4 to 16 us, ctx 32000 25 us, ctx 100000 48 us
//
// Warps 0-3 and 4-7: softmax of the even and odd tiles; 8 and 9: TMA loads of the even and
// odd tiles, 10 and 11: their scales, with the pages' numbers some tiles ahead; 12 and
// 13: the products Q and V take part in, each issued as soon as its own operands are
// there; 14: the queries' terms and rows' tables, a segment ahead.
#pragma once

#include <climits>
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "mod_common.cuh"
#include "sm100_ptx8.cuh"
#include "tree_e4m3_internal.h"
#include "tree_walk.cuh"

namespace osattn {
namespace tree8 {

using tree::BN;
using tree::Walk;
using tree::kBadArg;

constexpr int kThreads = 512;
constexpr int kWarpLoad = 8, kWarpScale = 10, kWarpScores = 12, kWarpOut = 13, kWarpQuery = 14;
constexpr uint32_t kTmemCols = 512, kOCol0 = 256;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTop = 10.f;    // weights are formed as 2^10 times themselves,
constexpr float kMost = 15.8f;  // and m moves before they pass e5m2's 57344 (2^15.8 = 57052)
constexpr float kFine1 = 8.f, kFine2 = 128.f;  // see weights_of
constexpr float kNoPage = -1.f;
constexpr float kLeastScale = 7.8886090522101181e-31f;  // 2^-100
// l is summed as 2^-20 weight / s_v: up to 2^(15.8 + 100 - 20) a key, so that 2^30 keys of the
// least scale, a block of zeros', stay below 2^127.  (Without the 2^-20 some 4700 keys
// passed it.)  At s_v = 2^112 a row's greatest key still adds 2^-122; fp32 loses bits from there on.
constexpr float kSumLog2 = -20.f, kSumUnit = 9.5367431640625e-07f;

enum : uint32_t {
  kSiteQ = 101,
  kSiteQEmpty,
  kSiteK,
  kSiteV,
  kSiteScale,
  kSiteEmpty,
  kSiteS,
  kSiteVote,
  kSiteMove,
  kSiteP,
  kSitePv,
  kSiteOEmpty,
  kSiteMerge,
  kSiteZero
};

constexpr int up16(int x) { return (x + 15) / 16 * 16; }

// Column of term c of the weights of group g's first row: the terms of two groups of rows
// lie side by side, so that a thread writes them as 16 bytes.
template <int NG>
__host__ __device__ constexpr int out_col(int g, int c) {
  return (g ^ 1) < NG ? 48 * (g / 2) + 16 * c + 8 * (g & 1) : 24 * g + 8 * c;
}

// NG: groups of 8 rows of a tile.
template <int HD, bool kF16, int NG>
struct Cfg {
  static constexpr int kRows = 8 * NG;
  static constexpr int kTerms = kF16 ? 3 : 2;             // of a query row
  static constexpr int kSGroup = 8 * kTerms;  // columns of a group of rows
  static constexpr int kSCols = up16(NG * kSGroup), kOCols = up16(NG * 24);
  static constexpr int kTileBytes = BN * HD;
  static constexpr int kQBytes = kSCols * HD, kPBytes = kOCols * BN;
  static_assert(kSCols <= 128 && kOCols <= 128, "tensor memory columns");
};

template <int kRows>
struct __align__(16) Shared {
  uint64_t q_full[2], q_empty[2];              // 32 and 256 arrivals
  // a slot holds a K tile, a V tile and their keys' scales
  uint64_t k_full[6], v_full[6], scale_full[6], empty[6];  // 1, 1, 64, 1 arrivals
  uint64_t s_full[2];
  uint64_t vote[2], move[2];  // 4 arrivals: the warps of a warpgroup
  uint64_t p_full[2];         // 128 arrivals
  uint64_t pv_done[2];
  uint64_t o_empty;           // 256 arrivals: the accumulators have been read
  uint64_t merge;             // 256 arrivals: both states of the segment are stored
  uint64_t drain[2];
  uint32_t tmem_base;
  int abort_flag;
  Walk start;
  int warp_sum[kThreads / 32];
  uint32_t flag[2][2];        // [warpgroup][tile parity]: number of the tile + 1 if m has to move
  // of the rows, a segment's in turn
  struct __align__(16) Table {
    float fac[kRows];    // scale log2(e) 2^-k, 0 for no row, NaN for a row that is not finite
    float fall[kRows];   // -slope log2(e)
    float depth[kRows];  // of the row's draft
    int lo[kRows];       // first key of the context that the row sees (INT_MAX: none)
    unsigned long long mask[kRows];  // drafts that it sees, those a window away left out
    int sees[kRows];
    int any;
  } table[2];
  float k_scale[6][BN], v_scale[6][BN];  // kNoPage in v_scale: the key's page does not exist
  __align__(16) float rise[2][4][kRows];   // kTop - m of a warpgroup's rows, a copy for each warp
  __align__(16) float alpha[2][4][kRows], step[2][4][kRows];  // likewise, of the last move
  float top[2][4][kRows];                  // greatest x of a tile, by warp
  float m[2][kRows], l[2][4][kRows];   // the segment's states
  struct End {
    float f[2], lse;   // factors of the two accumulators
    int h, tok;        // of O's row (h = -1: no row)
  } end[2][4][kRows / 2];  // of the rows that a warpgroup finishes, a copy for each warp
};

template <int HD, bool kF16, int NG>
struct Mem {
  using C = Cfg<HD, kF16, NG>;
  static constexpr int kFixed = 2 * C::kQBytes + 2 * C::kPBytes + static_cast<int>(sizeof(Shared<C::kRows>));
  static constexpr int kFit = (232448 - kFixed) / (2 * C::kTileBytes);
  static constexpr int kSlots = kFit < 6 ? kFit : 6;  // of K tiles, and as many of V tiles
  static constexpr int kRing = 2 * kSlots * C::kTileBytes;
  static constexpr int kBytes = kRing + kFixed;
  static_assert(kSlots >= 3, "tiles in flight");
};

// n / d for 0 <= n < 2^31, d fixed: mul is 2^(31 + ceil(log2 d)) / d rounded up.
struct Divisor {
  uint32_t mul, shift, d;
  __device__ __forceinline__ int of(int n) const {
    return static_cast<int>(d == 1u ? n : __umulhi(static_cast<uint32_t>(n), mul) >> shift);
  }
};

struct Params {
  const uint16_t* Q;
  long long q_sb, q_sh, q_sn;
  uint16_t* O;
  long long o_sb, o_sh, o_sn;
  float* LSE;  // [B, H, T]
  const int32_t* table;
  const int32_t* ctx;
  const long long* mask;  // [B, T] or null
  const float* k_scale;   // [num_pages, Hkv, scales]
  const float* v_scale;
  int scales;             // of a page
  Divisor by_page, by_block;  // by the rows of a page, the tokens of a scale
  int B, H, Hkv, group, T;
  int rows;       // T * group
  int tile_rows;  // of a unit
  int row_tiles;
  int lanes, list_heads;  // key heads of a group, groups
  static constexpr bool kLeads = false;  // (the first form is 2 to 5 % slower with them)
  int max_pages, page, num_pages;
  int box_rows;  // keys of one TMA box: min(page, 128)
  int window;
  float scale_log2;       // scale log2(e)
  float cap2, inv_cap2;   // cap log2(e), 0 without a cap
  float cap_k[4];         // cap2 tanh(z) = z (k0 + z^2 (k1 + ..)) for |z| <= 0.4
  const float* slopes;
  float* o_part;    // [2 grid][tile_rows][d]
  float* lse_part;  // [2 grid][tile_rows]
  int* head;        // [B + 1]
  unsigned int* status;
  uint64_t wait_limit_ns;
};

template <uint32_t N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// (the list counts groups of lanes heads, of which this CTA has one)
template <class P>
__device__ __forceinline__ bool next_segment(const P& p, Walk& w) {
  if (!tree::walk_next(p, w)) return false;
  w.hk = w.hk * p.lanes + static_cast<int>(blockIdx.x % static_cast<unsigned>(p.lanes));
  return true;
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > limit_ns) return;
  }
}

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A load that stays where it is written, so that it is under way when its value is wanted.
template <class T>
__device__ __forceinline__ T load_ahead(const T* p) {
  uint32_t r;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(r) : "l"(p));
  return *reinterpret_cast<const T*>(&r);
}

__device__ __forceinline__ void copy_ahead(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Two halves as e4m3, and back (exact).
__device__ __forceinline__ uint16_t e4m3_of(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return r;
}
__device__ __forceinline__ __half2 halves_of(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return *reinterpret_cast<const __half2*>(&r);
}
// x as term[0] + term[1] / 16 + ..; each remainder is exact in fp16.
template <int N>
__device__ __forceinline__ void terms_of(__half2 x, uint16_t* term) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    term[i] = e4m3_of(x);
    if (i + 1 < N) x = __hmul2(__hsub2(x, halves_of(term[i])), __float2half2_rn(16.f));
  }
}

// Two halves as e5m2.
__device__ __forceinline__ uint16_t e5m2_of(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return r;
}

// Four non-negative fp16 values (lo: 0 and 1) as three e5m2 terms whose sum they are: a
// term is the value's upper byte, rounded; the remainder is exact in fp16, and after two
// terms there are 3 bits of it, or less than half of e5m2's least value.
// kFine: the value is term[0] + term[1] 2^-3 + term[2] 2^-7, which fills e5m2's range from above
// (remainders of values up to 2^15.8 are at most 2^12 and 2^8) and keeps all but 2^-24 of
// values below its least step, too.  (Without the factors the part of 100000 keys 2^-26 below
// the row's greatest was off by 40 %; B8 H32 kv8 ctx 6000 d128, 16 rows 35.1 us without, 36.5
// with them, 4 rows 29 us either way.)
template <bool kFine>
__device__ __forceinline__ void weights_of(uint32_t lo, uint32_t hi, uint32_t* term) {
  __half2 x[2] = {*reinterpret_cast<__half2*>(&lo), *reinterpret_cast<__half2*>(&hi)};
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if constexpr (kFine) {
      if (i > 0) {
        const __half2 finer = __float2half2_rn(i == 1 ? kFine1 : kFine2 / kFine1);
        x[0] = __hmul2(x[0], finer);
        x[1] = __hmul2(x[1], finer);
      }
      if (i == 2) {  // (a cvt: NaN has to stay)
        term[2] = __byte_perm(e5m2_of(x[0]), e5m2_of(x[1]), 0x5410);
        return;
      }
    }
    uint32_t e[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      e[k] = *reinterpret_cast<uint32_t*>(&x[k]);
      if (i < 2) {
        e[k] += 0x00800080u;
        const uint32_t kept = e[k] & 0xff00ff00u;
        x[k] = __hsub2(x[k], *reinterpret_cast<const __half2*>(&kept));
      }
    }
    term[i] = __byte_perm(e[0], e[1], 0x7531);
  }
}

template <bool kF16>
__device__ __forceinline__ float widen(uint16_t x) {
  if constexpr (kF16) return __half2float(__ushort_as_half(x));
  else return __uint_as_float(static_cast<uint32_t>(x) << 16);
}

__device__ __forceinline__ void load8(const float* p, uint64_t* x) {
  const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(p), b = *reinterpret_cast<const ulonglong2*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

// Eight values of each lane joined over the warp; lane bits 4, 3, 2 choose the one that
// the lane gets (the row's bits 2, 1, 0).  Halves of the rows change sides until a lane
// has one.
template <class F>
__device__ __forceinline__ float over_warp(float* v, F join) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 16, n = 4; n > 0; off >>= 1, n >>= 1) {
    const bool upper = (lane & off) != 0;
#pragma unroll
    for (int r = 0; r < n; ++r) {
      const float mine = upper ? v[r + n] : v[r], other = upper ? v[r] : v[r + n];
      v[r] = join(mine, __shfl_xor_sync(0xffffffffu, other, off));
    }
  }
  v[0] = join(v[0], __shfl_xor_sync(0xffffffffu, v[0], 2));
  return join(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}
__device__ __forceinline__ int row_of_lane(int lane) { return ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1); }

// Eight base-2 logits capped: cap2 tanh(z), z = y / cap2, by mod_common.cuh's polynomial
// for |z| <= 0.4, which is all that the near form has (size: the greatest |z| so far);
// the far form takes the others from e^{2 z}, off by 2^-20 of the cap at most.
template <bool kFar>
__device__ __forceinline__ void cap_scores(const Params& p, uint64_t* y, float& size) {
  const uint64_t inv = f2_pack(p.inv_cap2, p.inv_cap2), k0 = f2_pack(p.cap_k[0], p.cap_k[0]),
                 k1 = f2_pack(p.cap_k[1], p.cap_k[1]), k2 = f2_pack(p.cap_k[2], p.cap_k[2]),
                 k3 = f2_pack(p.cap_k[3], p.cap_k[3]);
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const uint64_t v = f2_mul(y[r], inv), v2 = f2_mul(v, v);
    float z0, z1;
    f2_unpack(v, z0, z1);
    size = fmax3(size, fabsf(z0), fabsf(z1));  // (NaN stays NaN in either form)
    y[r] = f2_mul(v, f2_fma(v2, f2_fma(v2, f2_fma(v2, k3, k2), k1), k0));
    if constexpr (kFar) {
      float c0, c1;
      f2_unpack(y[r], c0, c1);
      const float f0 = fmaf(cap_r(z0, 2.f * kLog2e), -2.f * p.cap2, p.cap2);
      const float f1 = fmaf(cap_r(z1, 2.f * kLog2e), -2.f * p.cap2, p.cap2);
      y[r] = f2_pack(fabsf(z0) <= 0.4f ? c0 : f0, fabsf(z1) <= 0.4f ? c1 : f1);
    }
  }
}

// ------------------------------------------------------------------ softmax
template <int HD, bool kF16, int NG, int MODE, class Sh>
__device__ __forceinline__ void softmax_role(const Params& p, Sh* sh, uint8_t* sV, uint8_t* sP, uint32_t tmem, int t,
                                             WaitCtl wc) {
  using C = Cfg<HD, kF16, NG>;
  constexpr int kSlots = Mem<HD, kF16, NG>::kSlots;
  constexpr int kRows = C::kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, me = quarter * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t s_addr = lane_base + static_cast<uint32_t>(t * 128);
  const uint32_t o_addr = lane_base + kOCol0 + static_cast<uint32_t>(t * 128);
  uint8_t* const my_p = sP + t * C::kPBytes + me * 16;
  float* const rise = sh->rise[t][quarter];
  float* const alphas = sh->alpha[t][quarter];
  float* const steps = sh->step[t][quarter];
  uint32_t cnt = 0, moves = 0, seg = 0, tiles = 0;  // tiles of this warpgroup; phases of `move`; segments; all tiles
  bool ok = true;
  for (Walk w = sh->start; ok && next_segment(p, w); ++seg) {
    const int buf = seg & 1;
    const auto& tab = sh->table[buf];
    const int ctx = w.ctx, end = ctx + p.T;
    const int last = w.tile0 + w.n - 1;  // tile i is key tile last - i
    ok = warp_wait(&sh->q_full[buf], (seg >> 1) & 1u, wc, kSiteQ);
    if (!ok) break;
    const bool any = tab.any != 0;  // whether a row sees anything
    // m of a row that has seen nothing yet is kTop: its exponents are its logits
    unsigned blank = 0u;  // of rows lane, lane + 32: they see something, but have not yet
    bool unset = any;     // whether there is such a row
    for (int r = lane; r < kRows; r += 32) {
      rise[r] = 0.f;
      blank |= tab.sees[r] ? 1u << (r / 32) : 0u;
    }
    __syncwarp();
    uint64_t l[kRows / 2];
#pragma unroll
    for (int r = 0; r < kRows / 2; ++r) l[r] = 0ull;
    // the scales of this tile's key, and, when they are there early enough, of the next one's
    float ks = 0.f, vs = 1.f;
    bool have = false;
    auto fetch = [&](uint32_t n) {
      ks = sh->k_scale[n % kSlots][me];
      vs = sh->v_scale[n % kSlots][me];
    };
    for (int i = t; i < w.n; i += 2) {
      const int key = (last - i) * BN + me;
      const bool masked = tree::tile_masked(p, ctx, (last - i) * BN);
      bool seen = any;
      unsigned hidden[NG];  // rows that do not see the key
#pragma unroll
      for (int g = 0; g < NG; ++g) hidden[g] = 0u;
      if (masked) {
        seen = false;
        const int u = key - ctx;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const bool sees = u < 0 ? key >= tab.lo[8 * g + r] : u < 64 && ((tab.mask[8 * g + r] >> (u & 63)) & 1ull);
            hidden[g] |= sees ? 0u : 1u << r;
            seen = seen || sees;
          }
        }
      }
      // a key's own place, which for a draft is its depth
      [[maybe_unused]] float before = 0.f;  // places from the key to the context's end (a draft's: its depth)
      if constexpr (mode_slopes(MODE))
        before = static_cast<float>(key >= ctx && key < end ? -tree::depth_of(tree::mask_of(p, w.b, key - ctx)) : ctx - key);
      const uint32_t n = tiles + static_cast<uint32_t>(i), slot = n % kSlots;
      if (!have) {
        ok = warp_wait(&sh->scale_full[slot], (n / kSlots) & 1u, wc, kSiteScale);
        if (!ok) break;
        fetch(n);
      }
      if (vs == kNoPage) {  // (reads as zeros)
        if (seen) atomicMax(p.status, kBadArg);
        vs = 1.f;
      }
      vs = vs < kLeastScale ? kLeastScale : vs;  // (values of a scale of 0 are 0, and their keys count all the same)
      const float lv = seen ? lg2_approx(vs) : 0.f, inv = seen ? kSumUnit * rcp_approx(vs) : 0.f;
      const uint64_t ks2 = f2_pack(ks, ks), lv2 = f2_pack(lv, lv), inv2 = f2_pack(inv, inv);
      const uint64_t finer2 = f2_pack(0.0625f, 0.0625f);
      [[maybe_unused]] const uint64_t before2 = f2_pack(before, before);
      ok = warp_wait(&sh->s_full[t], cnt & 1u, wc, kSiteS);
      if (!ok) break;
      tc_fence_after_sync();
      uint64_t x[kRows / 2];    // exponents of the weights
      float most4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, most;  // the greatest (four chains)
      [[maybe_unused]] float size = 0.f;
      uint32_t raw[NG * C::kSGroup];
      #pragma unroll
      for (int c = 0; c < NG * C::kTerms; ++c) tmem_ld_32x32b_x8(s_addr + 8 * c, raw + 8 * c);
      tmem_ld_wait();
      reg_fence<NG * C::kSGroup>(raw);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t* s = raw + g * C::kSGroup;
        uint64_t y[4], up[4];
        load8(rise + 8 * g, up);
        auto pair = [&](int c, int r) {
          return f2_pack(__uint_as_float(s[8 * c + 2 * r]), __uint_as_float(s[8 * c + 2 * r + 1]));
        };
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          uint64_t a = pair(1, r);
          if constexpr (kF16) a = f2_fma(pair(2, r), finer2, a);
          y[r] = f2_fma(a, finer2, pair(0, r));
        }
        uint64_t fac[4];
        load8(tab.fac + 8 * g, fac);
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = f2_mul(y[r], f2_mul(fac[r], ks2));
        if constexpr (mode_cap(MODE)) cap_scores<true>(p, y, size);
        if constexpr (mode_slopes(MODE)) {
          uint64_t fall[4], depth[4];
          load8(tab.fall + 8 * g, fall);
          load8(tab.depth + 8 * g, depth);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            y[r] = f2_fma(fall[r], f2_add(depth[r], before2) & 0x7fffffff7fffffffull, y[r]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = f2_add(y[r], f2_add(up[r], lv2));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[4 * g + r] = y[r];
          float e0, e1;
          f2_unpack(y[r], e0, e1);
          most4[r] = fmax3(most4[r], e0, e1);
        }
      }
      most = fmax3(fmaxf(most4[0], most4[1]), most4[2], most4[3]);
      if (masked) {
        most = -INFINITY;
#pragma unroll
        for (int r = 0; r < kRows / 2; ++r) {
          float e0, e1;
          f2_unpack(x[r], e0, e1);
          if ((hidden[r / 4] >> (2 * (r & 3))) & 1u) e0 = -INFINITY;
          if ((hidden[r / 4] >> (2 * (r & 3) + 1)) & 1u) e1 = -INFINITY;
          x[r] = f2_pack(e0, e1);
          most = fmax3(most, e0, e1);
        }
      }
      tc_fence_before_sync();
      const bool over = unset || __any_sync(0xffffffffu, most > kMost);
      if (lane == 0) {
        if (over) sh->flag[t][cnt & 1] = cnt + 1;
        mbar_arrive(&sh->vote[t]);  // S has been read, too
      }
      // the last tile's product has read P and written O
      if (cnt > 0) ok = warp_wait(&sh->pv_done[t], (cnt - 1) & 1u, wc, kSitePv);
      if (!ok) break;
      // the next tile's scales, if they are there
      have = i + 2 < w.n && __all_sync(0xffffffffu, mbar_test(&sh->scale_full[(n + 2) % kSlots], ((n + 2) / kSlots) & 1u));
      if (have) fetch(n + 2);
      // The weights' terms: at once where this warp has no reason to move m, and once more
      // where another one has.
      bool formed = false, settled = false;
      for (bool now = !over;; now = true) {
        if (now) {
          formed = true;
          uint32_t h[kRows / 2], even[3][2];  // fp16 pairs; terms of the last even group
#pragma unroll
          for (int r = 0; r < kRows / 2; ++r) {
            float e0, e1;
            f2_unpack(x[r], e0, e1);
            e0 = ex2_approx(e0);
            e1 = ex2_approx(e1);
            l[r] = f2_fma(f2_pack(e0, e1), inv2, l[r]);
            h[r] = pack_f16x2(e0, e1);
          }
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            uint32_t term[2][3];
            weights_of<true>(h[4 * g], h[4 * g + 1], term[0]);
            weights_of<true>(h[4 * g + 2], h[4 * g + 3], term[1]);
#pragma unroll
            for (int c = 0; c < 3; ++c) {
              const int col = out_col<NG>(g & ~1, c);
              uint8_t* dst = my_p + (col / 16) * (BN * 16) + col % 16;
              if ((g & 1) == 0) {
                even[c][0] = term[0][c];
                even[c][1] = term[1][c];
                if (g + 1 == NG) *reinterpret_cast<uint2*>(dst) = make_uint2(term[0][c], term[1][c]);
              } else {
                *reinterpret_cast<uint4*>(dst) = make_uint4(even[c][0], even[c][1], term[0][c], term[1][c]);
              }
            }
          }
        }
        if (settled) break;
        settled = true;
        ok = warp_wait(&sh->vote[t], cnt & 1u, wc, kSiteVote);
        if (!ok || *reinterpret_cast<volatile uint32_t*>(&sh->flag[t][cnt & 1]) != cnt + 1) break;
        if (formed) {  // take the tile out of the sums again (to 2^-24 of them)
          const uint64_t less = f2_pack(-inv, -inv);
#pragma unroll
          for (int r = 0; r < kRows / 2; ++r) {
            float e0, e1;
            f2_unpack(x[r], e0, e1);
            l[r] = f2_fma(f2_pack(ex2_approx(e0), ex2_approx(e1)), less, l[r]);
          }
        }
        // m moves to the rows' greatest x; each warp keeps a copy of all rows' m
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float v[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) f2_unpack(x[4 * g + r], v[2 * r], v[2 * r + 1]);
          const float great = over_warp(v, [](float a, float b) { return fmaxf(a, b); });
          if ((lane & 3) == 0) sh->top[t][quarter][8 * g + row_of_lane(lane)] = great;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->move[t]);
        ok = warp_wait(&sh->move[t], moves & 1u, wc, kSiteMove);
        if (!ok) break;
        ++moves;
        for (int r = lane; r < kRows; r += 32) {
          const float great = fmaxf(fmaxf(sh->top[t][0][r], sh->top[t][1][r]), fmaxf(sh->top[t][2][r], sh->top[t][3][r]));
          const bool first = (blank >> (r / 32)) & 1u;  // from nothing to the tile's greatest, if there is one
          const float step = first ? (great == -INFINITY ? 0.f : great - kTop) : fmaxf(great - kTop, 0.f);
          if (great != -INFINITY) blank &= ~(1u << (r / 32));
          rise[r] -= step;
          steps[r] = step;
          alphas[r] = first ? 1.f : ex2_approx(-step);
        }
        unset = __any_sync(0xffffffffu, blank != 0u);
        __syncwarp();
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          uint64_t al[4], st[4];
          load8(alphas + 8 * g, al);
          load8(steps + 8 * g, st);
          bool any = false;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            l[4 * g + r] = f2_mul(l[4 * g + r], al[r]);
            x[4 * g + r] = f2_add(x[4 * g + r], st[r] ^ 0x8000000080000000ull);
            any = any || al[r] != 0x3f8000003f800000ull;
          }
          if (i != t && any) {  // (any: the same for all threads)
            tc_fence_after_sync();
            uint32_t o[24];
#pragma unroll
            for (int c = 0; c < 3; ++c) tmem_ld_32x32b_x8(o_addr + out_col<NG>(g, c), o + 8 * c);
            tmem_ld_wait();
            reg_fence<24>(o);
#pragma unroll
            for (int c = 0; c < 24; c += 2) {
              float o0, o1;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(o[c]), __uint_as_float(o[c + 1])), al[(c & 7) / 2]), o0, o1);
              o[c] = __float_as_uint(o0);
              o[c + 1] = __float_as_uint(o1);
            }
#pragma unroll
            for (int c = 0; c < 3; ++c) tmem_st_32x32b_x8(o_addr + out_col<NG>(g, c), o + 8 * c);
          }
        }
        tmem_st_wait();
        tc_fence_before_sync();
      }
      if (!ok) break;
      if (masked) {  // rows of V that no row of the tile sees may hold anything
        ok = warp_wait(&sh->v_full[slot], (n / kSlots) & 1u, wc, kSiteZero);
        if (!ok) break;
        if (!seen) {
          uint4* v = reinterpret_cast<uint4*>(sV + slot * C::kTileBytes + me * HD);
#pragma unroll
          for (int c = 0; c < HD / 16; ++c) v[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_async_smem();
      mbar_arrive(&sh->p_full[t]);
      ++cnt;
    }
    if (!ok) break;
    // ---- the segment's end: both states, then four rows of each group a warpgroup
    const bool had = t < w.n;
    if (had) ok = warp_wait(&sh->pv_done[t], (cnt - 1) & 1u, wc, kSitePv);
    // (without a tile of its own: the last segment's states have been read)
    else if (seg > 0) ok = warp_wait(&sh->o_empty, (seg - 1) & 1u, wc, kSiteOEmpty);
    if (!ok) break;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float v[8];
#pragma unroll
      for (int r = 0; r < 4; ++r) f2_unpack(l[4 * g + r], v[2 * r], v[2 * r + 1]);
      const float sum = over_warp(v, [](float a, float b) { return a + b; });
      if ((lane & 3) == 0) sh->l[t][quarter][8 * g + row_of_lane(lane)] = sum;
    }
    if (quarter == 0)
      for (int r = lane; r < kRows; r += 32) sh->m[t][r] = had && !((blank >> (r / 32)) & 1u) ? kTop - rise[r] : -INFINITY;
    mbar_arrive(&sh->merge);
    ok = warp_wait(&sh->merge, seg & 1u, wc, kSiteMerge);
    if (!ok) break;
    tc_fence_after_sync();
    const bool whole = !w.head_cut && !w.tail_cut;
    const int row0 = w.rt * p.tile_rows, count = min(p.tile_rows, p.rows - row0);
    const long long slot = (2 * static_cast<long long>(blockIdx.x) + (w.head_cut ? 0 : 1)) * p.tile_rows;
    // a lane a row: factors and places (every warp for itself, the same values)
    if (lane < kRows / 2) {
      const int row = 8 * (lane >> 2) + 4 * t + (lane & 3);  // rows 4 t .. of each group
      typename Sh::End e;
      e.h = -1;
      if (row < count) {
        const float m0 = sh->m[0][row], m1 = sh->m[1][row];
        const float M = fmaxf(m0, m1);
        const float f0 = m0 == -INFINITY ? 0.f : ex2_approx(m0 - M), f1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - M);
        const float l0 = (sh->l[0][0][row] + sh->l[0][1][row]) + (sh->l[0][2][row] + sh->l[0][3][row]);
        const float l1 = (sh->l[1][0][row] + sh->l[1][1][row]) + (sh->l[1][2][row] + sh->l[1][3][row]);
        const float L = fmaf(l0, f0, l1 * f1);
        const bool empty = L == 0.f || tab.sees[row] == 0;
        const float rcp = empty ? 0.f : kSumUnit / L;
        e.f[0] = f0 * rcp;
        e.f[1] = f1 * rcp;
        e.lse = empty ? -INFINITY : (M + (log2f(L) - (kTop + kSumLog2))) * kLn2;
        e.tok = (row0 + row) / p.group;
        e.h = w.hk * p.group + (row0 + row) - e.tok * p.group;
        if (quarter == 0) {
          if (whole) p.LSE[(static_cast<long long>(w.b) * p.H + e.h) * p.T + e.tok] = e.lse;
          else p.lse_part[slot + row] = e.lse;
        }
      }
      sh->end[t][quarter][lane] = e;
    }
    __syncwarp();
#pragma unroll 1
    for (int g = 0; g < NG; ++g) {
      uint32_t a[2][12];
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (s == 0 || w.n > 1) {
#pragma unroll
          for (int c = 0; c < 3; ++c) tmem_ld_32x32b_x4(lane_base + kOCol0 + s * 128 + out_col<NG>(g, c) + 4 * t, a[s] + 4 * c);
        }
      tmem_ld_wait();
      reg_fence<12>(a[0]);
      reg_fence<12>(a[1]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const typename Sh::End e = sh->end[t][quarter][4 * g + r];
        if (e.h < 0) continue;
        auto sum = [&](int s) {
          return fmaf(__uint_as_float(a[s][8 + r]), 1.f / kFine2, fmaf(__uint_as_float(a[s][4 + r]), 1.f / kFine1, __uint_as_float(a[s][r])));
        };
        float o = sum(0) * e.f[0];
        if (w.n > 1) o = fmaf(sum(1), e.f[1], o);
        if (e.lse == -INFINITY) o = 0.f;
        if (me < HD) {
          if (whole) {
            const uint32_t packed = kF16 ? pack_f16x2(o, 0.f) : pack_bf16x2(o, 0.f);
            p.O[w.b * p.o_sb + e.h * p.o_sh + e.tok * p.o_sn + me] = static_cast<uint16_t>(packed);
          } else {
            p.o_part[(slot + 8 * g + 4 * t + r) * HD + me] = o;
          }
        }
      }
    }
    tc_fence_before_sync();
    mbar_arrive(&sh->o_empty);
    mbar_arrive(&sh->q_empty[buf]);
    tiles += static_cast<uint32_t>(w.n);
  }
}

// ------------------------------------------------------------------ queries
// One warp: the rows' tables, and their elements as e4m3 terms in the K-major layout
// without a swizzle (16-byte pieces of all rows side by side).
template <int HD, bool kF16, int NG, class Sh>
__device__ __forceinline__ void query_role(const Params& p, Sh* sh, uint8_t* sQ, WaitCtl wc) {
  using C = Cfg<HD, kF16, NG>;
  constexpr int kPer = HD / 4;  // elements of a row a lane
  const int lane = threadIdx.x & 31;
  uint32_t seg = 0;
  bool ok = true;
  for (Walk w = sh->start; ok && next_segment(p, w); ++seg) {
    const int buf = seg & 1;
    if (seg >= 2) ok = warp_wait(&sh->q_empty[buf], ((seg >> 1) - 1) & 1u, wc, kSiteQEmpty);
    if (!ok) break;
    auto& tab = sh->table[buf];
    const int row0 = w.rt * p.tile_rows, count = min(p.tile_rows, p.rows - row0);
    bool any = false;
    for (int r = lane; r < C::kRows; r += 32) {
      unsigned long long mask = 0ull;
      float slope = 0.f;
      if (r < count) {
        const int tok = (row0 + r) / p.group;
        mask = tree::mask_of(p, w.b, tok);
        if (p.slopes) slope = __ldg(p.slopes + w.hk * p.group + (row0 + r) - tok * p.group) * kLog2e;
      }
      const int depth = tree::depth_of(mask);
      tab.sees[r] = mask != 0ull;
      any = any || mask != 0ull;
      tab.depth[r] = static_cast<float>(depth);
      tab.fall[r] = -slope;
      tab.lo[r] = mask == 0ull ? INT_MAX : (p.window > 0 ? max(0, w.ctx + depth - p.window + 1) : 0);
      if (mask != 0ull && p.window > 0 && p.T >= p.window)  // (depths are -1 .. T - 1)
        for (int u = 0; u < p.T; ++u)
          if (((mask >> u) & 1ull) && abs(depth - tree::depth_of(tree::mask_of(p, w.b, u))) >= p.window) mask &= ~(1ull << u);
      tab.mask[r] = mask;
    }
    any = __any_sync(0xffffffffu, any);
    if (lane == 0) tab.any = any;
    // Four lanes a row, eight rows at once.
    uint8_t* q = sQ + buf * C::kQBytes;
    const int part = lane & 3;
    auto load = [&](int g, uint4* e) {
      const int r = 8 * g + (lane >> 2), row = row0 + r, tok = row / p.group;
      const uint16_t* src = p.Q + w.b * p.q_sb + (w.hk * p.group + row - tok * p.group) * p.q_sh + tok * p.q_sn + kPer * part;
#pragma unroll
      for (int i = 0; i < kPer / 8; ++i)
        e[i] = r < count ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0u, 0u, 0u, 0u);
    };
    auto greatest = [&](const uint4* e) {  // magnitudes, as two 16-bit values at a time
      unsigned most = 0u;
#pragma unroll
      for (int i = 0; i < kPer / 8; ++i)
        most = __vmaxu2(most, __vmaxu2(__vmaxu2(e[i].x & 0x7fff7fffu, e[i].y & 0x7fff7fffu),
                                       __vmaxu2(e[i].z & 0x7fff7fffu, e[i].w & 0x7fff7fffu)));
      most = max(most & 0xffffu, most >> 16);
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      return widen<kF16>(static_cast<uint16_t>(max(most, __shfl_xor_sync(0xffffffffu, most, 2))));
    };
    auto exponent = [](float great) {  // that brings it to 2^7 ..
      return great == 0.f ? 0 : min(7 - (static_cast<int>(__float_as_uint(great) >> 23) - 127), 107);
    };
#pragma unroll 1
    for (int g = 0; g < NG; ++g) {
      const int r = 8 * g + (lane >> 2);
      uint4 e[kPer / 8];
      load(g, e);
      const float great = greatest(e);
      const int k = exponent(great);
      const float up = __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
      if (part == 0)
        tab.fac[r] = !(great <= 3.402823466e38f) ? __uint_as_float(0x7fc00000u) : (r < count ? p.scale_log2 * down : 0.f);
      uint8_t* dst = q + part * (kPer / 16) * (C::kSCols * 16) + (g * C::kSGroup + (lane >> 2)) * 16;
#pragma unroll
      for (int i = 0; i < kPer / 16; ++i) {  // 16 elements, a piece
        const uint32_t v[8] = {e[2 * i].x, e[2 * i].y, e[2 * i].z, e[2 * i].w,
                               e[2 * i + 1].x, e[2 * i + 1].y, e[2 * i + 1].z, e[2 * i + 1].w};
        uint16_t term[8][C::kTerms];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          terms_of<C::kTerms>(__floats2half2_rn(widen<kF16>(static_cast<uint16_t>(v[j])) * up,
                                                widen<kF16>(static_cast<uint16_t>(v[j] >> 16)) * up), term[j]);
#pragma unroll
        for (int c = 0; c < C::kTerms; ++c)
          *reinterpret_cast<uint4*>(dst + i * (C::kSCols * 16) + 8 * c * 16) =
              make_uint4(__byte_perm(term[0][c], term[1][c], 0x5410), __byte_perm(term[2][c], term[3][c], 0x5410),
                         __byte_perm(term[4][c], term[5][c], 0x5410), __byte_perm(term[6][c], term[7][c], 0x5410));
      }
    }
    fence_async_smem();
    mbar_arrive(&sh->q_full[buf]);
  }
}

// ------------------------------------------------------------------ loads
// Two warps, for the even and odd tiles: lanes 0-15 load box x of a K tile, 16-31 of V.
// Two more copy the scales of four keys a lane, 4 bytes at a time.  The pages' numbers
// are fetched kAhead tiles before they are needed: one by one their latency would be
// that of a tile.  (One warp for all of it took 1300 cycles a tile, the time in which
// HBM brings one.)  A box before every window or behind the drafts, or whose page number
// is not one of the pool's, is read from behind the pool, which fills it with zeros.
constexpr int kAhead = 2;

// A tile, with the page of lane x's box (x < 16, and again from 16 on).
struct Tile {
  int page, in_page, hk;  // in_page -1: the lane's box holds no key
};
// The tiles in order; kStep 2: those of one parity.
template <int kStep = 2>
struct Tiles {
  Walk w;
  int left = 0, at = 0;  // tiles of w's segment that are still to come; the next one's place
  bool skip;
  Tile queue[kAhead];
  bool there[kAhead];

  template <class P>
  __device__ __forceinline__ bool step(const P& p) {
    if (left == 0) {
      if (!next_segment(p, w)) return false;
      left = w.n;
      at = w.tile0 + w.n;
    }
    --left;
    --at;
    return true;
  }
  template <class P>
  __device__ __forceinline__ bool find(const P& p, Tile& x) {
    if (kStep == 2) {
      if (skip && !step(p)) return false;
      skip = true;
    }
    if (!step(p)) return false;
    const int box = threadIdx.x & 15, key = at * BN + box * p.box_rows;
    x.hk = w.hk;
    x.page = x.in_page = -1;
    if (box * p.box_rows < BN && key < w.ctx + p.T && key + p.box_rows > tree::first_key(p, w.ctx)) {
      const int page = p.by_page.of(key);  // < max_pages: ctx + T fits the table
      x.in_page = key - page * p.page;
      x.page = load_ahead(p.table + static_cast<long long>(w.b) * p.max_pages + page);
    }
    return true;
  }
  template <class P>
  __device__ __forceinline__ Tiles(const P& p, const Walk& start, int parity) : w(start), skip(parity != 0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) there[i] = find(p, queue[i]);
  }
  template <class P>
  __device__ __forceinline__ bool next(const P& p, Tile& x) {
    if (!there[0]) return false;
    x = queue[0];
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i) {
      queue[i] = queue[i + 1];
      there[i] = there[i + 1];
    }
    there[kAhead - 1] = there[kAhead - 1] && find(p, queue[kAhead - 1]);
    return true;
  }
};

template <int HD, int kSlots, class P, class Sh>
__device__ __forceinline__ void load_role(const CUtensorMap* tmK, const CUtensorMap* tmV, const P& p, Sh* sh,
                                          uint8_t* sK, uint8_t* sV, int parity, WaitCtl wc) {
  constexpr int kTileBytes = BN * HD;
  const int lane = threadIdx.x & 31, box = lane & 15;
  const bool loads = box * p.box_rows < BN;
  const CUtensorMap* tm = lane < 16 ? tmK : tmV;
  uint64_t* const full = lane < 16 ? sh->k_full : sh->v_full;
  uint8_t* const ring = (lane < 16 ? sK : sV) + box * p.box_rows * HD;
  Tiles<> tiles(p, sh->start, parity);
  Tile x;
  uint32_t n = parity;
  while (tiles.next(p, x)) {
    const uint32_t s = n % kSlots;
    if (n >= kSlots && !warp_wait(&sh->empty[s], (n / kSlots - 1) & 1u, wc, kSiteEmpty)) break;
    if (box == 0) mbar_arrive_expect_tx(&full[s], kTileBytes);
    __syncwarp();
    const bool good = x.in_page >= 0 && x.page >= 0 && x.page < p.num_pages;
    if (loads) tma_load_4d(ring + s * kTileBytes, tm, &full[s], 0, good ? x.in_page : 0, x.hk, good ? x.page : p.num_pages);
    n += 2;
  }
  // Let every load of this warp land before the CTA can exit.
  // (No tile of number n or later: a slot of one from n - kSlots on is not filled again.)
  if (box == 0)
    for (uint32_t i = (n > kSlots ? n - kSlots : parity); i < n; ++i)
      if (((n - i) & 1) == 0) drain_wait(&full[i % kSlots], (i / kSlots) & 1u, wc.limit_ns);
  __syncwarp();
}

template <int kSlots, class Sh>
__device__ __forceinline__ void scale_role(const Params& p, Sh* sh, int parity, WaitCtl wc) {
  const int lane = threadIdx.x & 31;
  const int box = 4 * lane / p.box_rows, in_box = 4 * lane - box * p.box_rows;  // of keys 4 lane ..
  Tiles<> tiles(p, sh->start, parity);
  Tile x;
  uint32_t n = parity;
  while (tiles.next(p, x)) {
    const uint32_t s = n % kSlots;
    if (n >= kSlots && !warp_wait(&sh->empty[s], (n / kSlots - 1) & 1u, wc, kSiteEmpty)) break;
    const bool needed = x.in_page >= 0, good = needed && x.page >= 0 && x.page < p.num_pages;
    const int page = __shfl_sync(0xffffffffu, good ? x.page : (needed ? -2 : -1), box);
    const int row = __shfl_sync(0xffffffffu, x.in_page, box) + in_box;
    float* const ks = &sh->k_scale[s][4 * lane];
    float* const vs = &sh->v_scale[s][4 * lane];
    if (page >= 0) {
      const long long at = (static_cast<long long>(page) * p.Hkv + x.hk) * p.scales;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int block = p.by_block.of(row + j);
        copy_ahead(ks + j, p.k_scale + at + block);
        copy_ahead(vs + j, p.v_scale + at + block);
      }
    } else {
      const float v = page == -2 ? kNoPage : 1.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ks[j] = 0.f;
        vs[j] = v;
      }
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh->scale_full[s])) : "memory");
    mbar_arrive(&sh->scale_full[s]);
    n += 2;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}

// ------------------------------------------------------------------ MMA issuers
template <int HD, bool kF16, int NG, class Sh>
__device__ __forceinline__ void scores_role(const Params& p, Sh* sh, uint32_t tmem, uint8_t* sK, uint8_t* sQ, WaitCtl wc) {
  using C = Cfg<HD, kF16, NG>;
  constexpr int kSlots = Mem<HD, kF16, NG>::kSlots;
  // rows of 128 or 64 bytes, swizzled as a whole; 8-row groups 8 HD bytes apart
  const uint64_t k_desc = sdesc_of(smem_u32(sK), 16, 8 * HD, HD == 128 ? 2u : 4u);
  const uint64_t q_desc = sdesc_of(smem_u32(sQ), C::kSCols * 16, 128, 0);
  constexpr uint32_t kTile = C::kTileBytes >> 4, id = idesc_e4m3_f32(128, C::kSCols, 0, 0);
  uint32_t n = 0, seg = 0, used[2] = {0, 0};
  bool ok = true;
  for (Walk w = sh->start; ok && next_segment(p, w); ++seg) {
    const int buf = seg & 1;
    ok = warp_wait(&sh->q_full[buf], (seg >> 1) & 1u, wc, kSiteQ);
    for (int i = 0; ok && i < w.n; ++i, ++n) {
      const int t = i & 1;
      const uint32_t s = n % kSlots;
      ok = warp_wait(&sh->k_full[s], (n / kSlots) & 1u, wc, kSiteK);
      // the columns' last scores have been read
      if (used[t] > 0) ok = ok && warp_wait(&sh->vote[t], (used[t] - 1) & 1u, wc, kSiteVote);
      if (!ok) break;
      ++used[t];
      tc_fence_after_sync();
      const uint64_t a = sdesc_add(k_desc, s * kTile), b = sdesc_add(q_desc, buf * (C::kQBytes >> 4));
#pragma unroll
      for (int kk = 0; kk < HD / 32; ++kk)
        mma_e4m3_ss(tmem + t * 128, sdesc_add(a, kk * 2), sdesc_add(b, kk * 2 * C::kSCols), id, kk > 0);
      mma_commit<true>(&sh->s_full[t]);
    }
  }
  mma_commit<true>(&sh->drain[0]);
  drain_wait(&sh->drain[0], 0, wc.limit_ns);
  __syncwarp();
}

template <int HD, bool kF16, int NG, class Sh>
__device__ __forceinline__ void out_role(const Params& p, Sh* sh, uint32_t tmem, uint8_t* sV, uint8_t* sP, WaitCtl wc) {
  using C = Cfg<HD, kF16, NG>;
  constexpr int kSlots = Mem<HD, kF16, NG>::kSlots;
  // V along its rows: one block of d elements; at d = 64 the second half of the 128 rows
  // of A repeats the first (a leading offset of 0)
  const uint64_t v_desc = sdesc_of(smem_u32(sV), 0, 8 * HD, HD == 128 ? 2u : 4u);
  const uint64_t p_desc = sdesc_of(smem_u32(sP), 128, BN * 16, 0);
  constexpr uint32_t kTile = C::kTileBytes >> 4, id = idesc_e4m3_f32(128, C::kOCols, 1, 1) | kIdescBE5m2;
  uint32_t n = 0, seg = 0, used[2] = {0, 0};
  bool ok = true;
  for (Walk w = sh->start; ok && next_segment(p, w); ++seg) {
    for (int i = 0; ok && i < w.n; ++i, ++n) {
      const int t = i & 1;
      const uint32_t s = n % kSlots;
      ok = warp_wait(&sh->p_full[t], used[t] & 1u, wc, kSiteP);
      if (i == 0 && seg > 0) ok = ok && warp_wait(&sh->o_empty, (seg - 1) & 1u, wc, kSiteOEmpty);
      ok = ok && warp_wait(&sh->v_full[s], (n / kSlots) & 1u, wc, kSiteV);
      if (!ok) break;
      ++used[t];
      tc_fence_after_sync();
      const uint64_t a = sdesc_add(v_desc, s * kTile), b = sdesc_add(p_desc, t * (C::kPBytes >> 4));
#pragma unroll
      for (int kk = 0; kk < BN / 32; ++kk)
        mma_e4m3_ss(tmem + kOCol0 + t * 128, sdesc_add(a, kk * (32 * HD >> 4)), sdesc_add(b, kk * (512 >> 4)), id,
                    i >= 2 || kk > 0);
      mma_commit<true>(&sh->pv_done[t]);
      mma_commit<true>(&sh->empty[s]);  // (its scores and scales have been read: P is there)
    }
  }
  mma_commit<true>(&sh->drain[1]);
  drain_wait(&sh->drain[1], 0, wc.limit_ns);
  __syncwarp();
}

template <int HD, bool kF16, int NG, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    tree_e4m3_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Params p) {
  using C = Cfg<HD, kF16, NG>;
  using M = Mem<HD, kF16, NG>;
  using Sh = Shared<C::kRows>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles' alignment
    if (threadIdx.x == 0) atomicExch(p.status, 3u /* OSATTN_ERR_CUDA */);
    return;
  }
  uint8_t* sK = smem;
  uint8_t* sV = sK + M::kSlots * C::kTileBytes;
  uint8_t* sQ = smem + M::kRing;
  uint8_t* sP = sQ + 2 * C::kQBytes;
  Sh* sh = reinterpret_cast<Sh*>(sP + 2 * C::kPBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->q_full[i], 32);
      mbar_init(&sh->q_empty[i], 256);
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->vote[i], 4);
      mbar_init(&sh->move[i], 4);
      mbar_init(&sh->p_full[i], 128);
      mbar_init(&sh->pv_done[i], 1);
      sh->flag[i][0] = sh->flag[i][1] = 0u;
    }
    for (int s = 0; s < M::kSlots; ++s) {
      mbar_init(&sh->k_full[s], 1);
      mbar_init(&sh->v_full[s], 1);
      mbar_init(&sh->scale_full[s], 64);
      mbar_init(&sh->empty[s], 1);
    }
    mbar_init(&sh->o_empty, 256);
    mbar_init(&sh->merge, 256);
    mbar_init(&sh->drain[0], 1);
    mbar_init(&sh->drain[1], 1);
    sh->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kWarpLoad && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kWarpOut) {
    tmem_alloc(&sh->tmem_base, kTmemCols);
    tmem_relinquish();
  }
  __syncthreads();
  tree::find_start<kThreads>(p, sh, blockIdx.x / p.lanes, gridDim.x / p.lanes);
  // the combine kernel may take its place (it waits for this one to end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sh->tmem_base;
  const WaitCtl wc{&sh->abort_flag, p.status, p.status + 1, p.wait_limit_ns};
  // with more than 8 rows: 256 x 184 + 256 x 72 = 512 x 128 registers
  if (warp < kWarpLoad) {
    if constexpr (NG > 1) regs_inc<184>();
    softmax_role<HD, kF16, NG, MODE>(p, sh, sV, sP, tmem, warp >> 2, wc);
  } else {
    if constexpr (NG > 1) regs_dec<72>();
    if (warp < kWarpScale) load_role<HD, M::kSlots>(&tmK, &tmV, p, sh, sK, sV, warp - kWarpLoad, wc);
    else if (warp < kWarpScores) scale_role<M::kSlots>(p, sh, warp - kWarpScale, wc);
    else if (warp == kWarpScores) scores_role<HD, kF16, NG>(p, sh, tmem, sK, sQ, wc);
    else if (warp == kWarpOut) out_role<HD, kF16, NG>(p, sh, tmem, sV, sP, wc);
    else if (warp == kWarpQuery) query_role<HD, kF16, NG>(p, sh, sQ, wc);
  }

  __syncwarp();
  tmem_st_wait();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kWarpOut) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ combine
// kWays warps a row (1, or 8 where many CTAs share a unit) join the partials of the
// CTAs that share the row's unit, in CTA order.  Rows of units that one CTA did whole
// are done already.  A dependent launch: it waits for the main kernel's end.
template <int HD, bool kF16, int kWays, class P>
__global__ void __launch_bounds__(256) tree_e4m3_combine(const __grid_constant__ P p, int grid) {
  constexpr int CPL = HD / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_unit = (p.tile_rows * kWays + 7) / 8;
  const int unit_all = blockIdx.x / per_unit, in = blockIdx.x - unit_all * per_unit;
  const int row = kWays == 1 ? in * 8 + warp : in;
  const int way = kWays == 1 ? 0 : warp;
  const int units = p.Hkv * p.row_tiles;
  const int b = unit_all / units, unit = unit_all - b * units;
  const int hk = unit / p.row_tiles, rt = unit - hk * p.row_tiles;
  const int at = rt * p.tile_rows + row;
  if (row >= p.tile_rows || at >= p.rows) return;  // (the whole block if kWays > 1)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int of_b = p.list_heads * p.row_tiles, n_b = (p.head[b + 1] - p.head[b]) / of_b;
  const int lead = tree::lead_of(p, p.head[p.B], grid / p.lanes), base = p.head[b] + lead * of_b * b;
  const int group = hk / p.lanes, lane_head = hk - group * p.lanes;
  const int places = p.head[p.B] + lead * of_b * p.B;
  const long long total = places, G = tree::shares(places, grid / p.lanes);
  const long long x0 = base + static_cast<long long>(group * p.row_tiles + rt) * (n_b + lead) + lead,
                  x1 = x0 + n_b - 1;
  // the share that holds list position x: the largest c with c total / G <= x
  const int c0 = static_cast<int>(((x0 + 1) * G - 1) / total), c1 = static_cast<int>(((x1 + 1) * G - 1) / total);
  if (c0 == c1) return;
  auto row_of = [&](int c) { return static_cast<long long>(2 * (c * p.lanes + lane_head) + (c == c0 ? 1 : 0)) * p.tile_rows + row; };
  float top = -INFINITY;
  for (int c = c0 + way + kWays * lane; c <= c1; c += 32 * kWays) top = fmaxf(top, p.lse_part[row_of(c)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  float l = 0.f, acc[CPL];
#pragma unroll
  for (int k = 0; k < CPL; ++k) acc[k] = 0.f;
  for (int cb = c0 + way; cb <= c1; cb += 32 * kWays) {
    const int n = min(32, (c1 - cb) / kWays + 1);
    const float lse = lane < n ? p.lse_part[row_of(cb + kWays * lane)] : -INFINITY;
    const float weight = lse == -INFINITY ? 0.f : expf(lse - top);  // (NaN stays NaN)
#pragma unroll 8
    for (int x = 0; x < n; ++x) {
      const float w = __shfl_sync(0xffffffffu, weight, x);
      const float* src = p.o_part + row_of(cb + kWays * x) * HD + lane * CPL;
      float o[CPL];
      if constexpr (CPL == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        o[0] = v.x; o[1] = v.y; o[2] = v.z; o[3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        o[0] = v.x; o[1] = v.y;
      }
#pragma unroll
      for (int k = 0; k < CPL; ++k) acc[k] = fmaf(w, o[k], acc[k]);
      l += w;
    }
  }
  if constexpr (kWays > 1) {
    __shared__ float joined[kWays][HD + 2];
#pragma unroll
    for (int k = 0; k < CPL; ++k) joined[warp][lane * CPL + k] = acc[k];
    if (lane == 0) {
      joined[warp][HD] = top;
      joined[warp][HD + 1] = l;
    }
    __syncthreads();
    if (warp != 0) return;
    for (int x = 1; x < kWays; ++x) top = fmaxf(top, joined[x][HD]);
    l = 0.f;
#pragma unroll
    for (int k = 0; k < CPL; ++k) acc[k] = 0.f;
    for (int x = 0; x < kWays; ++x) {
      const float lx = joined[x][HD + 1], w = lx == 0.f ? 0.f : expf(joined[x][HD] - top);
      l = fmaf(lx, w, l);
#pragma unroll
      for (int k = 0; k < CPL; ++k) acc[k] = fmaf(joined[x][lane * CPL + k], w, acc[k]);
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int tok = at / p.group, h = hk * p.group + at - tok * p.group;
  uint16_t* dst = p.O + b * p.o_sb + h * p.o_sh + tok * p.o_sn + lane * CPL;
#pragma unroll
  for (int k = 0; k < CPL; k += 2)
    *reinterpret_cast<uint32_t*>(dst + k) = kF16 ? pack_f16x2(acc[k] * inv, acc[k + 1] * inv) : pack_bf16x2(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0) p.LSE[(static_cast<long long>(b) * p.H + h) * p.T + tok] = l == 0.f ? -INFINITY : top + logf(l);
}

}  // namespace tree8
}  // namespace osattn
