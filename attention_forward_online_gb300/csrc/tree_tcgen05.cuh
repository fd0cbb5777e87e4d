// tree_tcgen05.cuh - attention of drafted tokens over a paged cache: T <= 64
// tokens a sequence (one: the ordinary decode step) attend to the cached keys
// and to those drafts that their mask names, on the tcgen05 tensor cores.
// Built for sm_103a; bf16 or fp16, d = 64 or 128.
//
// What it has to do is read the visible cache once, 4 d bytes a key and key
// head, so the design is about keeping HBM busy:
//   - The query heads of a key head and the drafts of a sequence are the rows
//     of one 128-row operand (row = token x group + head of the group), so a
//     key tile is loaded once for all of them.
//   - One CTA per SM, persistent.  The key tiles of all sequences, key heads
//     and row tiles form one list, cut into equal shares; a share's piece of
//     one (sequence, key head, row tile) is a segment.  Ragged lengths need no
//     plan on the host, and the loads of the next segment run while the last
//     one is finished.  A segment that is not the whole of its unit leaves
//     O / l in fp32 and its LSE, folded by the combine kernel in CTA order:
//     no atomics.
//   - Within a segment the even key tiles go to accumulator 0 and the odd ones
//     to accumulator 1, each with its own running (m, l), so that two
//     softmax warpgroups work while the tensor core fills the other's scores;
//     the two states are merged once at the segment's end.
//
// Warps 0-3 and 4-7: softmax of the even and odd tiles, one row a thread (a
// warp whose 32 rows hold no token only keeps the barriers' count: a decode
// step fills a few rows of the 128); 8-11 rescale O; 12 and 14 TMA producers of
// Q and K, and of V (lane x loads box x of a tile, a box lying in one page);
// 13 MMA issue; 15 what masks leave.  Tensor memory: S0, S1 (P in 16 bits over
// them), O0, O1.
//
// Measured (bf16; GPU time of both kernels replayed as a graph; "of measured": of
// this GPU type's copy rate, 6.78 TB/s):
//   B64 H32 kv8 T1 ctx 4096 .. 8192 d128   258 to 267 us, 6.05 to 6.25 TB/s, 89 to
//     92 % of measured
//   B8 H32 kv8 T27 ctx 3000 .. 6000 d128 cap 30, pages of 32    58 us, 38 %:
//     the first scores come after 9 us (every CTA's 6 slots fill together), the
//     tiles at 5.3 TB/s after that, the last tile's softmax, the partial and the
//     join take 12
//   B2 H16 kv2 T64 ctx 50000 .. 100000 d64 fp16 slopes    85 us: 4 row tiles a
//     key head, bound by their softmax
//   B1 H32 kv8 T1 ctx 700 d128   12.5 us, latency
//   B300 H8 kv8 T1 ctx 300 d64  132 us: 8 us a unit of 3 tiles, the chain from
//     its scores to its output, which units of one CTA do not overlap
#pragma once

#include <climits>
#include <cmath>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mod_common.cuh"
#include "sm100_ptx.cuh"
#include "softmax_tile.cuh"
#include "tc_attn_mma.cuh"
#include "tree_internal.h"

namespace osattn {
namespace tree {

constexpr int BM = 128;
constexpr int BN = 128;
constexpr int kThreads = 512;
constexpr int kCorrWarp0 = 8, kProducerWarp = 12, kMmaWarp = 13, kProducerVWarp = 14;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol0 = 256;
constexpr float kLn2 = 0.6931471805599453f;
constexpr unsigned kBadArg = 1u;  // OSATTN_ERR_INVALID_ARG in the status word

enum : uint32_t {
  kSiteQ = 81,
  kSiteQEmpty = 82,
  kSiteK = 83,
  kSiteV = 84,
  kSiteKEmpty = 85,
  kSiteVEmpty = 86,
  kSiteS = 87,
  kSiteAlpha = 88,
  kSiteP = 89,
  kSiteO = 90,
  kSiteOEmpty = 91,
  kSiteMerge = 92,
  kSiteZero = 93,
  kSiteSeen = 94
};

template <int HD, int MODE>
struct Cfg {
  static constexpr int kTileBytes = BN * HD * 2;
  // slots of K tiles, and as many of V tiles; the slopes' operands take the
  // place of one K tile at d = 128 (at d = 64 there is room)
  static constexpr int kKSlots = HD == 128 ? (MODE == kModSlopes ? 2 : 3) : 6;
  static constexpr int kVSlots = HD == 128 ? 3 : 6;
  static constexpr int kTileRegion = (1 + kKSlots + kVSlots) * kTileBytes;
  // the key rows' operand, then the query rows' (the heads of a group differ)
  static constexpr int kTableBytes = MODE == kModSlopes ? 2 * kSlopeRowsBytes : 0;
};

// A share's next segment; every role walks the same ones.
struct Walk {
  int at, end;  // list positions
  int b, base;  // sequence and its first list position
  int ctx, first, n_b;
  // the segment
  int hk, rt, tile0, n;
  bool head_cut, tail_cut;  // misses the unit's first or last tiles
};

// The keys of a sequence that some draft sees: the context from `first` on
// (first = ctx: none of it) and the drafts whose bit is set.  Masks need not be
// trees: a draft may be on no line, or a window away from all that name it, and
// where no draft has depth 0 the window's first keys are nobody's.
constexpr int kSeenSlots = 4;  // segments that seen_role may be ahead
struct Seen {
  unsigned long long drafts;
  int first;
};

struct __align__(16) Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[6], k_empty[6], v_full[6], v_empty[6];
  uint64_t s_full[2];
  uint64_t alpha_full[2];  // 128 arrivals
  uint64_t p_full[2];      // 256 arrivals: softmax and correction
  uint64_t o_full;         // the segment's last product is done
  uint64_t o_empty;        // 256 arrivals: the accumulators have been read
  uint64_t merge;          // 256 arrivals: both states of the segment are stored
  uint64_t mma_drain;
  uint64_t seen_full[kSeenSlots], seen_empty[kSeenSlots];  // 1 and 128 arrivals a segment, if there are masks
  uint32_t tmem_base;
  int abort_flag;
  Seen seen[kSeenSlots];  // of the segment's sequence
  Walk start;  // of this CTA's share, before its first segment
  int warp_sum[16];
  // Within a segment alpha_bits of the accumulator's rows, [accumulator][row];
  // at its end the states m, l.
  union {
    uint16_t alpha[2][BM];
    float2 state[2][BM];
  };
  Walk walk[8];  // of the softmax warps: their registers hold the scores
};

template <int HD, int MODE>
constexpr int smem_bytes() {
  return Cfg<HD, MODE>::kTileRegion + Cfg<HD, MODE>::kTableBytes + static_cast<int>(sizeof(Bars));
}

struct Params {
  uint16_t* O;
  long long o_sb, o_sh, o_sn;
  float* LSE;  // [B, H, T]
  const int32_t* table;
  const int32_t* ctx;
  const long long* mask;  // [B, T] or null
  int B, H, Hkv, group, T;
  int tok_tile;   // tokens of a row tile: its rows are tok_tile * group <= 128
  int row_tiles;  // ceil(T / tok_tile)
  int max_pages, page, num_pages;
  int box_rows;   // keys of one TMA box: min(page, 128)
  int window;
  float scale, scale_log2;  // |scale|, |scale| * log2(e) (positive_scale)
  uint32_t neg_q;           // kIdescNegA if the scale is negative
  CapArgs cap;
  const float* slopes;
  float* o_part;    // [2 grid][slot_rows][d]
  float* lse_part;  // [2 grid][slot_rows]
  int slot_rows;    // tok_tile' * group, tok_tile' = min(T, tok_tile)
  int* head;        // [B + 1]: first list position of each sequence, and the list's length
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

// Cached keys of a sequence, kept within its page table.
__device__ __forceinline__ int ctx_of(const Params& p, int b) {
  const long long room = static_cast<long long>(p.max_pages) * p.page - p.T;
  const int c = __ldg(p.ctx + b);
  return c < 0 ? 0 : (c > room ? static_cast<int>(room) : c);
}
// First key that any draft can see, and the key tiles [first, first + n).
__device__ __forceinline__ int first_key(const Params& p, int ctx) {
  return p.window > 0 ? max(0, ctx - p.window + 1) : 0;
}
__device__ __forceinline__ void key_tiles(const Params& p, int ctx, int& first, int& n) {
  first = first_key(p, ctx) / BN;
  n = (ctx + p.T + BN - 1) / BN - first;  // T >= 1: at least one
}

__device__ __forceinline__ unsigned long long draft_bits(int T) {
  return T >= 64 ? ~0ull : (1ull << T) - 1;
}
// The drafts that draft t of sequence b sees.
__device__ __forceinline__ unsigned long long mask_of(const Params& p, int b, int t) {
  if (!p.mask) return t >= 63 ? ~0ull : (2ull << t) - 1;
  return static_cast<unsigned long long>(__ldg(p.mask + static_cast<long long>(b) * p.T + t)) &
         draft_bits(p.T);
}
// A draft's place behind the context (of a tree: how many other drafts lie on its
// line).  A draft with an empty mask, which others may see, has -1.
__device__ __forceinline__ int depth_of(unsigned long long mask) { return __popcll(mask) - 1; }

// The whole warp calls it.
__device__ __forceinline__ Seen seen_of(const Params& p, int b, int ctx) {
  const int lane = threadIdx.x & 31;
  unsigned long long m0 = lane < p.T ? mask_of(p, b, lane) : 0ull;
  unsigned long long m1 = lane + 32 < p.T ? mask_of(p, b, lane + 32) : 0ull;
  const int d0 = depth_of(m0), d1 = depth_of(m1);
  // (a draft that sees any draft sees the context)
  const int least = __reduce_min_sync(0xffffffffu, min(m0 ? d0 : INT_MAX, m1 ? d1 : INT_MAX));
  if (p.window > 0 && p.T >= p.window) {
#pragma unroll 1
    for (int u = 0; u < p.T; ++u) {
      const int d = __shfl_sync(0xffffffffu, u < 32 ? d0 : d1, u & 31);
      if (abs(d0 - d) >= p.window) m0 &= ~(1ull << u);
      if (abs(d1 - d) >= p.window) m1 &= ~(1ull << u);
    }
  }
  m0 |= m1;
  const unsigned lo = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(m0));
  const unsigned hi = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(m0 >> 32));
  Seen s;
  s.drafts = static_cast<unsigned long long>(hi) << 32 | lo;
  s.first = least == INT_MAX ? ctx : (p.window > 0 ? min(max(0, ctx + least - p.window + 1), ctx) : 0);
  return s;
}
__device__ __forceinline__ bool key_seen(const Seen& s, int ctx, int key) {
  const int u = key - ctx;
  return u < 0 ? key >= s.first : u < 64 && ((s.drafts >> u) & 1ull) != 0ull;
}
// Whether some draft sees one of the keys [key, key + n), n >= 1.
__device__ __forceinline__ bool any_seen(const Seen& s, int ctx, int key, int n) {
  if (key < ctx && s.first < ctx && key + n > s.first) return true;
  const int from = max(key - ctx, 0), to = min(key + n - ctx, 64);
  return from < to && ((s.drafts >> from) & (~0ull >> (64 - (to - from)))) != 0ull;
}

// Whether the slopes of a key head's query heads all go through the MMA step.
__device__ __forceinline__ bool slopes_linear(const Params& p, int hk) {
  bool ok = true;
  for (int g = 0; g < p.group; ++g) ok = ok && slope_linear(__ldg(p.slopes + hk * p.group + g), p.scale);
  return ok;
}

// Whether some draft does not see all keys of the tile from k0 on: it holds
// drafts or keys behind them, or keys before some draft's window.
__device__ __forceinline__ bool tile_masked(const Params& p, int ctx, int k0) {
  return k0 + BN > ctx || (p.window > 0 && k0 < ctx + p.T - p.window);
}

// Shares of a list of `total` key tiles: no share is empty.
__device__ __forceinline__ int shares(int total, int grid) { return total < grid ? total : grid; }

__device__ __forceinline__ bool walk_next(const Params& p, Walk& w) {
  if (w.at >= w.end) return false;
  const int units = p.Hkv * p.row_tiles;
  int in = w.at - w.base;
  if (in >= units * w.n_b) {
    w.base += units * w.n_b;
    ++w.b;
    w.ctx = ctx_of(p, w.b);
    key_tiles(p, w.ctx, w.first, w.n_b);
    in = w.at - w.base;
  }
  const int unit = in / w.n_b, tile = in - unit * w.n_b;
  w.hk = unit / p.row_tiles;
  w.rt = unit - w.hk * p.row_tiles;
  w.tile0 = w.first + tile;
  w.n = min(w.n_b - tile, w.end - w.at);
  w.head_cut = tile > 0;
  w.tail_cut = tile + w.n < w.n_b;
  w.at += w.n;
  return true;
}

// ------------------------------------------------------------------ softmax
template <int HD, bool kF16, int MODE>
__device__ __forceinline__ void softmax_role(const Params& p, Bars* bars, uint32_t tmem, int t,
                                             WaitCtl wc) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t s_addr = lane_base + static_cast<uint32_t>(t * BN);
  const int tl = row / p.group, g = row - tl * p.group;
  TileScore<kF16, MODE> ts;
  ts.c = p.scale_log2;
  ts.off = 0.f;
  ts.cap = &p.cap;
  uint32_t s_phase = 0, seg = 0;
  bool ok = true;
  Walk& at = bars->walk[warp];
  if (lane == 0) at = bars->start;
  __syncwarp();
  for (; ok; ++seg) {
    Walk w = at;
    const bool more = walk_next(p, w);
    __syncwarp();
    if (lane == 0) at = w;
    __syncwarp();
    if (!more) break;
    const int ctx = w.ctx, tile0 = w.tile0, n = w.n;
    const int tok = w.rt * p.tok_tile + tl;
    const bool live = tl < p.tok_tile && tok < p.T;
    const bool warp_live = __any_sync(0xffffffffu, live);
    // the drafts that the row sees: those of its line, without the ones that
    // are a window away
    auto row_mask = [&](int b) {
      unsigned long long mask = live ? mask_of(p, b, tok) : 0ull;
      if (p.window > 0 && p.T >= p.window) {  // (depths are -1 .. T - 1)
        const int depth = depth_of(mask);
        for (int u = 0; u < p.T; ++u)
          if (((mask >> u) & 1) && abs(depth - depth_of(mask_of(p, b, u))) >= p.window) mask &= ~(1ull << u);
      }
      return mask;
    };
    int depth = 0;
    bool sees = false;  // a padding token sees nothing: its row is zeroed at the end
    if (live) {
      const unsigned long long mask = mask_of(p, w.b, tok);
      sees = mask != 0ull;
      depth = depth_of(mask);
    }
    const int lo = p.window > 0 ? max(0, ctx + depth - p.window + 1) : 0;  // first key of the row's context
    [[maybe_unused]] bool linear = false;
    if constexpr (mode_slopes(MODE)) {
      const float slope = live ? __ldg(p.slopes + w.hk * p.group + g) : 0.f;
      ts.slope2 = slope * kModLog2e;
      linear = MODE == kModSlopes && slopes_linear(p, w.hk);
    }
    float m = -INFINITY, l = 0.f;
    // the last segment's states, where alpha goes now, have been read
    if (seg > 0) ok = __all_sync(0xffffffffu, mbar_wait(&bars->o_empty, (seg - 1) & 1u, wc, kSiteOEmpty));
    for (int i = t; ok && i < n; i += 2) {
      ok = mbar_wait(&bars->s_full[t], s_phase & 1u, wc, kSiteS);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ++s_phase;
      tc_fence_after_sync();
      auto publish = [&](uint16_t alpha) {
        bars->alpha[t][row] = alpha;
        mbar_arrive(&bars->alpha_full[t]);
      };
      if (!warp_live) {
        publish(0x3f80);  // 1: nothing to rescale
        tc_fence_before_sync();
        mbar_arrive(&bars->p_full[t]);
        continue;
      }
      const int k0 = (tile0 + i) * BN;
      const bool tail = k0 + BN > ctx;  // holds drafts or keys behind them
      const bool masked = tile_masked(p, ctx, k0);
      if constexpr (mode_slopes(MODE)) {
        // distances fall along the context; drafts are at the distance of
        // their depths
        ts.d0 = static_cast<float>(k0 - (ctx + depth));
        ts.both_sides = !linear || masked;
        ts.off = ts.both_sides ? 0.f : ts.slope2 * ts.d0;
      }
      // Tiles that every row sees, where one pass does; the others by the rolled loop.
      TileMask mk;
      bool done = false;
      if (!masked)
        done = ts.template tile<false, false, MODE != kModCapSlopes>(s_addr, mk, [](int) { return 0xffffffffu; },
                                                                     ts.by_place(), m, l, publish);
      if (!done) {
        const unsigned long long mask = tail ? row_mask(at.b) : 0ull;
        // visible keys of a chunk: context keys [lo, ctx), then the mask
        auto bits_of = [&](int ch) {
          const int c0 = k0 + 32 * ch;
          uint32_t bits = bit_range(lo - c0, sees ? ctx - c0 : 0);
          const int sh = ctx - c0;  // where draft 0 falls
          if (sh >= 0 && sh < 32) bits |= static_cast<uint32_t>(mask << sh);
          else if (sh < 0 && sh > -64) bits |= static_cast<uint32_t>(mask >> -sh);
          return bits;
        };
        mk.classify(bits_of);
        // lane x holds the depths of drafts x and 32 + x
        [[maybe_unused]] float dep0 = 0.f, dep1 = 0.f;
        if constexpr (mode_slopes(MODE)) {
          if (tail) {
            if (lane < p.T) dep0 = static_cast<float>(depth_of(mask_of(p, at.b, lane)));
            if (lane + 32 < p.T) dep1 = static_cast<float>(depth_of(mask_of(p, at.b, lane + 32)));
          }
        }
        // before the drafts by place; lane x fetches the depth of the draft in column x of the chunk
        auto gap = [&](int ch) {
          const int before = ctx - (k0 + 32 * ch), u = lane - before;
          const float a = __shfl_sync(0xffffffffu, dep0, u & 31), b = __shfl_sync(0xffffffffu, dep1, u & 31);
          const float draft = u < 32 ? a : b, own = static_cast<float>(depth), first = ts.d0 + static_cast<float>(32 * ch);
          return [=](int e) {
            const float at = __shfl_sync(0xffffffffu, draft, e) - own;
            return e < before ? first + static_cast<float>(e) : at;
          };
        };
        if (mode_cap(MODE) && p.cap.large)
          ts.template tile_rolled<true>(s_addr, mk, bits_of, gap, m, l, publish);
        else
          ts.template tile_rolled<false>(s_addr, mk, bits_of, gap, m, l, publish);
      }
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&bars->p_full[t]);
    }
    if (!ok) break;
    // ---- merge the two states; warpgroup t finishes columns t d/2 .. of both
    // (every alpha of the segment has been used: its products are done)
    ok = mbar_wait(&bars->o_full, seg & 1u, wc, kSiteO);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    bars->state[t][row] = make_float2(m, l);
    mbar_arrive(&bars->merge);
    ok = mbar_wait(&bars->merge, seg & 1u, wc, kSiteMerge);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    tc_fence_after_sync();
    const float2 s0 = bars->state[0][row], s1 = bars->state[1][row];
    const float M = fmaxf(s0.x, s1.x);
    const float f0 = s0.x == -INFINITY ? 0.f : ex2_approx(s0.x - M);
    const float f1 = s1.x == -INFINITY ? 0.f : ex2_approx(s1.x - M);
    const float L = fmaf(s0.y, f0, s1.y * f1);
    const bool empty = L == 0.f || !sees;
    const float inv = empty ? 0.f : 1.f / L;
    const float g0 = f0 * inv, g1 = f1 * inv;
    const bool head_cut = at.head_cut, whole = !head_cut && !at.tail_cut;
    const int b = at.b, h = at.hk * p.group + g;
    const int slot = 2 * static_cast<int>(blockIdx.x) + (head_cut ? 0 : 1);
    constexpr int kHalf = HD / 2;
    const uint32_t o_addr = lane_base + kOCol0 + static_cast<uint32_t>(t * kHalf);
    uint16_t* orow = p.O + b * p.o_sb + h * p.o_sh + tok * p.o_sn + t * kHalf;
    const long long prow = static_cast<long long>(slot) * p.slot_rows + row;
    float* part = p.o_part + prow * HD + t * kHalf;
#pragma unroll
    for (int ch = 0; ch < kHalf / 32; ++ch) {
      if (!warp_live) break;
      uint32_t a0[32], a1[32];
      tmem_ld_32x32b_x32(o_addr + ch * 32, a0);
      if (n > 1) tmem_ld_32x32b_x32(o_addr + HD + ch * 32, a1);
      tmem_ld_wait();
      reg_fence32(a0);
      reg_fence32(a1);
      float o[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        o[e] = __uint_as_float(a0[e]) * g0;
        if (n > 1) o[e] = fmaf(__uint_as_float(a1[e]), g1, o[e]);
        if (empty) o[e] = 0.f;
      }
      if (live) {
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(orow + ch * 32);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            dst[e] = make_uint4(pack2<kF16>(o[8 * e], o[8 * e + 1]), pack2<kF16>(o[8 * e + 2], o[8 * e + 3]),
                                pack2<kF16>(o[8 * e + 4], o[8 * e + 5]), pack2<kF16>(o[8 * e + 6], o[8 * e + 7]));
        } else {
          float4* dst = reinterpret_cast<float4*>(part + ch * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
    }
    tc_fence_before_sync();
    mbar_arrive(&bars->o_empty);
    if (live && t == 0) {
      const float lse = empty ? -INFINITY : (M + log2f(L)) * kLn2;
      if (whole)
        p.LSE[(static_cast<long long>(b) * p.H + h) * p.T + tok] = lse;
      else
        p.lse_part[prow] = lse;
    }
  }
}

// ------------------------------------------------------------------ correction
template <int HD, int MODE>
__device__ __forceinline__ void correction_role(const Params& p, Bars* bars, uint8_t* sV, uint32_t tmem,
                                                WaitCtl wc) {
  using C = Cfg<HD, MODE>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  uint32_t a_phase[2] = {0, 0}, vc = 0, seg = 0;  // vc: V tiles so far
  bool ok = true;
  for (Walk w = bars->start; ok && walk_next(p, w); ++seg) {
    // The rows of V of keys that no draft sees are zeroed below.
    for (int i = 0; ok && i < w.n; ++i, ++vc) {
      const int t = i & 1;
      const int k0 = (w.tile0 + i) * BN;
      const int lo = first_key(p, w.ctx);
      if (k0 < lo || k0 + BN > w.ctx || (p.mask && tile_masked(p, w.ctx, k0))) {
        ok = mbar_wait(&bars->v_full[vc % C::kVSlots], (vc / C::kVSlots) & 1u, wc, kSiteZero);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // (a chain's drafts see themselves, and the first has depth 0)
        bool hidden = k0 + row < lo || k0 + row >= w.ctx + p.T;
        if (p.mask) {
          ok = warp_wait(&bars->seen_full[seg % kSeenSlots], seg / kSeenSlots & 1u, wc, kSiteSeen);
          if (!ok) break;
          hidden = !key_seen(bars->seen[seg % kSeenSlots], w.ctx, k0 + row);
        }
        if (hidden) {
          uint8_t* v = sV + (vc % C::kVSlots) * C::kTileBytes + row * 128;
#pragma unroll
          for (int cb = 0; cb < HD / 64; ++cb)
#pragma unroll
            for (int x = 0; x < 8; ++x)
              *reinterpret_cast<uint4*>(v + cb * BN * 128 + x * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async();
      }
      ok = mbar_wait(&bars->alpha_full[t], a_phase[t] & 1u, wc, kSiteAlpha);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ++a_phase[t];
      const float alpha = alpha_of(bars->alpha[t][row]);
      // the accumulator's earlier products are done: S_t of this tile was
      // issued after them
      if (i >= 2 && __any_sync(0xffffffffu, alpha != 1.f)) {
        tc_fence_after_sync();
        const uint64_t a2 = f2_pack(alpha, alpha);
        const uint32_t o_addr = lane_base + kOCol0 + static_cast<uint32_t>(t * HD);
#pragma unroll
        for (int ch = 0; ch < HD / 32; ++ch) {
          uint32_t orr[32];
          tmem_ld_32x32b_x32(o_addr + ch * 32, orr);
          tmem_ld_wait();
          reg_fence32(orr);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float b0, b1;
            f2_unpack(f2_mul(f2_pack(__uint_as_float(orr[2 * e]), __uint_as_float(orr[2 * e + 1])), a2), b0, b1);
            orr[2 * e] = __float_as_uint(b0);
            orr[2 * e + 1] = __float_as_uint(b1);
          }
          tmem_st_32x32b_x32(o_addr + ch * 32, orr);
        }
        tmem_st_wait();
      }
      tc_fence_before_sync();
      mbar_arrive(&bars->p_full[t]);
    }
    if (p.mask && ok) {  // (waited for in every segment: the phases stay in step)
      ok = warp_wait(&bars->seen_full[seg % kSeenSlots], seg / kSeenSlots & 1u, wc, kSiteSeen);
      mbar_arrive(&bars->seen_empty[seg % kSeenSlots]);
    }
  }
}

// One warp, where there are masks: what the drafts of each segment's sequence see,
// and the status for pages that do not exist but hold a key that some draft sees.
// A warp of its own, some segments ahead: in the producers or the correction warps
// this costs registers and code (one token over 700 keys, without masks, 12.5 ->
// 13.2 us), and waiting for each segment's end it takes issue slots from the
// softmax (8 trees of 27 drafts over 6000 keys 57.6 -> 60.4 us).
__device__ __forceinline__ void seen_role(const Params& p, Bars* bars, WaitCtl wc) {
  if (!p.mask) return;
  const int lane = threadIdx.x & 31;
  uint32_t seg = 0;
  bool ok = true;
  for (Walk w = bars->start; ok && walk_next(p, w); ++seg) {
    const Seen s = seen_of(p, w.b, w.ctx);
    const uint32_t slot = seg % kSeenSlots;
    if (seg >= kSeenSlots) ok = warp_wait(&bars->seen_empty[slot], (seg / kSeenSlots - 1) & 1u, wc, kSiteSeen);
    if (!ok) break;
    if (lane == 0) {
      bars->seen[slot] = s;
      mbar_arrive(&bars->seen_full[slot]);
    }
    __syncwarp();
    const int last = min((w.tile0 + w.n) * BN, w.ctx + p.T) - 1;
    for (int at = w.tile0 * BN / p.page + lane; at <= last / p.page; at += 32)
      if (any_seen(s, w.ctx, at * p.page, p.page)) {
        const int page = __ldg(p.table + static_cast<long long>(w.b) * p.max_pages + at);
        if (page < 0 || page >= p.num_pages) atomicMax(p.status, kBadArg);
      }
    __syncwarp();
  }
}

// ------------------------------------------------------------------ producers
// One warp loads Q and K, another V; lane x loads box x of each tile.  A box
// before every window or behind the drafts, or whose page number is not one of
// the pool's, is read from behind the pool, which fills it with zeros; the latter
// also sets the status (with masks seen_role does, which knows what they leave).
template <int HD, bool kF16, int MODE, bool kV>
__device__ __forceinline__ void producer_role(const CUtensorMap* tmQ, const CUtensorMap* tmKV, const Params& p,
                                              Bars* bars, uint8_t* sQ, uint8_t* ring, uint8_t* slopes,
                                              WaitCtl wc) {
  using C = Cfg<HD, MODE>;
  constexpr int kSlots = kV ? C::kVSlots : C::kKSlots;
  uint64_t* const full = kV ? bars->v_full : bars->k_full;
  uint64_t* const empty = kV ? bars->v_empty : bars->k_empty;
  const int lane = threadIdx.x & 31;
  const int boxes = BN / p.box_rows;
  const uint32_t q_bytes = static_cast<uint32_t>(p.tok_tile * p.group * HD * 2);
  uint32_t n = 0, seg = 0;  // tiles and segments so far
  bool ok = true;
  for (Walk w = bars->start; ok && walk_next(p, w); ++seg) {
    if constexpr (!kV) {
      if (seg > 0) {
        ok = warp_wait(&bars->q_empty, (seg - 1) & 1u, wc, kSiteQEmpty);
        if (!ok) break;
      }
      if constexpr (MODE == kModSlopes) {
        if (slopes_linear(p, w.hk)) {
          for (int row = lane; row < 128; row += 32) {
            const int tl = row / p.group, tok = w.rt * p.tok_tile + tl;
            const bool live = tl < p.tok_tile && tok < p.T;
            const float slope = live ? __ldg(p.slopes + w.hk * p.group + row - tl * p.group) : 0.f;
            slope_fill_q<kF16>(slopes + kSlopeRowsBytes, row, slope, p.scale);
          }
          fence_proxy_async();
        }
        __syncwarp();
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full, q_bytes);
#pragma unroll
        for (int cb = 0; cb < HD / 64; ++cb)
          tma_load_4d(sQ + cb * BM * 128, tmQ, &bars->q_full, cb * 64, w.hk * p.group, w.rt * p.tok_tile, w.b);
      }
    }
    const int lo = first_key(p, w.ctx), end = w.ctx + p.T;
    for (int i = 0; ok && i < w.n; ++i) {
      const int s = static_cast<int>(n % kSlots);
      const uint32_t use = n / kSlots;
      const int key = (w.tile0 + i) * BN + lane * p.box_rows;
      int page = p.num_pages, in_page = 0;
      if (lane < boxes && key < end && key + p.box_rows > lo) {
        const int at = key / p.page;  // < max_pages: ctx + T fits the table
        in_page = key - at * p.page;
        page = __ldg(p.table + static_cast<long long>(w.b) * p.max_pages + at);
        if (page < 0 || page >= p.num_pages) {
          page = p.num_pages;
          if (!p.mask) atomicMax(p.status, kBadArg);
        }
      }
      if (use > 0) ok = warp_wait(&empty[s], (use - 1) & 1u, wc, kV ? kSiteVEmpty : kSiteKEmpty);
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], C::kTileBytes);
      __syncwarp();
      if (lane < boxes)
#pragma unroll
        for (int cb = 0; cb < HD / 64; ++cb)
          tma_load_4d(ring + s * C::kTileBytes + cb * BN * 128 + lane * p.box_rows * 128, tmKV, &full[s],
                      cb * 64, in_page, w.hk, page);
      ++n;
    }
    if (!ok) {
      ++seg;  // its Q is in flight
      break;
    }
  }
  // Let every load of this warp land before the CTA can exit.
  if (lane == 0) {
    if (!kV && seg > 0) drain_wait(&bars->q_full, (seg - 1) & 1u, wc.limit_ns);
    for (uint32_t x = (n > kSlots ? n - kSlots : 0); x < n; ++x)
      drain_wait(&full[x % kSlots], (x / kSlots) & 1u, wc.limit_ns);
  }
  __syncwarp();
}

// ------------------------------------------------------------------ MMA issuer
template <int HD, bool kF16, int MODE>
__device__ __forceinline__ void mma_role(const Params& p, Bars* bars, uint32_t tmem, uint8_t* sQ,
                                         uint8_t* sK, uint8_t* sV, uint8_t* slopes, WaitCtl wc) {
  using C = Cfg<HD, MODE>;
  const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
  const uint64_t k_desc = sdesc_sw128(smem_u32(sK), 16, 1024);        // slot 0, K-major
  const uint64_t v_desc = sdesc_sw128(smem_u32(sV), BN * 128, 1024);  // slot 0, MN-major
  constexpr uint64_t kStep = static_cast<uint64_t>(C::kTileBytes >> 4);
  const uint32_t s_id = idesc_f16_f32(128, 128, 0, kF16) | p.neg_q;
  uint32_t kc = 0, vc = 0, seg = 0, p_phase[2] = {0, 0};
  bool ok = true;
  for (Walk w = bars->start; ok && walk_next(p, w); ++seg) {
    [[maybe_unused]] const bool linear = MODE == kModSlopes && slopes_linear(p, w.hk);
    ok = warp_wait(&bars->q_full, seg & 1u, wc, kSiteQ);
    if (!ok) break;
    // scores of tile i into buffer i mod 2
    auto scores = [&](int i) {
      const uint32_t s = kc % C::kKSlots;
      if (!warp_wait(&bars->k_full[s], (kc / C::kKSlots) & 1u, wc, kSiteK)) return false;
      tc_fence_after_sync();
      mma_abt_id<HD>(tmem + (i & 1) * BN, q_desc, k_desc + s * kStep, s_id);
      if constexpr (MODE == kModSlopes) {
        if (linear && !tile_masked(p, w.ctx, (w.tile0 + i) * BN))
          mma_ss_k<1, true>(tmem + (i & 1) * BN, slope_rows_desc(smem_u32(slopes) + kSlopeRowsBytes),
                            slope_rows_desc(smem_u32(slopes)), idesc_f16_f32(128, 128, 0, kF16));
      }
      mma_commit<true>(&bars->s_full[i & 1]);
      mma_commit<true>(&bars->k_empty[s]);
      if (i == w.n - 1) mma_commit<true>(&bars->q_empty);
      ++kc;
      return true;
    };
    ok = scores(0);
    if (ok && w.n > 1) ok = scores(1);
    for (int i = 0; ok && i < w.n; ++i) {
      const int t = i & 1;
      ok = warp_wait(&bars->p_full[t], p_phase[t] & 1u, wc, kSiteP);
      if (!ok) break;
      ++p_phase[t];
      if (i == 0 && seg > 0) {
        ok = warp_wait(&bars->o_empty, (seg - 1) & 1u, wc, kSiteOEmpty);
        if (!ok) break;
      }
      const uint32_t s = vc % C::kVSlots;
      ok = warp_wait(&bars->v_full[s], (vc / C::kVSlots) & 1u, wc, kSiteV);
      if (!ok) break;
      tc_fence_after_sync();
      mma_tmem_a_128<HD, kF16, true>(tmem + kOCol0 + t * HD, tmem + t * BN, v_desc + s * kStep, i >= 2);
      mma_commit<true>(&bars->v_empty[s]);
      ++vc;
      if (i == w.n - 1) mma_commit<true>(&bars->o_full);
      if (i + 2 < w.n) ok = scores(i + 2);
    }
  }
  mma_commit<true>(&bars->mma_drain);
  drain_wait(&bars->mma_drain, 0, wc.limit_ns);
  __syncwarp();
}

// Where this CTA's share starts in the list; CTA 0 also writes every sequence's
// first position, and the list's length, for the combine kernel.
__device__ __forceinline__ void find_start(const Params& p, Bars* bars) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = p.Hkv * p.row_tiles;
  // This thread's sequence of a block of kThreads of them, and the scan of
  // the block's tiles: position of the sequence's first, and the block's sum.
  int ctx = 0, first = 0, n_b = 0, base = 0;
  auto scan_block = [&](int b0, int before) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    n_b = 0;
    if (b < p.B) {
      ctx = ctx_of(p, b);
      key_tiles(p, ctx, first, n_b);
    }
    const int mine = n_b * units;
    int scan = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, scan, off);
      if (lane >= off) scan += y;
    }
    if (lane == 31) bars->warp_sum[warp] = scan;
    __syncthreads();
    int all = 0;
    base = before + scan - mine;
    for (int x = 0; x < kThreads / 32; ++x) {
      const int y = bars->warp_sum[x];
      if (x < warp) base += y;
      all += y;
    }
    __syncthreads();
    return all;
  };
  int total = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) total += scan_block(b0, total);
  const int G = shares(total, gridDim.x), c = blockIdx.x;
  const int at = c < G ? static_cast<int>(static_cast<long long>(c) * total / G) : 0;
  const int end = c < G ? static_cast<int>((c + 1ll) * total / G) : 0;
  if (threadIdx.x == 0) {
    bars->start.at = at;
    bars->start.end = end;
  }
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    if (p.B > kThreads) before += scan_block(b0, before);  // else the scan at hand
    const int b = b0 + static_cast<int>(threadIdx.x);
    if (b < p.B) {
      if (at >= base && at < base + n_b * units) {
        bars->start.b = b;
        bars->start.base = base;
        bars->start.ctx = ctx;
        bars->start.first = first;
        bars->start.n_b = n_b;
      }
      if (blockIdx.x == 0) {
        p.head[b] = base;
        if (__ldg(p.ctx + b) != ctx) atomicMax(p.status, kBadArg);
      }
    }
  }
  if (threadIdx.x == 0 && blockIdx.x == 0) p.head[p.B] = total;
}

template <int HD, bool kF16, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const Params p) {
  using C = Cfg<HD, MODE>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // see fwd_mod_kernel
    if (threadIdx.x == 0) atomicExch(p.status, 3u /* OSATTN_ERR_CUDA */);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kTileBytes;
  uint8_t* sV = sK + C::kKSlots * C::kTileBytes;
  uint8_t* slopes = smem + C::kTileRegion;
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kTileRegion + C::kTableBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < C::kKSlots; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < C::kVSlots; ++s) {
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->alpha_full[t], 128);
      mbar_init(&bars->p_full[t], 256);
    }
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->o_empty, 256);
    mbar_init(&bars->merge, 256);
    mbar_init(&bars->mma_drain, 1);
    for (int s = 0; s < kSeenSlots; ++s) {
      mbar_init(&bars->seen_full[s], 1);
      mbar_init(&bars->seen_empty[s], 128);
    }
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
  // rows of Q that no load writes stay zero
  if (p.tok_tile * p.group < BM)
    for (int x = threadIdx.x; x < C::kTileBytes / 16; x += kThreads)
      reinterpret_cast<uint4*>(sQ)[x] = make_uint4(0u, 0u, 0u, 0u);
  if constexpr (MODE == kModSlopes) {
    if (threadIdx.x < BN) slope_fill_k<kF16>(slopes, threadIdx.x);
  }
  fence_proxy_async();
  __syncthreads();
  find_start(p, bars);
  // the combine kernel may take its place (it waits for this one to end)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{&bars->abort_flag, p.status, p.status + 1, p.wait_limit_ns};

  // 256 x 184 + 128 x 88 + 128 x 56 = 512 x 128 registers
  if (warp < kCorrWarp0) {
    regs_inc<184>();
    softmax_role<HD, kF16, MODE>(p, bars, tmem, warp >> 2, wc);
  } else if (warp < kProducerWarp) {
    regs_dec<88>();
    correction_role<HD, MODE>(p, bars, sV, tmem, wc);
  } else {
    regs_dec<56>();
    if (warp == kProducerWarp)
      producer_role<HD, kF16, MODE, false>(&tmQ, &tmK, p, bars, sQ, sK, slopes, wc);
    else if (warp == kProducerVWarp)
      producer_role<HD, kF16, MODE, true>(&tmQ, &tmV, p, bars, sQ, sV, slopes, wc);
    else if (warp == kMmaWarp)
      mma_role<HD, kF16, MODE>(p, bars, tmem, sQ, sK, sV, slopes, wc);
    else
      seen_role(p, bars, wc);
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

// ------------------------------------------------------------------ combine
// One warp a row joins the partials of the CTAs that share the row's unit, in
// CTA order; with many partials a unit, kWays warps (8, not 1) take every
// kWays-th of them and are joined in order too.  Rows of units that one CTA did
// whole are done already.  Runs as a dependent launch: resident before the
// main kernel ends where there is room, waiting for it in griddepcontrol.wait.
template <int HD, bool kF16, int kWays>
__global__ void __launch_bounds__(256) tree_combine_kernel(const Params p, int grid) {
  constexpr int CPL = HD / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_unit = (p.slot_rows * kWays + 7) / 8;
  const int unit_all = blockIdx.x / per_unit;
  const int row = kWays == 1 ? (blockIdx.x - unit_all * per_unit) * 8 + warp : blockIdx.x - unit_all * per_unit;
  const int way = kWays == 1 ? 0 : warp;
  const int units = p.Hkv * p.row_tiles;
  const int b = unit_all / units, unit = unit_all - b * units;
  const int hk = unit / p.row_tiles, rt = unit - hk * p.row_tiles;
  const int tl = row / p.group, g = row - tl * p.group;
  const int tok = rt * p.tok_tile + tl;
  if (row >= p.slot_rows || tl >= p.tok_tile || tok >= p.T) return;  // (the whole block if kWays > 1)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int base = p.head[b], n_b = (p.head[b + 1] - base) / units;
  const long long total = p.head[p.B], G = shares(p.head[p.B], grid);
  const long long x0 = base + static_cast<long long>(unit) * n_b, x1 = x0 + n_b - 1;
  // the share that holds list position x: the largest c with c total / G <= x
  const int c0 = static_cast<int>(((x0 + 1) * G - 1) / total), c1 = static_cast<int>(((x1 + 1) * G - 1) / total);
  if (c0 == c1) return;
  // a partial is the state (m, l) = (lse, 1) carrying O / l
  auto row_of = [&](int c) { return static_cast<long long>(2 * c + (c == c0 ? 1 : 0)) * p.slot_rows + row; };
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
  const int h = hk * p.group + g;
  uint16_t* dst = p.O + b * p.o_sb + h * p.o_sh + tok * p.o_sn + lane * CPL;
#pragma unroll
  for (int k = 0; k < CPL; k += 2)
    *reinterpret_cast<uint32_t*>(dst + k) = pack2<kF16>(acc[k] * inv, acc[k + 1] * inv);
  if (lane == 0) p.LSE[(static_cast<long long>(b) * p.H + h) * p.T + tok] = l == 0.f ? -INFINITY : top + logf(l);
}

// ------------------------------------------------------------------ host
constexpr int kLaunchRegs = 128;  // the setmaxnreg split above assumes it

template <int HD, bool kF16, int MODE>
cudaError_t set_attrs() {
  static_assert(smem_bytes<HD, MODE>() <= 232448, "shared memory per CTA");
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, tree_kernel<HD, kF16, MODE>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(tree_kernel<HD, kF16, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              smem_bytes<HD, MODE>());
}

template <int HD, bool kF16>
cudaError_t prepare() {
  cudaError_t e;
  if ((e = set_attrs<HD, kF16, kModPlain>()) != cudaSuccess) return e;
  if ((e = set_attrs<HD, kF16, kModCap>()) != cudaSuccess) return e;
  if ((e = set_attrs<HD, kF16, kModSlopes>()) != cudaSuccess) return e;
  return set_attrs<HD, kF16, kModCapSlopes>();
}

template <int HD, bool kF16, int MODE>
cudaError_t launch_mode(int grid, cudaStream_t s, const CUtensorMap& q, const CUtensorMap& k,
                        const CUtensorMap& v, const Params& p) {
  tree_kernel<HD, kF16, MODE><<<grid, kThreads, smem_bytes<HD, MODE>(), s>>>(q, k, v, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>(p.B) * p.Hkv * p.row_tiles;
  // 16 or more partials a unit, if the units are about alike: 8 warps a row (19 partials, H32 kv8 ctx
  // 32000: 34.5 us against 36.6 with one warp; at 9.5, B2 H16 kv2 T64 d64: 67.4 against 65.6)
  const int ways = grid >= 16 * units ? 8 : 1;
  const long long blocks = units * ((static_cast<long long>(p.slot_rows) * ways + 7) / 8);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute dep;
  dep.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  dep.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &dep;
  cfg.numAttrs = 1;
  return ways == 1 ? cudaLaunchKernelEx(&cfg, tree_combine_kernel<HD, kF16, 1>, p, grid)
                   : cudaLaunchKernelEx(&cfg, tree_combine_kernel<HD, kF16, 8>, p, grid);
}

template <int HD, bool kF16>
cudaError_t launch(const TreeArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v) {
  Params p;
  p.O = static_cast<uint16_t*>(a.O);
  p.o_sb = a.o_s[0];
  p.o_sh = a.o_s[1];
  p.o_sn = a.o_s[2];
  p.LSE = a.LSE;
  p.table = a.table;
  p.ctx = a.ctx;
  p.mask = reinterpret_cast<const long long*>(a.mask);
  p.B = a.B;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.group = a.H / a.Hkv;
  p.T = a.T;
  p.tok_tile = tree_tok_tile(p.group);
  p.row_tiles = (a.T + p.tok_tile - 1) / p.tok_tile;
  p.max_pages = a.max_pages;
  p.page = a.page;
  p.num_pages = a.num_pages;
  p.box_rows = a.page < BN ? a.page : BN;
  p.window = a.window;
  p.scale = positive_scale(a.scale);
  p.scale_log2 = p.scale * kModLog2e;
  p.neg_q = a.scale < 0.f ? kIdescNegA : 0u;
  p.cap = make_cap(p.scale, a.softcap, kF16);
  p.slopes = a.slopes;
  p.slot_rows = tree_slot_rows(p.group, a.T);
  const int grid = a.num_sms < kTreeMaxCtas ? a.num_sms : kTreeMaxCtas;
  p.head = static_cast<int*>(a.workspace);
  p.o_part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + tree_head_bytes(a.B));
  p.lse_part = p.o_part + static_cast<long long>(2) * kTreeMaxCtas * p.slot_rows * HD;
  p.status = a.status;
  p.wait_limit_ns = a.wait_limit_ns;
  if (a.slopes)
    return a.softcap > 0.f ? launch_mode<HD, kF16, kModCapSlopes>(grid, a.stream, q, k, v, p)
                           : launch_mode<HD, kF16, kModSlopes>(grid, a.stream, q, k, v, p);
  return a.softcap > 0.f ? launch_mode<HD, kF16, kModCap>(grid, a.stream, q, k, v, p)
                         : launch_mode<HD, kF16, kModPlain>(grid, a.stream, q, k, v, p);
}

}  // namespace tree
}  // namespace osattn
