// tree_e4m3_wide.cuh - the second form of attention of drafted tokens over e4m3
// pages, for more than 16 query rows a key head: the rows are the 128 rows of the
// products, as over 16-bit pages, and a thread of the softmax has one row.
//   S = Q K^T  [rows x 128 keys]   A: the rows' terms in shared memory, B: the K tile
//   O += P V   [rows x d]          A: the weights' terms in tensor memory, B: the V tile
//                                  read along its rows
// What a row knows (its factor, m, slope, depth) is in registers here, where the first
// form, with a key a thread, reads all rows' from shared memory; a scale covers 8 keys or
// more (otherwise the first form is taken), so a thread needs three values for 8 scores.
//
// Precision.  The terms of one operand go into one accumulator as they are:
//   q 2^k = q0 in e4m3 + q1 (+ q2 for fp16) in e5m2, 2^k bringing a row to [128, 256):
//     with the remainders' signs 4 + 4 (+ 3) bits, so elements down to 2^-13 of the
//     row's greatest are exact, smaller ones to 2^-21 of it
//   w = p s_v in fp16, as three e5m2 terms of one sum: to half of e5m2's least step, 2^-27 of
//     the row's greatest weight (the first form, with an accumulator a term, goes to 2^-34)
//
// What bounds it: the softmax (half of the issue slots, most of the rest of its time waiting
// for what it has issued), and behind it the chain from one tile's weights over 18 to 24
// products (12 of P V, for the three terms) to the next scores of its warpgroup.  The pass
// over a tile is a loop of 32 keys: unrolled over all 128, with m decided from weights at
// hand, it waited for instructions (B2 T64 below: 177 us).
// Measured (GPU time of both kernels replayed as a graph):
//   B8 H32 kv8 T27 ctx 3000 .. 6000 d128 cap 30 bf16, blocks of 32  60 to 62 us (16-bit
//     pages: 58)
//   B2 H16 kv2 T64 ctx 50000 .. 100000 d64 fp16 slopes  115 us, 2600 cycles a tile (16-bit
//     pages: 85 us): who drafts wide trees over long contexts keeps 16-bit pages
//   B8 H32 kv8 ctx 6000 d128 bf16  20 rows 47 us, 64 rows 50 us, 128 rows 60 us
//   B64 H32 kv8 ctx 4000 d128 bf16  20 rows 176 us, 64 rows 184 us, 128 rows 207 us
//
// Warps 0-3 and 4-7: softmax of the even and odd tiles; 8 and 9: TMA loads; 10: scales;
// 11: the products; 12-15: the queries' terms, and what is to be known of a tile's keys
// before its softmax.
#pragma once

#include "softmax_tile.cuh"
#include "tree_e4m3_tcgen05.cuh"

namespace osattn {
namespace tree8 {
namespace wide {

constexpr int kRows = 128;
constexpr int kWarpScale = 10, kWarpMma = 11, kWarpPrepare = 12;
constexpr int kChunk = 8, kChunks = BN / kChunk;  // keys that share a scale
constexpr int kRaw = 0, kNear = 1, kFar = 2;       // forms of exponents: see cap_scores

struct Params : tree8::Params {
  static constexpr bool kLeads = true;
  int lead;
};

enum : uint32_t { kSiteReady = 121, kSitePrepare = 122 };

// What the 8 keys of a chunk share.
struct __align__(16) Chunk {
  float ks, lv, inv;  // K's scale, log2 of V's and kSumUnit over it
};

struct __align__(16) Shared {
  uint64_t q_full, q_empty;  // 128 and 257 arrivals
  uint64_t k_full[6], v_full[6], scale_full[6], ready[6], empty[6];  // 1, 1, 64, 128, 1 arrivals
  uint64_t s_full[2];
  uint64_t p_full[2];  // 128 arrivals
  uint64_t o_full;     // the segment's last product is done
  uint64_t o_empty;    // 256 arrivals: the accumulators have been read
  uint64_t merge;      // 256 arrivals: both states of the segment are stored
  uint64_t joined;     // 128 arrivals: the warps' parts of what the rows see are there
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  Walk start;
  Walk walk[8];  // of the softmax warps: their registers hold the weights
  int warp_sum[kThreads / 32];
  unsigned long long see[2][4];  // [segment parity][warp]: drafts that a row of the warp sees
  int lo[2][4];                  // and the first key of the context
  float fac[kRows];              // scale log2(e) 2^-k, 0 for no row, NaN for a row that is not finite
  float k_scale[6][kChunks], v_scale[6][kChunks];
  Chunk chunk[6][kChunks];
  float2 bound[6][BN / 32];  // of 32 keys: the greatest |ks|, the greatest lv
  float before[6][BN];     // slopes, masked tiles: places from the key to the context's end
  float2 state[2][kRows];  // m, l
};

template <int HD, bool kF16>
struct Mem {
  static constexpr int kTerms = kF16 ? 3 : 2;
  static constexpr int kTileBytes = BN * HD;
  static constexpr int kQBytes = kTerms * kRows * HD;
  static constexpr int kFixed = kQBytes + static_cast<int>(sizeof(Shared));
  static constexpr int kFit = (232448 - kFixed) / (2 * kTileBytes);
  static constexpr int kSlots = kFit < 6 ? kFit : 6;  // of K tiles, and as many of V tiles
  static constexpr int kRing = 2 * kSlots * kTileBytes;
  static constexpr int kBytes = kRing + kFixed;
  static_assert(kSlots >= 4, "tiles in flight");
};

// The drafts that the row sees: those of its line, without the ones a window away.
__device__ __forceinline__ unsigned long long in_window(const Params& p, int b, unsigned long long mask) {
  if (mask != 0ull && p.window > 0 && p.T >= p.window) {  // (depths are -1 .. T - 1)
    const int depth = tree::depth_of(mask);
    for (int u = 0; u < p.T; ++u)
      if (((mask >> u) & 1ull) && abs(depth - tree::depth_of(tree::mask_of(p, b, u))) >= p.window) mask &= ~(1ull << u);
  }
  return mask;
}

// Bits [from, to) of 32.
__device__ __forceinline__ uint32_t bits_between(int from, int to) {
  from = max(from, 0);
  to = min(to, 32);
  return from < to ? (0xffffffffu >> (32 - (to - from))) << from : 0u;
}

// ------------------------------------------------------------------ softmax
template <int HD, bool kF16, int MODE>
__device__ __forceinline__ void softmax_role(const Params& p, Shared* sh, uint32_t tmem, int t, WaitCtl wc) {
  constexpr int kSlots = Mem<HD, kF16>::kSlots;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3, row = quarter * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
  const uint32_t s_addr = lane_base + static_cast<uint32_t>(t * 128);
  const uint32_t o_addr = lane_base + kOCol0 + static_cast<uint32_t>(t * 128);
  uint32_t cnt = 0, seg = 0, tiles = 0;
  bool ok = true;
  Walk& at = sh->walk[warp];
  if (lane == 0) at = sh->start;
  __syncwarp();
  for (; ok; ++seg) {
    Walk w = at;
    const bool more = next_segment(p, w);
    __syncwarp();
    if (lane == 0) at = w;
    __syncwarp();
    if (!more) break;
    const int ctx = w.ctx, n_tiles = w.n, last = w.tile0 + w.n - 1;  // tile i is key tile last - i
    const int row0 = w.rt * p.tile_rows, count = min(p.tile_rows, p.rows - row0);
    const bool live = row < count;
    const bool warp_live = quarter * 32 < count;
    const int tok = (row0 + (live ? row : 0)) / p.group, h = w.hk * p.group + row0 + (live ? row : 0) - tok * p.group;
    const unsigned long long own = live ? tree::mask_of(p, w.b, tok) : 0ull;
    const bool sees = own != 0ull;
    const int depth = tree::depth_of(own);
    const int lo = p.window > 0 ? max(0, ctx + depth - p.window + 1) : 0;  // first key of the row's context
    [[maybe_unused]] float fall = 0.f;
    [[maybe_unused]] uint64_t fall_e[4];  // what the places of a chunk's keys add to it
    if constexpr (mode_slopes(MODE)) {
      fall = live ? -__ldg(p.slopes + h) * kLog2e : 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) fall_e[e] = f2_pack(-2.f * e * fall, -(2.f * e + 1.f) * fall);
    }
    ok = warp_wait_idle(&sh->q_full, seg & 1u, wc, kSiteQ);
    if (!ok) break;
    const float fac = sh->fac[row];
    mbar_arrive(&sh->q_empty);
    float rise = 0.f;    // kTop - m; 0 for a row that has seen nothing yet: its exponents are its logits
    bool blank = sees;   // it sees something, but has not yet
    uint64_t l = 0ull;
    for (int i = t; i < n_tiles; i += 2) {
      const int k0 = (last - i) * BN;
      const bool masked = tree::tile_masked(p, ctx, k0);
      const uint32_t n = tiles + static_cast<uint32_t>(i), slot = n % kSlots;
      ok = warp_wait_idle(&sh->ready[slot], (n / kSlots) & 1u, wc, kSiteReady);
      ok = ok && warp_wait_idle(&sh->s_full[t], cnt & 1u, wc, kSiteS);
      if (!ok) break;
      ++cnt;
      tc_fence_after_sync();
      if (!warp_live) {
        tc_fence_before_sync();
        mbar_arrive(&sh->p_full[t]);
        continue;
      }
      const unsigned long long drafts = masked && k0 + BN > ctx ? in_window(p, at.b, own) : 0ull;
      // keys of 32 that the row sees
      auto bits_of = [&](int ch) {
        const int c0 = k0 + 32 * ch, from = ctx - c0;  // from: where draft 0 falls
        uint32_t bits = sees ? bits_between(lo - c0, ctx - c0) : 0u;
        if (from >= 0 && from < 32) bits |= static_cast<uint32_t>(drafts << from);
        else if (from < 0 && from > -64) bits |= static_cast<uint32_t>(drafts >> -from);
        return bits;
      };
      // Exponents of a chunk's weights (kRaw: scores times the chunk's factor).
      auto exponents = [&](auto hides, auto form, const uint32_t* s, int ch, int c, const Chunk& of, uint32_t bits, uint64_t* y) {
        constexpr bool kHides = decltype(hides)::value;
        constexpr int kForm = decltype(form)::value;
        const float a = fac * of.ks;
        float up = rise + of.lv;
        const uint64_t a2 = f2_pack(a, a);
        constexpr bool kMulFirst = mode_cap(MODE) || kForm == kRaw;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = f2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
          if constexpr (kMulFirst) y[e] = f2_mul(y[e], a2);
        }
        if constexpr (kForm != kRaw) {
          [[maybe_unused]] float size = 0.f;
          if constexpr (mode_cap(MODE)) cap_scores<kForm == kFar>(p, y, size);
          uint64_t add[4];
          if constexpr (mode_slopes(MODE) && kHides) {
            load8(&sh->before[slot][16 * ch + 8 * c], add);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              add[e] = f2_fma(f2_pack(fall, fall),
                              f2_add(add[e], f2_pack(static_cast<float>(depth), static_cast<float>(depth))) & 0x7fffffff7fffffffull,
                              f2_pack(up, up));
          } else if constexpr (mode_slopes(MODE)) {  // linear in the key's place
            up = fmaf(fall, static_cast<float>(ctx + depth - k0 - 16 * ch - 8 * c), up);
#pragma unroll
            for (int e = 0; e < 4; ++e) add[e] = f2_add(f2_pack(up, up), fall_e[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) add[e] = f2_pack(up, up);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = kMulFirst ? f2_add(y[e], add[e]) : f2_fma(y[e], a2, add[e]);
        }
        if constexpr (kHides) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x0, x1;
            f2_unpack(y[e], x0, x1);
            if (!((bits >> (8 * c + 2 * e)) & 1u)) x0 = -INFINITY;
            if (!((bits >> (8 * c + 2 * e + 1)) & 1u)) x1 = -INFINITY;
            y[e] = f2_pack(x0, x1);
          }
        }
      };
      // The greatest exponent.  (The cap is monotonic, and without distances a chunk's keys
      // have the rest in common.)
      auto greatest = [&](auto hides) {
        constexpr bool kHides = decltype(hides)::value, kLate = !mode_slopes(MODE);
        float most = -INFINITY;
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t s[32];
          tmem_ld_32x32b_x32(s_addr + 32 * ch, s);
          const uint32_t bits = kHides ? bits_of(ch) : 0u;
          tmem_ld_wait();
          reg_fence32(s);
          float m4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const Chunk of = sh->chunk[slot][4 * ch + c];
            uint64_t y[4];
            exponents(hides, std::integral_constant<int, kLate ? kRaw : kFar>{}, s + 8 * c, 2 * ch, c, of, bits, y);
            float x[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) f2_unpack(y[e], x[2 * e], x[2 * e + 1]);
            float top = fmax3(fmax3(fmax3(x[0], x[1], x[2]), x[3], x[4]), x[5], fmaxf(x[6], x[7]));
            if constexpr (kLate && mode_cap(MODE)) {
              const float z = top * p.inv_cap2, z2 = z * z;
              const float near = z * fmaf(z2, fmaf(z2, fmaf(z2, p.cap_k[3], p.cap_k[2]), p.cap_k[1]), p.cap_k[0]);
              const float far = fmaf(cap_r(z, 2.f * kLog2e), -2.f * p.cap2, p.cap2);
              top = top == -INFINITY ? top : (fabsf(z) <= 0.4f ? near : far);
            }
            m4[c] = kLate ? top + (rise + of.lv) : top;
          }
          most = fmax3(most, fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        }
        return most;
      };
      // Most tiles need no more than a bound to say that m stays: the loads return the
      // greatest magnitude of 32 scores.  (One pass that keeps the weights in registers until
      // their greatest is known has 64 fewer registers to work with, and code too long for the
      // instruction caches: B8 H32 kv8 T27 ctx 6000 d128 cap 30 99 us against 70.)
      bool stays = !masked && !blank;
      [[maybe_unused]] float size = 0.f;  // at least |y / cap|
#pragma unroll 1
      for (int ch = 0; ch < 4; ch += 2) {
        uint32_t s[2][32];
        float top[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) tmem_ld_absmax_32(s_addr + 32 * (ch + x), s[x], top[x]);
        tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float2 of = sh->bound[slot][ch + x];
          top[x] = fac * of.x * top[x];
          if constexpr (mode_cap(MODE)) {
            size = fmaxf(size, top[x] * p.inv_cap2);
            top[x] = fminf(top[x], p.cap2);
          }
          if constexpr (mode_slopes(MODE)) {
            const float far = static_cast<float>(ctx + depth - k0 - 32 * (ch + x));
            top[x] += fmaxf(fall * far, fall * (far - 31.f));
          }
          stays = stays && !(top[x] + (rise + of.y) > kMost);
        }
      }
      // Else m moves to the greatest where a weight would be too large (once does, but for
      // exponents beyond 2^24, where a difference is off by 2 and more).
      if (!__all_sync(0xffffffffu, stays)) {
#pragma unroll 1
        for (int moves = 0; moves < 3; ++moves) {
          const float most = masked ? greatest(std::true_type{}) : greatest(std::false_type{});
          const bool over = blank ? most > -INFINITY : most > kMost;
          if (!__any_sync(0xffffffffu, over)) break;
          float alpha = 1.f;
          if (over) {
            const float step = most - kTop;
            rise -= step;
            if (!blank) alpha = ex2_approx(-step);
            blank = false;
          }
          l = f2_mul(l, f2_pack(alpha, alpha));
          // (the accumulator's earlier products are done: S was issued behind them)
          if (i != t && __any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(o_addr + c, o);
              tmem_ld_wait();
              reg_fence32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st_32x32b_x32(o_addr + c, o);
            }
          }
          if (__all_sync(0xffffffffu, fabsf(rise) < 16777216.f)) break;
        }
      }
      // The weights' terms over the scores: of 32 keys term 0's 8 columns, then term 1's and
      // term 2's.
      auto weights = [&](auto hides, auto form) {
        constexpr bool kHides = decltype(hides)::value;
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t s[32], out[32];
          tmem_ld_32x32b_x32(s_addr + 32 * ch, s);
          const uint32_t bits = kHides ? bits_of(ch) : 0u;
          tmem_ld_wait();
          reg_fence32(s);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const Chunk of = sh->chunk[slot][4 * ch + c];
            uint64_t y[4], sum;
            uint32_t h2[4];
            exponents(hides, form, s + 8 * c, 2 * ch, c, of, bits, y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x0, x1;
              f2_unpack(y[e], x0, x1);
              x0 = ex2_approx(x0);
              x1 = ex2_approx(x1);
              sum = e == 0 ? f2_pack(x0, x1) : f2_add(sum, f2_pack(x0, x1));
              h2[e] = pack_f16x2(x0, x1);
            }
            l = f2_fma(sum, f2_pack(of.inv, of.inv), l);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t term[3];
              weights_of<false>(h2[2 * j], h2[2 * j + 1], term);
#pragma unroll
              for (int x = 0; x < 3; ++x) out[8 * x + 2 * c + j] = term[x];
            }
          }
          tmem_st_32x32b_x16(s_addr + 24 * ch, out);
          tmem_st_32x32b_x8(s_addr + 24 * ch + 16, out + 16);
        }
      };
      constexpr std::integral_constant<int, kNear> near;
      constexpr std::integral_constant<int, kFar> far;
      const bool small = mode_cap(MODE) && __all_sync(0xffffffffu, size <= 0.4f);
      if (masked) {
        if (small) weights(std::true_type{}, near);
        else weights(std::true_type{}, far);
      } else {
        if (small) weights(std::false_type{}, near);
        else weights(std::false_type{}, far);
      }
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&sh->p_full[t]);
    }
    if (!ok) break;
    // ---- the segment's end: warpgroup t finishes columns t d/2 .. of both accumulators
    ok = warp_wait_idle(&sh->o_full, seg & 1u, wc, kSitePv);
    if (!ok) break;
    float l0, l1;
    f2_unpack(l, l0, l1);
    sh->state[t][row] = make_float2(t < n_tiles && !blank ? kTop - rise : -INFINITY, l0 + l1);
    mbar_arrive(&sh->merge);
    ok = warp_wait_idle(&sh->merge, seg & 1u, wc, kSiteMerge);
    if (!ok) break;
    tc_fence_after_sync();
    const float2 s0 = sh->state[0][row], s1 = sh->state[1][row];
    const float M = fmaxf(s0.x, s1.x);
    const float f0 = s0.x == -INFINITY ? 0.f : ex2_approx(s0.x - M), f1 = s1.x == -INFINITY ? 0.f : ex2_approx(s1.x - M);
    const float L = fmaf(s0.y, f0, s1.y * f1);
    const bool empty = L == 0.f || !sees;
    const float rcp = empty ? 0.f : kSumUnit / L, g0 = f0 * rcp, g1 = f1 * rcp;
    const bool whole = !at.head_cut && !at.tail_cut;
    const long long part_row = (2 * static_cast<long long>(blockIdx.x) + (at.head_cut ? 0 : 1)) * p.tile_rows + row;
    constexpr int kHalf = HD / 2;
    const uint32_t from = lane_base + kOCol0 + static_cast<uint32_t>(t * kHalf);
    uint16_t* o_row = p.O + at.b * p.o_sb + h * p.o_sh + tok * p.o_sn + t * kHalf;
    float* part = p.o_part + part_row * HD + t * kHalf;
#pragma unroll 1
    for (int c = 0; warp_live && c < kHalf; c += 32) {
      uint32_t a0[32], a1[32];
      tmem_ld_32x32b_x32(from + c, a0);
      if (n_tiles > 1) tmem_ld_32x32b_x32(from + 128 + c, a1);
      tmem_ld_wait();
      reg_fence32(a0);
      reg_fence32(a1);
      float o[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        o[e] = __uint_as_float(a0[e]) * g0;
        if (n_tiles > 1) o[e] = fmaf(__uint_as_float(a1[e]), g1, o[e]);
        if (empty) o[e] = 0.f;
      }
      if (live && whole) {
        uint4* dst = reinterpret_cast<uint4*>(o_row + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[k] = kF16 ? pack_f16x2(o[8 * e + 2 * k], o[8 * e + 2 * k + 1]) : pack_bf16x2(o[8 * e + 2 * k], o[8 * e + 2 * k + 1]);
          dst[e] = make_uint4(x[0], x[1], x[2], x[3]);
        }
      } else if (live) {
        float4* dst = reinterpret_cast<float4*>(part + c);
#pragma unroll
        for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
      __syncwarp();
    }
    tc_fence_before_sync();
    mbar_arrive(&sh->o_empty);
    if (live && t == 0) {
      const float lse = empty ? -INFINITY : (M + (log2f(L) - (kTop + kSumLog2))) * kLn2;
      if (whole) p.LSE[(static_cast<long long>(at.b) * p.H + h) * p.T + tok] = lse;
      else p.lse_part[part_row] = lse;
    }
    tiles += static_cast<uint32_t>(n_tiles);
  }
}

// ------------------------------------------------------------------ queries and keys
// Four warps.  A thread a row: its elements' terms, in the K-major layout without a
// swizzle (16-byte pieces of all rows side by side).  Then, tile by tile ahead of the
// softmax: the chunks' scales as it takes them, and a thread a key where drafts are or a
// window starts: what no row sees leaves V.
template <int HD, bool kF16, int MODE>
__device__ __forceinline__ void prepare_role(const Params& p, Shared* sh, uint8_t* sQ, uint8_t* sV, WaitCtl wc) {
  using M = Mem<HD, kF16>;
  constexpr int kSlots = M::kSlots, kTerms = M::kTerms;
  const int me = threadIdx.x - 32 * kWarpPrepare, lane = me & 31, warp = me >> 5;
  uint32_t seg = 0, tiles = 0;
  bool ok = true;
  for (Walk w = sh->start; ok && next_segment(p, w); ++seg) {
    const int buf = seg & 1, ctx = w.ctx;
    const int row0 = w.rt * p.tile_rows, count = min(p.tile_rows, p.rows - row0);
    const bool live = me < count;
    const int row = row0 + (live ? me : 0), tok = row / p.group;
    const uint16_t* src = p.Q + w.b * p.q_sb + (w.hk * p.group + row - tok * p.group) * p.q_sh + tok * p.q_sn;
    auto load = [&](int i) { return live ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0u, 0u, 0u, 0u); };
    unsigned most = 0u;  // magnitudes, as two 16-bit values at a time
#pragma unroll 1
    for (int c = 0; c < HD / 8; c += 8) {
      uint4 e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = load(c + i);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        most = __vmaxu2(most, __vmaxu2(__vmaxu2(e[i].x & 0x7fff7fffu, e[i].y & 0x7fff7fffu),
                                       __vmaxu2(e[i].z & 0x7fff7fffu, e[i].w & 0x7fff7fffu)));
    }
    const float great = widen<kF16>(static_cast<uint16_t>(max(most & 0xffffu, most >> 16)));
    // 2^k brings it to 2^7 ..
    const int k = great == 0.f ? 0 : min(7 - (static_cast<int>(__float_as_uint(great) >> 23) - 127), 107);
    const float up = (p.scale_log2 < 0.f ? -1.f : 1.f) * __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
    // what the rows see
    const unsigned long long mask = live ? tree::mask_of(p, w.b, tok) : 0ull;
    const unsigned long long seen_drafts = in_window(p, w.b, mask);
    const int row_lo = mask == 0ull ? INT_MAX : (p.window > 0 ? max(0, ctx + tree::depth_of(mask) - p.window + 1) : 0);
    const unsigned see_lo = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(seen_drafts));
    const unsigned see_hi = __reduce_or_sync(0xffffffffu, static_cast<unsigned>(seen_drafts >> 32));
    const int warp_lo = __reduce_min_sync(0xffffffffu, row_lo);
    if (lane == 0) {
      sh->see[buf][warp] = static_cast<unsigned long long>(see_hi) << 32 | see_lo;
      sh->lo[buf][warp] = warp_lo;
    }
    __syncwarp();
    mbar_arrive(&sh->joined);
    if (seg > 0) ok = warp_wait_idle(&sh->q_empty, (seg - 1) & 1u, wc, kSiteQEmpty);
    if (!ok) break;
    sh->fac[me] = !(great <= 3.402823466e38f) ? __uint_as_float(0x7fc00000u) : (live ? fabsf(p.scale_log2) * down : 0.f);  // (not negative)
#pragma unroll 1
    for (int c = 0; c < HD / 16; ++c) {
      const uint4 e0 = load(2 * c), e1 = load(2 * c + 1);
      const uint32_t v[8] = {e0.x, e0.y, e0.z, e0.w, e1.x, e1.y, e1.z, e1.w};
      uint32_t out[kTerms][4];
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        uint32_t e[3][2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          __half2 r = __floats2half2_rn(widen<kF16>(static_cast<uint16_t>(v[j + x])) * up,
                                        widen<kF16>(static_cast<uint16_t>(v[j + x] >> 16)) * up);
          const uint16_t first = e4m3_of(r);
          e[0][x] = first;
          r = __hsub2(r, halves_of(first));  // exact, as is what follows
#pragma unroll
          for (int m = 1; m < kTerms; ++m) {
            e[m][x] = *reinterpret_cast<uint32_t*>(&r) + 0x00800080u;
            const uint32_t kept = e[m][x] & 0xff00ff00u;
            r = __hsub2(r, *reinterpret_cast<const __half2*>(&kept));
          }
        }
        out[0][j / 2] = __byte_perm(e[0][0], e[0][1], 0x5410);
#pragma unroll
        for (int m = 1; m < kTerms; ++m) out[m][j / 2] = __byte_perm(e[m][0], e[m][1], 0x7531);
      }
#pragma unroll
      for (int m = 0; m < kTerms; ++m)
        *reinterpret_cast<uint4*>(sQ + m * (kRows * HD) + c * (kRows * 16) + me * 16) =
            make_uint4(out[m][0], out[m][1], out[m][2], out[m][3]);
    }
    fence_async_smem();
    mbar_arrive(&sh->q_full);
    ok = warp_wait_idle(&sh->joined, seg & 1u, wc, kSitePrepare);
    if (!ok) break;
    const unsigned long long drafts = (sh->see[buf][0] | sh->see[buf][1]) | (sh->see[buf][2] | sh->see[buf][3]);
    const int lo = min(min(sh->lo[buf][0], sh->lo[buf][1]), min(sh->lo[buf][2], sh->lo[buf][3]));
    auto seen = [&](int key) {
      const int u = key - ctx;
      return u < 0 ? key >= lo : u < 64 && ((drafts >> u) & 1ull) != 0ull;
    };
    for (int i = 0; i < w.n; ++i) {
      const int k0 = (w.tile0 + w.n - 1 - i) * BN;
      const bool masked = tree::tile_masked(p, ctx, k0);
      const uint32_t n = tiles + static_cast<uint32_t>(i), slot = n % kSlots;
      ok = warp_wait_idle(&sh->scale_full[slot], (n / kSlots) & 1u, wc, kSiteScale);
      if (!ok) break;
      if (me < kChunks) {
        const float ks = sh->k_scale[slot][me];
        float vs = sh->v_scale[slot][me];
        bool any = lo != INT_MAX;
        if (masked) {
          any = false;
          for (int e = 0; e < kChunk; ++e) any = any || seen(k0 + kChunk * me + e);
        }
        if (vs == kNoPage) {  // (reads as zeros)
          if (any) atomicMax(p.status, kBadArg);
          vs = 1.f;
        }
        vs = vs < kLeastScale ? kLeastScale : vs;  // (values of a scale of 0 are 0, and their keys count all the same)
        const Chunk of = any ? Chunk{ks, lg2_approx(vs), kSumUnit * rcp_approx(vs)} : Chunk{0.f, 0.f, 0.f};
        sh->chunk[slot][me] = of;
        float k_most = fabsf(of.ks), lv_most = of.lv;
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
          k_most = fmaxf(k_most, __shfl_xor_sync(0xffffu, k_most, off));
          lv_most = fmaxf(lv_most, __shfl_xor_sync(0xffffu, lv_most, off));
        }
        if ((me & 3) == 0) sh->bound[slot][me / 4] = make_float2(k_most, lv_most);
      }
      if (masked) {
        const int key = k0 + me;
        if constexpr (mode_slopes(MODE))  // a key's own place, which for a draft is its depth
          sh->before[slot][me] = static_cast<float>(
              key >= ctx && key < ctx + p.T ? -tree::depth_of(tree::mask_of(p, w.b, key - ctx)) : ctx - key);
        ok = warp_wait_idle(&sh->v_full[slot], (n / kSlots) & 1u, wc, kSiteZero);
        if (!ok) break;
        if (!seen(key)) {  // (its row of V may hold anything)
          uint4* v = reinterpret_cast<uint4*>(sV + slot * M::kTileBytes + me * HD);
#pragma unroll
          for (int c = 0; c < HD / 16; ++c) v[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_smem();
      }
      mbar_arrive(&sh->ready[slot]);
    }
    tiles += static_cast<uint32_t>(w.n);
  }
}

// The scales of the chunks: lanes 0-15 K's, 16-31 V's.
template <int kSlots>
__device__ __forceinline__ void chunk_scale_role(const Params& p, Shared* sh, WaitCtl wc) {
  const int lane = threadIdx.x & 31, c = lane & 15;
  const int box = kChunk * c / p.box_rows, in_box = kChunk * c - box * p.box_rows;
  const float* const from = lane < 16 ? p.k_scale : p.v_scale;
  Tiles<1> tiles(p, sh->start, 0);
  Tile x;
  uint32_t n = 0;
  while (tiles.next(p, x)) {
    const uint32_t s = n % kSlots;
    if (n >= kSlots && !warp_wait_idle(&sh->empty[s], (n / kSlots - 1) & 1u, wc, kSiteEmpty)) break;
    const bool needed = x.in_page >= 0, good = needed && x.page >= 0 && x.page < p.num_pages;
    const int page = __shfl_sync(0xffffffffu, good ? x.page : (needed ? -2 : -1), box);
    const int row = __shfl_sync(0xffffffffu, x.in_page, box) + in_box;
    float* const to = lane < 16 ? &sh->k_scale[s][c] : &sh->v_scale[s][c];
    if (page >= 0) copy_ahead(to, from + (static_cast<long long>(page) * p.Hkv + x.hk) * p.scales + p.by_block.of(row));
    else *to = lane < 16 ? 0.f : (page == -2 ? kNoPage : 1.f);
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&sh->scale_full[s])) : "memory");
    mbar_arrive(&sh->scale_full[s]);
    ++n;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
}

// ------------------------------------------------------------------ MMA issuer
template <int HD, bool kF16>
__device__ __forceinline__ void mma_role(const Params& p, Shared* sh, uint32_t tmem, uint8_t* sK, uint8_t* sV, uint8_t* sQ,
                                         WaitCtl wc) {
  using M = Mem<HD, kF16>;
  constexpr int kSlots = M::kSlots;
  // rows of 128 or 64 bytes, swizzled as a whole; 8-row groups 8 HD bytes apart
  const uint64_t k_desc = sdesc_of(smem_u32(sK), 16, 8 * HD, HD == 128 ? 2u : 4u);
  const uint64_t v_desc = sdesc_of(smem_u32(sV), 0, 8 * HD, HD == 128 ? 2u : 4u);
  const uint64_t q_desc = sdesc_of(smem_u32(sQ), kRows * 16, 128, 0);
  constexpr uint32_t kTile = M::kTileBytes >> 4, kS = idesc_e4m3_f32(128, BN, 0, 0),
                     kO = idesc_e4m3_f32(128, HD, 0, 1) | kIdescAE5m2;
  uint32_t kc = 0, vc = 0, seg = 0, used[2] = {0, 0};
  bool ok = true;
  for (Walk w = sh->start; ok && next_segment(p, w); ++seg) {
    ok = warp_wait_idle(&sh->q_full, seg & 1u, wc, kSiteQ);
    if (!ok) break;
    // scores of tile i into buffer i mod 2, behind the products that read the buffer's weights
    auto scores = [&](int i) {
      const uint32_t s = kc % kSlots;
      if (!warp_wait_idle(&sh->k_full[s], (kc / kSlots) & 1u, wc, kSiteK)) return false;
      ++kc;
      tc_fence_after_sync();
#pragma unroll
      for (int m = 0; m < M::kTerms; ++m)
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk)
          mma_e4m3_ss(tmem + (i & 1) * 128, sdesc_add(q_desc, (m * kRows * HD + kk * 2 * kRows * 16) >> 4),
                      sdesc_add(k_desc, s * kTile + kk * 2), m == 0 ? kS : kS | kIdescAE5m2, m > 0 || kk > 0);
      mma_commit<true>(&sh->s_full[i & 1]);
      if (i == w.n - 1) mma_commit<true>(&sh->q_empty);
      return true;
    };
    ok = scores(0);
    if (ok && w.n > 1) ok = scores(1);
    for (int i = 0; ok && i < w.n; ++i) {
      const int t = i & 1;
      const uint32_t s = vc % kSlots;
      ok = warp_wait_idle(&sh->p_full[t], used[t] & 1u, wc, kSiteP);
      if (i == 0 && seg > 0) ok = ok && warp_wait_idle(&sh->o_empty, (seg - 1) & 1u, wc, kSiteOEmpty);
      ok = ok && warp_wait_idle(&sh->v_full[s], (vc / kSlots) & 1u, wc, kSiteV);
      ok = ok && warp_wait_idle(&sh->ready[s], (vc / kSlots) & 1u, wc, kSiteReady);
      if (!ok) break;
      ++used[t];
      ++vc;
      tc_fence_after_sync();
#pragma unroll
      for (int kk = 0; kk < BN / 32; ++kk)
#pragma unroll
        for (int m = 0; m < 3; ++m)
          mma_e4m3_ts(tmem + kOCol0 + t * 128, tmem + t * 128 + 24 * kk + 8 * m, sdesc_add(v_desc, s * kTile + kk * (32 * HD >> 4)),
                      kO, i >= 2 || kk > 0 || m > 0);
      mma_commit<true>(&sh->empty[s]);  // (its scores and scales have been read: P is there)
      if (i == w.n - 1) mma_commit<true>(&sh->o_full);
      if (i + 2 < w.n) ok = scores(i + 2);
    }
  }
  mma_commit<true>(&sh->drain);
  drain_wait(&sh->drain, 0, wc.limit_ns);
  __syncwarp();
}

template <int HD, bool kF16, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    tree_e4m3_wide_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ Params p) {
  using M = Mem<HD, kF16>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled tiles' alignment
    if (threadIdx.x == 0) atomicExch(p.status, 3u /* OSATTN_ERR_CUDA */);
    return;
  }
  uint8_t* sK = smem;
  uint8_t* sV = sK + M::kSlots * M::kTileBytes;
  uint8_t* sQ = smem + M::kRing;
  Shared* sh = reinterpret_cast<Shared*>(sQ + M::kQBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(&sh->q_full, 128);
    mbar_init(&sh->q_empty, 257);
    for (int s = 0; s < M::kSlots; ++s) {
      mbar_init(&sh->k_full[s], 1);
      mbar_init(&sh->v_full[s], 1);
      mbar_init(&sh->scale_full[s], 64);
      mbar_init(&sh->ready[s], 128);
      mbar_init(&sh->empty[s], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh->s_full[t], 1);
      mbar_init(&sh->p_full[t], 128);
    }
    mbar_init(&sh->o_full, 1);
    mbar_init(&sh->o_empty, 256);
    mbar_init(&sh->merge, 256);
    mbar_init(&sh->joined, 128);
    mbar_init(&sh->drain, 1);
    sh->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kWarpLoad && lane == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kWarpMma) {
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
  // 256 x 184 + 256 x 72 = 512 x 128 registers
  if (warp < kWarpLoad) {
    regs_inc<184>();
    softmax_role<HD, kF16, MODE>(p, sh, tmem, warp >> 2, wc);
  } else {
    regs_dec<72>();
    if (warp < kWarpScale) load_role<HD, M::kSlots>(&tmK, &tmV, p, sh, sK, sV, warp - kWarpLoad, wc);
    else if (warp == kWarpScale) chunk_scale_role<M::kSlots>(p, sh, wc);
    else if (warp == kWarpMma) mma_role<HD, kF16>(p, sh, tmem, sK, sV, sQ, wc);
    else prepare_role<HD, kF16, MODE>(p, sh, sQ, sV, wc);
  }

  __syncwarp();
  tmem_st_wait();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kWarpMma) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace wide
}  // namespace tree8
}  // namespace osattn
