// softmax_tile.cuh - the elementwise work of one row of a 128-key score tile,
// shared by the forward kernels with modified scores and over a paged cache.
//
// One thread has a row and holds its 128 scores in registers.  The max that P
// is formed against comes from the max that the tensor-memory loads return,
// where the modification of the scores is monotonic or its spread over 32 keys
// is small (a lower bound of the max will do, see kMaxSlack); the modification
// then takes the shift by the max into its last multiply-add, and P follows in
// the same pass.  Every instruction here costs time: the tiles' softmaxes are
// bound by issue and latency, not by one pipe.  (A rolled loop that reads each
// chunk of 32 scores again from tensor memory is a fourth of the code, and
// 10 to 25 % slower.)
#pragma once

#include <cstdint>

#include "mod_common.cuh"
#include "sm100_ptx.cuh"

namespace osattn {

constexpr int kChunks = 4;
constexpr uint32_t kMinusInf = 0xff800000u;

// The max that P is formed against is moved only when it grows by more than
// this (log2 units), so that the accumulator in tensor memory is left alone on
// almost every tile.  P may then exceed 1, by 2^8 and by as much as the max was
// a lower bound only: fp32 sums and 16-bit P keep their relative precision.
// It is kept a whole number, so that the factor of the accumulator is a power
// of two, exact in the upper 16 bits of an fp32.
constexpr float kMaxSlack = 8.f;
__device__ __forceinline__ float next_max(float m, float mx) { return mx > m + kMaxSlack ? ceilf(mx) : m; }
__device__ __forceinline__ uint16_t alpha_bits(float m, float m_new) {
  return static_cast<uint16_t>(__float_as_uint(m_new == m ? 1.f : ex2_approx(m - m_new)) >> 16);
}
__device__ __forceinline__ float alpha_of(uint16_t bits) { return __uint_as_float(static_cast<uint32_t>(bits) << 16); }

using Chunk = uint32_t[32];

__device__ __forceinline__ uint64_t pair_of(const Chunk& v, int e) {
  return f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
}
__device__ __forceinline__ void set_pair(Chunk& v, int e, uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  v[e] = __float_as_uint(a);
  v[e + 1] = __float_as_uint(b);
}

// 32 scores of a row, and the greatest of their magnitudes (NaN aside).
__device__ __forceinline__ void tmem_ld_absmax_32(uint32_t taddr, Chunk& v, float& size) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x32.max.abs.f32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
      "%32, [%33];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]),
        "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
        "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]),
        "=r"(v[30]), "=r"(v[31]), "=f"(size)
      : "r"(taddr));
}

using Row = Chunk[kChunks];

// The row's scores and the max (kAbs: the greatest magnitude) of each chunk,
// formed by the loads.
template <bool kAbs>
__device__ __forceinline__ void load_row(uint32_t s_addr, Row& v, float (&top)[kChunks]) {
#pragma unroll
  for (int ch = 0; ch < kChunks; ++ch) {
    if constexpr (kAbs) tmem_ld_absmax_32(s_addr + ch * 32, v[ch], top[ch]);
    else tmem_ld_red_32x32b_x32<true>(s_addr + ch * 32, v[ch], top[ch]);
  }
  tmem_ld_wait();
#pragma unroll
  for (int ch = 0; ch < kChunks; ++ch) {
    reg_fence32(v[ch]);
    asm volatile("" : "+f"(top[ch]));
  }
}

__device__ __forceinline__ float chunk_max(const Chunk& v) {
  float a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = fmaxf(__uint_as_float(v[i]), __uint_as_float(v[4 + i]));
#pragma unroll
  for (int j = 8; j < 32; j += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = fmax3(a[i], __uint_as_float(v[j + i]), __uint_as_float(v[j + 4 + i]));
  return fmaxf(fmax3(a[0], a[1], a[2]), a[3]);
}
__device__ __forceinline__ float chunk_min(const Chunk& v) {
  float a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = fminf(__uint_as_float(v[i]), __uint_as_float(v[4 + i]));
#pragma unroll
  for (int j = 8; j < 32; j += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = fmin3(a[i], __uint_as_float(v[j + i]), __uint_as_float(v[j + 4 + i]));
  return fminf(fmin3(a[0], a[1], a[2]), a[3]);
}

__device__ __forceinline__ float chunk_absmax(const Chunk& v) { return fmaxf(chunk_max(v), -chunk_min(v)); }

// Bits [from, to) of 32, for any from and to.
__device__ __forceinline__ uint32_t bit_range(int from, int to) {
  const int a = min(max(from, 0), 32), b = min(max(to, 0), 32);
  uint32_t m;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(max(b - a, 0)));
  return m;
}

// What a warp's rows see of a tile, chunk by chunk: bit ch of `partial` set if
// some row sees some but not every key of it, of `none` if no row sees one.
// A mask costs only the chunks it cuts, and keys that no row of the warp sees
// cost nothing.  bits_of(ch): the row's visible keys of chunk ch.
struct TileMask {
  uint32_t partial = 0u, none = 0u;
  template <typename BitsOf>
  __device__ __forceinline__ void classify(BitsOf&& bits_of) {
#pragma unroll
    for (int ch = 0; ch < kChunks; ++ch) {
      const uint32_t bits = bits_of(ch);
      if (!__any_sync(0xffffffffu, bits != 0u)) none |= 1u << ch;
      else if (!__all_sync(0xffffffffu, bits == 0xffffffffu)) partial |= 1u << ch;
    }
  }
};

// `fill` at the row's masked keys.  Tests of single bits of a word cost one
// instruction for several predicates, against two comparisons a key.
__device__ __forceinline__ void mask_chunk(Chunk& v, uint32_t bits, uint32_t fill) {
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = (bits & (1u << e)) ? v[e] : fill;
}

// How one tile's scores become base-2 logits for one row: x = cap(s) c + off
// (+ bias), where cap(s) c is cap2 tanh(s |scale| / cap) with a cap and s c
// without.  c > 0: a negative scale's sign is in the scores (the MMA negates
// an operand), and a scale of 0 is a c too small to matter.
template <bool kF16, int MODE>
struct TileScore {
  float c;                // |scale| * log2(e)
  float off;              // constant part of the bias
  const CapArgs* cap;
  float slope2, d0;       // both_sides: - slope2 |d0 + e| (or another distance)
  bool both_sides;
  const float* strip;     // learned bias of the tile's first key for this row, or null: off has it
  float strip_lo;         // least bias of the head
  bool strip_close;       // the head's biases lie within kSpread of each other
  int near_lo, near_hi;   // first keys x of chunks, from the tile's first, with near_lo < x < near_hi
                          // have distances within (-R, R): the strip; others one bias per side
  float far_lo, far_hi;

  // How far a lower bound of the row max may be off: P then reaches
  // 2^(kMaxSlack + this), which has to stay a finite 16-bit value, and in bf16
  // leaves fp32 sums of 2^30 values of V below 2^56 finite.
  static constexpr float kSpread = kF16 ? 7.f : 32.f;

  // Distances that grow by one from key to key: of key e of chunk ch.
  __device__ __forceinline__ auto by_place() const {
    const float d = d0;
    return [d](int ch) { return [d, ch](int e) { return d + static_cast<float>(32 * ch + e); }; };
  }

  // cap(s) c of one score
  __device__ __forceinline__ float raw(float s) const {
    if constexpr (mode_cap(MODE)) return fmaf(cap_r(s, cap->c1), -2.f * cap->cap2, cap->cap2);
    else return s * c;
  }

  // One tile of the row: S at s_addr becomes P = 2^(x - m) in 16 bits over its
  // first 64 columns.  Moves m, publishes the factor of the accumulator by
  // publish(alpha_bits) as soon as it is known, and updates l.
  // gap(ch)(e): the distance of key e of chunk ch, for both_sides.
  // kMasked: some rows of the warp may not see all of the tile.
  // kShort: with a shorter way for small capped scores (its code costs kernels
  // of few tiles 2 us).
  // kDirectOnly: without code for tiles whose logits have to be formed before
  // their max; false for such a tile, with nothing done.
  template <bool kMasked, bool kShort, bool kDirectOnly, typename BitsOf, typename Gap, typename Publish>
  __device__ __forceinline__ bool tile(uint32_t s_addr, const TileMask& k, BitsOf&& bits_of, Gap&& gap,
                                       float& m, float& l, Publish&& publish) const {
    Row v;
    float top[kChunks];
    constexpr bool kFree = kShort && !kMasked && MODE == kModCap;
    load_row<kFree || MODE == kModCapSlopes>(s_addr, v, top);
    if constexpr (kFree) {
      // Scores so small that the tile's own max is not needed (free_logits), and
      // the accumulator's factor (1, but for a max below free_max so far) comes
      // before anything else.
      if (__all_sync(0xffffffffu, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) <= cap->s_free)) {
        const float m_new = fmaxf(m, free_max(kF16));
        publish(alpha_bits(m, m_new));
        const float sum = exps<false, true, 2>(s_addr, v, k, bits_of, -m_new);
        l = fmaf(l, m_new == m ? 1.f : ex2_approx(m - m_new), sum);
        m = m_new;
        return true;
      }
#pragma unroll
      for (int ch = 0; ch < kChunks; ++ch) top[ch] = chunk_max(v[ch]);
    }
    if constexpr (kMasked) {
      // Masked scores, which may hold anything: out of the max, and 0 where
      // scores share a reciprocal.
#pragma unroll
      for (int ch = 0; ch < kChunks; ++ch) {
        if ((k.partial >> ch) & 1u) {
          const uint32_t bits = bits_of(ch);
          if constexpr (MODE == kModCapSlopes) {
            mask_chunk(v[ch], bits, 0u);
            top[ch] = chunk_absmax(v[ch]);
          } else {
            mask_chunk(v[ch], bits, kMinusInf);
            top[ch] = chunk_max(v[ch]);
            if constexpr (mode_cap(MODE)) mask_chunk(v[ch], bits, 0u);
          }
        }
        if ((k.none >> ch) & 1u) {
          top[ch] = -INFINITY;
          if constexpr (mode_cap(MODE)) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[ch][e] = 0u;
          }
        }
      }
    }
    const float best_raw = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    bool direct = true;  // uniform over the warp
    if constexpr (MODE == kModCap) {
      const float least = fminf(fminf(chunk_min(v[0]), chunk_min(v[1])), fminf(chunk_min(v[2]), chunk_min(v[3])));
      const float size = fmaxf(best_raw, -least);
      direct = __all_sync(0xffffffffu, size <= cap->s_max);
    }
    if constexpr (MODE == kModSlopes) direct = !both_sides;
    if constexpr (MODE == kModCapSlopes) direct = false;
    if constexpr (mode_rel(MODE)) direct = strip == nullptr;
    if (kDirectOnly && !direct) return false;
    float m_new, sum;
    if (kDirectOnly || direct) {
      m_new = next_max(m, best_raw == -INFINITY ? -INFINITY : raw(best_raw) + off);
      publish(alpha_bits(m, m_new));
      // a row with no key so far has m_new = -inf and every x = -inf: against
      // 0 each p is exactly 0
      const float n = off - (m_new == -INFINITY ? 0.f : m_new);
      sum = exps<kMasked, true, 3>(s_addr, v, k, bits_of, n);
    } else if constexpr (MODE != kModPlain) {
      float best = -INFINITY;
      const bool bound = mode_rel(MODE) && strip_close;
      if (bound && best_raw != -INFINITY) best = raw(best_raw) + strip_lo;
#pragma unroll
      for (int ch = 0; ch < kChunks; ++ch) {
        if (kMasked && ((k.none >> ch) & 1u)) continue;
        logits(v[ch], ch, gap, MODE == kModCapSlopes && small_scores(top[ch]));
        if (kMasked && mode_cap(MODE) && ((k.partial >> ch) & 1u)) mask_chunk(v[ch], bits_of(ch), kMinusInf);
        if (!bound) best = fmaxf(best, chunk_max(v[ch]));
      }
      m_new = next_max(m, best);
      publish(alpha_bits(m, m_new));
      sum = exps<kMasked, false, 0>(s_addr, v, k, bits_of, m_new == -INFINITY ? 0.f : -m_new);
    }
    l = fmaf(l, m_new == m ? 1.f : ex2_approx(m - m_new), sum);
    m = m_new;
    return true;
  }

  // The same for a masked tile by a rolled loop that reads each chunk from
  // tensor memory twice: a third of the instructions, for tiles that a CTA
  // meets once or twice, whose code then comes from far (8 trees of 27 drafts over
  // 6000 keys: 58 us against 65; a prompt's many masked tiles would be 10 to 25 %
  // slower).
  // kFine: with the cap's polynomial where a chunk's scores are small, for caps
  // above 64: the other form is off by up to 2^-20 of the cap, 6e-5 at a cap of 64.
  // (Its code costs: with it for all caps that tree, cap 30, takes 3 us more.)
  template <bool kFine, typename BitsOf, typename Gap, typename Publish>
  __device__ __forceinline__ void tile_rolled(uint32_t s_addr, const TileMask& k, BitsOf&& bits_of, Gap&& gap,
                                              float& m, float& l, Publish&& publish) const {
    auto load = [&](int ch, Chunk& v) {
      tmem_ld_32x32b_x32(s_addr + ch * 32, v);
      tmem_ld_wait();
      reg_fence32(v);
      const uint32_t bits = bits_of(ch);
      bool small = false;
      if constexpr (mode_cap(MODE)) {
        mask_chunk(v, bits, 0u);
        if constexpr (kFine) small = small_scores(chunk_absmax(v));
      }
      logits(v, ch, gap, small);
      mask_chunk(v, bits, kMinusInf);
    };
    float best = -INFINITY;
#pragma unroll 1
    for (int ch = 0; ch < kChunks; ++ch) {
      if ((k.none >> ch) & 1u) continue;
      Chunk v;
      load(ch, v);
      best = fmaxf(best, chunk_max(v));
    }
    const float m_new = next_max(m, best);
    publish(alpha_bits(m, m_new));
    const float n = m_new == -INFINITY ? 0.f : -m_new;
    float sum = 0.f;
#pragma unroll 1
    for (int ch = 0; ch < kChunks; ++ch) {
      uint32_t pk[16];
      if ((k.none >> ch) & 1u) {
#pragma unroll
        for (int e = 0; e < 16; ++e) pk[e] = 0u;
      } else {
        Chunk v;
        load(ch, v);
        float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float p0 = ex2_approx(__uint_as_float(v[2 * e]) + n), p1 = ex2_approx(__uint_as_float(v[2 * e + 1]) + n);
          a[(2 * e) & 3] += p0;
          a[(2 * e + 1) & 3] += p1;
          if constexpr (kF16) pk[e] = pack_f16x2(p0, p1);
          else pk[e] = pack_bf16x2(p0, p1);
        }
        sum += (a[0] + a[1]) + (a[2] + a[3]);
      }
      tmem_st_32x32b_x16(s_addr + ch * 16, pk);
    }
    l = fmaf(l, m_new == m ? 1.f : ex2_approx(m - m_new), sum);
    m = m_new;
  }

  // Whether the cap's polynomial serves all of the warp's rows; size: the greatest
  // magnitude of the row's scores.
  __device__ __forceinline__ bool small_scores(float size) const {
    return __all_sync(0xffffffffu, size <= cap->s_max);
  }

  // x in place of the 32 scores of chunk ch, less the constant part of the bias.
  // small: small_scores of the chunk.
  template <typename Gap>
  __device__ __forceinline__ void logits(Chunk& v, int ch, Gap&& gap, bool small) const {
    if (mode_cap(MODE) && small) {
#pragma unroll
      for (int e = 0; e < 32; e += 2) set_pair(v, e, cap_pair<3>(pair_of(v, e), 0ull));
    } else if constexpr (mode_cap(MODE)) {
      // cap2 - 2 cap2 / (1 + E): one reciprocal for four scores, 1 + E kept
      // below 2^30 so that four multiply without overflow (the tanh is 1 to
      // the last bit long before)
      const CapArgs& a = *cap;
      const uint64_t c1 = f2_pack(a.c1, a.c1), one = f2_pack(1.f, 1.f);
      const uint64_t mul = f2_pack(-2.f * a.cap2, -2.f * a.cap2), n = f2_pack(a.cap2, a.cap2);
#pragma unroll
      for (int e = 0; e < 32; e += 4) {
        float z0, z1, z2, z3, px, py;
        f2_unpack(f2_mul(pair_of(v, e), c1), z0, z1);
        f2_unpack(f2_mul(pair_of(v, e + 2), c1), z2, z3);
        const uint64_t ua = f2_add(f2_pack(ex2_approx(min30(z0)), ex2_approx(min30(z1))), one);
        const uint64_t ub = f2_add(f2_pack(ex2_approx(min30(z2)), ex2_approx(min30(z3))), one);
        f2_unpack(f2_mul(ua, ub), px, py);  // u0 u2, u1 u3
        const float q = rcp_approx(px * py);
        const uint64_t r = f2_mul(f2_pack(q, q), f2_pack(py, px));  // 1 / (u0 u2), 1 / (u1 u3)
        set_pair(v, e, f2_fma(f2_mul(r, ub), mul, n));
        set_pair(v, e + 2, f2_fma(f2_mul(r, ua), mul, n));
      }
    } else if constexpr (mode_rel(MODE)) {
      const uint64_t c2 = f2_pack(c, c);
      if (ch * 32 > near_lo && ch * 32 < near_hi) {
        const float* at = strip + ch * 32;
#pragma unroll
        for (int e = 0; e < 32; e += 2) set_pair(v, e, f2_fma(pair_of(v, e), c2, f2_pack(at[e], at[e + 1])));
      } else {
        const float far = ch * 32 <= near_lo ? far_lo : far_hi;
        const uint64_t b2 = f2_pack(far, far);
#pragma unroll
        for (int e = 0; e < 32; e += 2) set_pair(v, e, f2_fma(pair_of(v, e), c2, b2));
      }
    }
    if constexpr (MODE == kModPlain) {
      const uint64_t c2 = f2_pack(c, c);
#pragma unroll
      for (int e = 0; e < 32; e += 2) set_pair(v, e, f2_mul(pair_of(v, e), c2));
    }
    if constexpr (mode_slopes(MODE)) {
      const float mul = mode_cap(MODE) ? 1.f : c;
      const auto dist = gap(ch);
#pragma unroll
      for (int e = 0; e < 32; ++e)
        v[e] = __float_as_uint(fmaf(-slope2, fabsf(dist(e)), __uint_as_float(v[e]) * mul));
    }
  }

  // cap2 tanh(s |scale| / cap) + n of two scores by the polynomial (n2: n twice).
  template <int kDegree>
  __device__ __forceinline__ uint64_t cap_pair(uint64_t s, uint64_t n2) const {
    const uint64_t u = f2_mul(s, s);
    if constexpr (kDegree == 2) {
      const uint64_t k0 = f2_pack(cap->q[0], cap->q[0]), k1 = f2_pack(cap->q[1], cap->q[1]),
                     k2 = f2_pack(cap->q[2], cap->q[2]);
      return f2_fma(f2_fma(f2_fma(k2, u, k1), u, k0), s, n2);
    } else {
      const uint64_t k0 = f2_pack(cap->k[0], cap->k[0]), k1 = f2_pack(cap->k[1], cap->k[1]),
                     k2 = f2_pack(cap->k[2], cap->k[2]), k3 = f2_pack(cap->k[3], cap->k[3]);
      return f2_fma(f2_fma(f2_fma(f2_fma(k3, u, k2), u, k1), u, k0), s, n2);
    }
  }

  // x + n of two raw scores (direct tiles); n2: n twice, with off in it.
  template <int kDegree>
  __device__ __forceinline__ uint64_t direct_pair(uint64_t s, uint64_t n2) const {
    if constexpr (MODE == kModCap) return cap_pair<kDegree>(s, n2);
    else return f2_fma(s, f2_pack(c, c), n2);
  }

  // P in 16 bits over the first 64 columns of the row's scores, and the sum:
  // 2^(x + n) from raw scores (kDirect, n with off), or 2^(v + n).  kMasked:
  // chunks that no row of the warp sees are zeros.
  template <bool kMasked, bool kDirect, int kDegree, typename BitsOf>
  __device__ __forceinline__ float exps(uint32_t s_addr, const Row& v, const TileMask& k, BitsOf&& bits_of,
                                        float n) const {
    uint64_t rs_a = 0, rs_b = 0;  // packed partial sums (bit pattern 0 = 0.0f)
    const uint64_t n2 = f2_pack(n, n);
#pragma unroll
    for (int ch = 0; ch < kChunks; ++ch) {
      uint32_t pk[16];
      if (kMasked && ((k.none >> ch) & 1u)) {
#pragma unroll
        for (int e = 0; e < 16; ++e) pk[e] = 0u;
      } else {
        // capped scores: a masked one was set to 0, not -inf
        constexpr bool kCut = kMasked && kDirect && MODE == kModCap;
        uint32_t bits = 0u;
        if constexpr (kCut) bits = ((k.partial >> ch) & 1u) ? bits_of(ch) : 0xffffffffu;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint64_t s = pair_of(v[ch], 2 * e);
          float x0, x1;
          f2_unpack(kDirect ? direct_pair<kDegree>(s, n2) : f2_add(s, n2), x0, x1);
          if constexpr (kCut) {
            x0 = (bits & (1u << (2 * e))) ? x0 : -INFINITY;
            x1 = (bits & (2u << (2 * e))) ? x1 : -INFINITY;
          }
          const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
          const uint64_t pp = f2_pack(p0, p1);
          if (e & 1)
            rs_b = f2_add(rs_b, pp);
          else
            rs_a = f2_add(rs_a, pp);
          if constexpr (kF16) pk[e] = pack_f16x2(p0, p1);
          else pk[e] = pack_bf16x2(p0, p1);
        }
      }
      tmem_st_32x32b_x16(s_addr + ch * 16, pk);
    }
    float r0, r1, r2, r3;
    f2_unpack(rs_a, r0, r1);
    f2_unpack(rs_b, r2, r3);
    return (r0 + r1) + (r2 + r3);
  }
};

// Writes 32 16-bit values of a row, from column col0 (a multiple of 8), into a
// 128-row tile in shared memory in the layout of 64-column TMA boxes with the
// 128-byte swizzle: 16-byte chunk x of a row's 128 bytes sits at chunk
// x ^ (row mod 8).
__device__ __forceinline__ void stage_row32(uint8_t* tile, int row, int col0, const uint32_t (&pk)[16]) {
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int col = col0 + 8 * x;
    *reinterpret_cast<uint4*>(tile + (col / 64) * 128 * 128 + row * 128 + ((((col % 64) / 8) ^ (row & 7)) * 16)) =
        make_uint4(pk[4 * x], pk[4 * x + 1], pk[4 * x + 2], pk[4 * x + 3]);
  }
}

// 4-D tiled store of one box from shared memory (c0 innermost); rows outside
// the tensor are not written.
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int c0, int c1,
                                             int c2, int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
               : "memory");
}
// The stores issued by this thread have read their shared memory, which may
// then be given up; they land before the kernel ends.
__device__ __forceinline__ void tma_store_drain() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}

}  // namespace osattn
