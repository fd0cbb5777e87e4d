// softmax_tile.cuh - the elementwise work of one row of a 128-key score tile,
// shared by the forward kernels with modified scores and over a paged cache.
// A thread holds the row's 128 scores in registers.
#pragma once

#include <cstdint>

#include "mod_common.cuh"
#include "sm100_ptx.cuh"

namespace osattn {

constexpr int kTileKeys = 128;

// The running max is moved only when it grows by more than this (log2 units):
// P then stays below 2^8, which neither fp32 sums nor 16-bit P mind, and the
// accumulator in tensor memory is left alone on almost every tile.
constexpr float kMaxSlack = 8.f;

// Bits [from, to) of 32, for any from and to.
__device__ __forceinline__ uint32_t bit_range(int from, int to) {
  const int a = min(max(from, 0), 32), b = min(max(to, 0), 32);
  uint32_t m;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(max(b - a, 0)));
  return m;
}

// -inf (or another value) where the row's bit is clear.  Tests of single bits of a word cost one
// instruction for several predicates, against two comparisons a score.
template <uint32_t kFill = 0xff800000u>
__device__ __forceinline__ void mask_tile(uint32_t (&v)[kTileKeys], const uint32_t (&bits)[4]) {
#pragma unroll
  for (int e = 0; e < kTileKeys; ++e)
    v[e] = (bits[e >> 5] & (1u << (e & 31))) ? v[e] : kFill;
}

__device__ __forceinline__ uint64_t pair_of(const uint32_t (&v)[kTileKeys], int e) {
  return f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
}
__device__ __forceinline__ void set_pair(uint32_t (&v)[kTileKeys], int e, uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  v[e] = __float_as_uint(a);
  v[e + 1] = __float_as_uint(b);
}

__device__ __forceinline__ void scale_tile(uint32_t (&v)[kTileKeys], float c) {
  const uint64_t c2 = f2_pack(c, c);
#pragma unroll
  for (int e = 0; e < kTileKeys; e += 2) set_pair(v, e, f2_mul(pair_of(v, e), c2));
}

// Row max: 3-input instructions in 8 chains.
__device__ __forceinline__ float max_tile(const uint32_t (&v)[kTileKeys]) {
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = fmaxf(__uint_as_float(v[i]), __uint_as_float(v[i + 8]));
#pragma unroll
  for (int j = 16; j < kTileKeys; j += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      a[i] = fmax3(a[i], __uint_as_float(v[j + i]), __uint_as_float(v[j + 8 + i]));
  return fmax3(fmax3(a[0], a[1], a[2]), fmax3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
}

// Largest 2 y log2(e) / cap for which four 1 + E multiply without overflow
// (2^30 to the fourth); the tanh is 1 to the last bit long before.
constexpr float kCapFast = 30.f;

// Scores to capped base-2 logits, cap2 - 2 cap2 / (1 + E) (see cap_r).  `fast`:
// no exponent is above kCapFast; four reciprocals are then made from one and
// six multiplications in pairs: the unit that does reciprocals and
// exponentials, which bounds this pass, has 1.25 instructions a score to do
// instead of 2.
__device__ __forceinline__ void cap_tile(uint32_t (&v)[kTileKeys], float c1, float cap2, bool fast) {
  const uint64_t c1p = f2_pack(c1, c1), one = f2_pack(1.f, 1.f);
  const uint64_t mul = f2_pack(-2.f * cap2, -2.f * cap2), add = f2_pack(cap2, cap2);
  if (fast) {
#pragma unroll
    for (int e = 0; e < kTileKeys; e += 4) {
      float z0, z1, z2, z3, px, py;
      f2_unpack(f2_mul(pair_of(v, e), c1p), z0, z1);
      f2_unpack(f2_mul(pair_of(v, e + 2), c1p), z2, z3);
      const uint64_t ua = f2_add(f2_pack(ex2_approx(z0), ex2_approx(z1)), one);
      const uint64_t ub = f2_add(f2_pack(ex2_approx(z2), ex2_approx(z3)), one);
      f2_unpack(f2_mul(ua, ub), px, py);      // u0 u2, u1 u3
      const float q = rcp_approx(px * py);
      const uint64_t r = f2_mul(f2_pack(q, q), f2_pack(py, px));  // 1 / (u0 u2), 1 / (u1 u3)
      set_pair(v, e, f2_fma(f2_mul(r, ub), mul, add));
      set_pair(v, e + 2, f2_fma(f2_mul(r, ua), mul, add));
    }
  } else {
#pragma unroll
    for (int e = 0; e < kTileKeys; ++e)
      v[e] = __float_as_uint(fmaf(cap_r(__uint_as_float(v[e]), c1), -2.f * cap2, cap2));
  }
}

// P = 2^(v cm + neg) in 16 bits over columns s_addr .. + 63, and its sum.
template <bool kF16>
__device__ __forceinline__ float exp_tile(const uint32_t (&v)[kTileKeys], float cm, float neg,
                                          uint32_t s_addr) {
  const uint64_t cm2 = f2_pack(cm, cm), nm2 = f2_pack(neg, neg);
  uint64_t rs_a = 0, rs_b = 0;  // packed partial sums (bit pattern 0 = 0.0f)
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t pk[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      float x0, x1;
      f2_unpack(f2_fma(pair_of(v, half * 64 + 2 * e), cm2, nm2), x0, x1);
      const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
      const uint64_t pp = f2_pack(p0, p1);
      if (e & 1)
        rs_b = f2_add(rs_b, pp);
      else
        rs_a = f2_add(rs_a, pp);
      if constexpr (kF16) pk[e] = pack_f16x2(p0, p1);
      else pk[e] = pack_bf16x2(p0, p1);
    }
    tmem_st_32x32b_x32(s_addr + half * 32, pk);
  }
  float r0, r1, r2, r3;
  f2_unpack(rs_a, r0, r1);
  f2_unpack(rs_b, r2, r3);
  return (r0 + r1) + (r2 + r3);
}

// The running max for a row whose tile has max `mx`: unchanged while mx is
// within kMaxSlack of it.
__device__ __forceinline__ float next_max(float m, float mx) { return mx > m + kMaxSlack ? mx : m; }

}  // namespace osattn
