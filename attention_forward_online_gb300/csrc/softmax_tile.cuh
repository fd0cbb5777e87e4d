// softmax_tile.cuh - the elementwise work of one row of a 128-key score tile,
// shared by the forward kernels with modified scores and over a paged cache.
// A thread holds the row's 128 scores in registers, as four chunks of 32.
#pragma once

#include <cstdint>

#include "mod_common.cuh"
#include "sm100_ptx.cuh"

namespace osattn {

constexpr int kTileKeys = 128;
constexpr int kChunks = 4;
constexpr uint32_t kMinusInf = 0xff800000u;

// The running max is moved only when it grows by more than this (log2 units):
// P then stays below 2^8, which neither fp32 sums nor 16-bit P mind, and the
// accumulator in tensor memory is left alone on almost every tile.
constexpr float kMaxSlack = 8.f;
__device__ __forceinline__ float next_max(float m, float mx) { return mx > m + kMaxSlack ? mx : m; }

using Row = uint32_t[kTileKeys];

__device__ __forceinline__ uint64_t pair_of(const Row& v, int e) {
  return f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
}
__device__ __forceinline__ void set_pair(Row& v, int e, uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  v[e] = __float_as_uint(a);
  v[e + 1] = __float_as_uint(b);
}

// The row's scores and the max of each chunk, formed by the loads.
__device__ __forceinline__ void load_row(uint32_t s_addr, Row& v, float (&ext)[kChunks]) {
#pragma unroll
  for (int ch = 0; ch < kChunks; ++ch) tmem_ld_red_32x32b_x32<true>(s_addr + ch * 32, v + ch * 32, ext[ch]);
  tmem_ld_wait();
#pragma unroll
  for (int ch = 0; ch < kChunks; ++ch) {
    reg_fence32(v + ch * 32);
    asm volatile("" : "+f"(ext[ch]));
  }
}

__device__ __forceinline__ float chunk_max(const Row& v, int ch) {
  float a[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = fmaxf(__uint_as_float(v[ch * 32 + i]), __uint_as_float(v[ch * 32 + 4 + i]));
#pragma unroll
  for (int j = 8; j < 32; j += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = fmax3(a[i], __uint_as_float(v[ch * 32 + j + i]), __uint_as_float(v[ch * 32 + j + 4 + i]));
  return fmaxf(fmax3(a[0], a[1], a[2]), a[3]);
}

__device__ __forceinline__ float row_min(const Row& v) {
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = fminf(__uint_as_float(v[i]), __uint_as_float(v[i + 8]));
#pragma unroll
  for (int j = 16; j < kTileKeys; j += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      a[i] = fmin3(a[i], __uint_as_float(v[j + i]), __uint_as_float(v[j + 8 + i]));
  return fmin3(fmin3(a[0], a[1], a[2]), fmin3(a[3], a[4], a[5]), fminf(a[6], a[7]));
}

__device__ __forceinline__ float max4(const float (&e)[kChunks]) {
  return fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
}

// Bits [from, to) of 32, for any from and to.
__device__ __forceinline__ uint32_t bit_range(int from, int to) {
  const int a = min(max(from, 0), 32), b = min(max(to, 0), 32);
  uint32_t m;
  asm("bmsk.clamp.b32 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(max(b - a, 0)));
  return m;
}

// What a warp's rows see of a tile, chunk by chunk: bit ch of `partial` set if
// some row sees some but not every key of it, of `none` if no row sees one.
// bits: the row's visible keys.  A mask costs only the chunks it cuts, and
// keys that no row of the warp sees cost nothing.
struct TileMask {
  uint32_t bits[kChunks];
  uint32_t partial, none;
};
__device__ __forceinline__ void classify(TileMask& k) {
  k.partial = k.none = 0u;
#pragma unroll
  for (int ch = 0; ch < kChunks; ++ch) {
    if (!__any_sync(0xffffffffu, k.bits[ch] != 0u)) k.none |= 1u << ch;
    else if (!__all_sync(0xffffffffu, k.bits[ch] == 0xffffffffu)) k.partial |= 1u << ch;
  }
}

// `fill` at the row's masked keys of chunk ch.  Tests of single bits of a word
// cost one instruction for several predicates, against two comparisons a key.
__device__ __forceinline__ void mask_chunk(Row& v, int ch, uint32_t bits, uint32_t fill) {
#pragma unroll
  for (int e = 0; e < 32; ++e) v[ch * 32 + e] = (bits & (1u << e)) ? v[ch * 32 + e] : fill;
}

// -inf at masked keys; keeps ext in step.
__device__ __forceinline__ void apply_mask(Row& v, float (&ext)[kChunks], const TileMask& k) {
#pragma unroll
  for (int ch = 0; ch < kChunks; ++ch) {
    if ((k.none >> ch) & 1u) ext[ch] = -INFINITY;
    if ((k.partial >> ch) & 1u) {
      mask_chunk(v, ch, k.bits[ch], kMinusInf);
      ext[ch] = chunk_max(v, ch);
    }
  }
}

__device__ __forceinline__ void scale_row(Row& v, float (&ext)[kChunks], float c) {
  const uint64_t c2 = f2_pack(c, c);
#pragma unroll
  for (int e = 0; e < kTileKeys; e += 2) set_pair(v, e, f2_mul(pair_of(v, e), c2));
#pragma unroll
  for (int ch = 0; ch < kChunks; ++ch) ext[ch] = chunk_max(v, ch);
}

// Raw scores to capped base-2 logits, cap2 tanh(y / cap), and ext with them.
// Where every |y / cap| of the warp's rows is at most 0.6 (the usual case: a
// cap is far above most scores) the tanh is an odd polynomial of degree 9 in
// s (mod_common.cuh), 3 instructions a score and nothing for the
// multifunction unit.  Otherwise cap2 - 2 cap2 / (1 + E) with one reciprocal
// for four scores, 1 + E kept below 2^30 so that four multiply without
// overflow (the tanh is 1 to the last bit long before).
// Masked scores, which may hold anything, are set to 0 first.
__device__ __forceinline__ void cap_row(Row& v, float (&ext)[kChunks], const CapArgs& cap, bool masked,
                                        const TileMask& k) {
  if (masked) {
#pragma unroll
    for (int ch = 0; ch < kChunks; ++ch)
      if (((k.partial | k.none) >> ch) & 1u) {
        mask_chunk(v, ch, k.bits[ch], 0u);
        ext[ch] = chunk_max(v, ch);
      }
  }
  if (__all_sync(0xffffffffu, max4(ext) <= cap.s_max && row_min(v) >= -cap.s_max)) {
    const uint64_t k0 = f2_pack(cap.k[0], cap.k[0]), k1 = f2_pack(cap.k[1], cap.k[1]),
                   k2 = f2_pack(cap.k[2], cap.k[2]), k3 = f2_pack(cap.k[3], cap.k[3]),
                   k4 = f2_pack(cap.k[4], cap.k[4]);
#pragma unroll
    for (int e = 0; e < kTileKeys; e += 2) {
      const uint64_t s = pair_of(v, e), u = f2_mul(s, s);
      const uint64_t q = f2_fma(f2_fma(f2_fma(f2_fma(k4, u, k3), u, k2), u, k1), u, k0);
      set_pair(v, e, f2_mul(q, s));
    }
#pragma unroll
    for (int ch = 0; ch < kChunks; ++ch) ext[ch] = cap_small(ext[ch], cap);
  } else {
    const uint64_t c1 = f2_pack(cap.c1, cap.c1), one = f2_pack(1.f, 1.f);
    const uint64_t mul = f2_pack(-2.f * cap.cap2, -2.f * cap.cap2), add = f2_pack(cap.cap2, cap.cap2);
#pragma unroll
    for (int e = 0; e < kTileKeys; e += 4) {
      float z0, z1, z2, z3, px, py;
      f2_unpack(f2_mul(pair_of(v, e), c1), z0, z1);
      f2_unpack(f2_mul(pair_of(v, e + 2), c1), z2, z3);
      const uint64_t ua = f2_add(f2_pack(ex2_approx(min30(z0)), ex2_approx(min30(z1))), one);
      const uint64_t ub = f2_add(f2_pack(ex2_approx(min30(z2)), ex2_approx(min30(z3))), one);
      f2_unpack(f2_mul(ua, ub), px, py);  // u0 u2, u1 u3
      const float q = rcp_approx(px * py);
      const uint64_t r = f2_mul(f2_pack(q, q), f2_pack(py, px));  // 1 / (u0 u2), 1 / (u1 u3)
      set_pair(v, e, f2_fma(f2_mul(r, ub), mul, add));
      set_pair(v, e + 2, f2_fma(f2_mul(r, ua), mul, add));
    }
#pragma unroll
    for (int ch = 0; ch < kChunks; ++ch) ext[ch] = chunk_max(v, ch);
  }
}

// P = 2^(v cm + neg) in 16 bits over the first 64 columns of the row's scores,
// and its sum.  Chunks of `none` are zeros.
template <bool kF16>
__device__ __forceinline__ float exp_row(const Row& v, float cm, float neg, uint32_t s_addr, uint32_t none) {
  const uint64_t cm2 = f2_pack(cm, cm), nm2 = f2_pack(neg, neg);
  uint64_t rs_a = 0, rs_b = 0;  // packed partial sums (bit pattern 0 = 0.0f)
#pragma unroll
  for (int ch = 0; ch < kChunks; ++ch) {
    uint32_t pk[16];
    if ((none >> ch) & 1u) {
#pragma unroll
      for (int e = 0; e < 16; ++e) pk[e] = 0u;
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float x0, x1;
        f2_unpack(f2_fma(pair_of(v, ch * 32 + 2 * e), cm2, nm2), x0, x1);
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
// The stores issued by this thread are done.
__device__ __forceinline__ void tma_store_drain() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace osattn
