// mod_common.cuh - what the modified-score attention kernels share: the mask
// plan's layout, the score modes and the distance-bias table in shared memory.
//
// Logits (base e) of query row i of head h and key j, raw score s = <q, k>:
//   y = scale s;  y = cap tanh(y / cap) if capped;
//   y -= slopes[h] |j - p|                  (slopes), or
//   y += table[map[clamp(j - p, -R, R) + R]][h]   (learned biases by bucket),
// with p = i + q_offset the query's position among the keys; key j counts iff
// lo_i <= j < hi_i.  The kernels work in base 2 (everything times log2 e).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mod_internal.h"
#include "sm100_ptx.cuh"

namespace osattn {

constexpr float kModLog2e = 1.4426950408889634f;

// Score modes, a template argument of the kernels.  A mode is compiled for
// each pair that a call can ask for; a cap together with a learned bias is
// refused by the entry points (its backward pass would have to hold two
// factors per score in registers).
enum ScoreMode : int {
  kModPlain = 0,
  kModCap = 1,
  kModSlopes = 2,
  kModCapSlopes = 3,
  kModRel = 4,
  kModRelWide = 5  // forward and dQ at d = 128: ranges above kSmallRel
};
// Up to this range the table fits beside five K/V stages at d = 128 (180 would);
// 128 is where tables of bucketed distances commonly end.
constexpr int kSmallRel = 128;
__host__ __device__ constexpr bool mode_cap(int m) { return m == kModCap || m == kModCapSlopes; }
__host__ __device__ constexpr bool mode_slopes(int m) { return m == kModSlopes || m == kModCapSlopes; }
__host__ __device__ constexpr bool mode_rel(int m) { return m == kModRel || m == kModRelWide; }

// Mask plan: per 128-row query tile {smallest lo, largest hi, largest lo,
// smallest hi} (the first two over the rows that see a key, 0 and 0 if none
// does), [B][tiles]; then per query row {lo, hi}, [B][Nq], {0, 0} for a row
// that sees nothing.  Keys number at most 2^30; bit 30 of the third entry says
// that no row of the tile sees a key behind its own position.
constexpr int kPlanLeft = 1 << 30;
struct PlanView {
  const int4* tiles;  // null: every row sees [0, Nkv)
  const int2* rows;
};
struct PlanTile {
  int lo, hi, lo_max, hi_min;
  bool left;
};

__device__ __forceinline__ int4 plan_load(const PlanView& pv, int b, int n_tiles, int tile, int Nkv) {
  if (!pv.tiles) return make_int4(0, Nkv, 0, Nkv);
  return pv.tiles[static_cast<long long>(b) * n_tiles + tile];
}
__device__ __forceinline__ PlanTile plan_entry(int4 t) {
  return PlanTile{t.x, t.y, t.z & (kPlanLeft - 1), t.w, (t.z & kPlanLeft) != 0};
}
__device__ __forceinline__ PlanTile plan_tile(const PlanView& pv, int b, int n_tiles, int tile, int Nkv) {
  return plan_entry(plan_load(pv, b, n_tiles, tile, Nkv));
}

__device__ __forceinline__ int2 plan_row(const PlanView& pv, int b, int Nq, int i, int Nkv) {
  if (i >= Nq) return make_int2(0, 0);
  if (!pv.rows) return make_int2(0, Nkv);
  return pv.rows[static_cast<long long>(b) * Nq + i];
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Orders this thread's earlier shared-memory writes before later reads of
// them by the async proxy (tcgen05 MMAs, TMA).
__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Capped scores: with E = e^{2 y / cap} and r = 1 / (1 + E),
// tanh(y / cap) = 1 - 2 r, so cap tanh(y / cap) = cap - 2 cap r.  One ex2 and
// one reciprocal.  E is off by 2^-22 relative and the rounding of its exponent
// (2^-24 of at most 30), which moves r by a fourth of that at most; 1 + E, the
// reciprocal and, where four scores share one, four products add 2^-21 of r: in
// all below 2^-20 of the cap (seen: 2^-22), whatever the score.  That is 5e-5 in
// a logit at cap 50, where the one-instruction tanh (relative error 2^-11) would
// move it by 0.02.  E = inf gives r = 0.
// c1 = 2 scale log2(e) / cap.
__device__ __forceinline__ float cap_r(float s, float c1) { return rcp_approx(1.f + ex2_approx(s * c1)); }

// A cap's constants.  For |y / cap| <= 0.4, tanh(z) = z t(z^2) with t of degree
// 3: coefficients fitted here for the least relative error on that range
// (2^-23.3, reweighted least squares on Chebyshev points).  k[n] carries
// cap2 (scale / cap)^(2 n + 1), so that the polynomial is in the raw score:
// cap2 tanh = s (k0 + s^2 (k1 + ...)).  Degree 2 (2^-23.2) does up to 0.2.  s_max = 0.4 cap / |scale|, but at most
// 2^16 where |scale| / cap is below 2^-19 (k[3] leaves fp32's range there, and
// is not needed up to 2^16), and -1 where it is above 2^12: then only the
// other form is used.  c1 is kept finite (inf times a score of 0 is NaN).
struct CapArgs {
  float c1, cap2, s_max;  // c1 = 2 scale log2(e) / cap
  float inv2;             // 1 / cap2^2
  float k[4];
  float q[3];             // the same of degree 2, for |y / cap| <= 0.2, that is up to s_max / 2
  bool large;             // the cap is above 64
  float s_free;           // up to here, s_max / 2 at most, logits are within free_logits: 2^x needs no max
};
// Logits (base 2) of either sign that a tile may have to be formed against
// free_max or any greater max instead of its own, so that P stays below 2^15 and
// keeps the type's precision: bf16 has the exponents for 2^-15, but fp16 is at its
// smallest normal value 2^-14 with it.  There a tile's 128 P of 2^-7 or more sum
// to at least 1, as they do against their own max, and what is below fp16's
// smallest step beside them is as small a part of the row.
__host__ __device__ constexpr float free_logits(bool fp16) { return fp16 ? 11.f : 15.f; }
__host__ __device__ constexpr float free_max(bool fp16) { return fp16 ? -4.f : 0.f; }
inline CapArgs make_cap(float scale, float softcap, bool fp16) {
  CapArgs c{};
  if (!(softcap > 0.f)) return c;
  const double a = static_cast<double>(scale) / softcap;  // the tanh is odd: either sign
  c.large = softcap > 64.f;
  const double cap2 = static_cast<double>(softcap) * 1.4426950408889634;
  const double c1 = 2.0 * a * 1.4426950408889634;
  c.c1 = static_cast<float>(c1 > 3e38 ? 3e38 : c1 < -3e38 ? -3e38 : c1);
  c.cap2 = static_cast<float>(cap2);
  c.inv2 = static_cast<float>(1.0 / (cap2 * cap2));
  const double t[4] = {0.9999999019, -0.3333136247, 0.1327097680, -0.0475536037};
  const double size = a < 0 ? -a : a, low = 1.0 / 524288;
  const bool ok = size <= 4096.0;
  c.s_max = !ok ? -1.f : (size < low ? 65536.f : static_cast<float>(0.4 / size));
  const double t2[3] = {0.9999998948, -0.3332859090, 0.1301540755};
  const double unit = (scale < 0 ? -scale : scale) * 1.4426950408889634;  // logit of a score of 1
  const double free = free_logits(fp16) / unit;
  c.s_free = static_cast<float>(free < 0.5 * c.s_max ? free : 0.5 * c.s_max);
  double pw = a;
  for (int n = 0; n < 4; ++n, pw *= a * a) {
    c.k[n] = ok ? static_cast<float>(cap2 * t[n] * pw) : 0.f;
    if (n < 3) c.q[n] = ok ? static_cast<float>(cap2 * t2[n] * pw) : 0.f;
  }
  return c;
}
// min(x, 30); NaN stays NaN
__device__ __forceinline__ float min30(float x) {
  float y;
  asm("min.NaN.f32 %0, %1, 0f41F00000;" : "=f"(y) : "f"(x));
  return y;
}

// The kernels that negate an MMA operand for a negative scale work with its
// magnitude; 0 becomes a value whose products with finite scores vanish but
// that keeps -inf (a masked score) what it is.
inline float positive_scale(float scale) {
  const float a = scale < 0.f ? -scale : scale;
  return a > 1e-30f ? a : 1e-30f;
}
// Instruction descriptor bit that negates A.
constexpr uint32_t kIdescNegA = 1u << 13;

// mma_abt with the instruction descriptor given.
template <int KD>
__device__ __forceinline__ void mma_abt_id(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t id) {
  mma_ss_k<0, true>(d_tmem, a_desc, b_desc, id);
#pragma unroll
  for (int kk = 1; kk < KD / 16; ++kk) {
    const uint32_t off = static_cast<uint32_t>(((kk / 4) * (128 * 128) + (kk % 4) * 32) >> 4);
    mma_ss_k<1, true>(d_tmem, sdesc_add(a_desc, off), sdesc_add(b_desc, off), id);
  }
}

// Slopes on the tensor cores.  For keys on one side of a query,
// -slope |j - p| = +-slope (j - p) is linear in the key's place e in its tile;
// with one more MMA step of 16 inner elements, whose operands hold (hi, mid,
// lo, 0 ...) of slope / (2 scale) in each query row and (e, e, e, 0 ...) in key
// row e, twice, the scores come out as s +- (slope / scale) e and what is left
// of the bias is one constant per row and tile.  hi + mid + lo carry the
// quotient to 2^-24 in bf16 (three 8-bit pieces; fp16: to its smallest step),
// e < 128 is exact, and the products are summed in fp32 as s is.  Tiles with
// keys on both sides of a row that sees them get the bias score by score.
// The operands are 8 x 16-byte core matrices without swizzle; the other 8
// inner elements read the same matrix again (stride 0, hence the half), and
// so do all row groups where every query row is alike.
constexpr int kSlopeQBytes = 128;       // alike query rows: one core matrix
constexpr int kSlopeRowsBytes = 128 * 16;  // 128 different rows, of queries or keys
// Beyond either: score by score.  The sum s + (slope / scale) e is rounded to fp32
// before the constant is taken off, an error of 2^-23 of 128 |slope| in the logit of
// a key beside its query: 2e-5 at slope 1, where the common slopes end, but 1e-3 at
// 32.  (The quotient's pieces have to fit fp16.)
constexpr float kSlopeMax = 1.f, kSlopeScaledMax = 16384.f;

// Descriptor of rows of 8 elements read twice; sbo: to the next 8 rows.
__device__ __forceinline__ uint64_t sdesc_plain(uint32_t smem_addr, uint32_t sbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(sbo >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}
__device__ __forceinline__ uint64_t slope_q_desc(uint32_t at) { return sdesc_plain(at, 0); }
__device__ __forceinline__ uint64_t slope_rows_desc(uint32_t at) { return sdesc_plain(at, 128); }

__device__ __forceinline__ bool slope_linear(float slope, float scale) {
  return fabsf(slope) <= kSlopeMax && fabsf(slope / scale) <= kSlopeScaledMax;
}

template <bool kF16>
__device__ __forceinline__ uint16_t to_16(float x) {
  if constexpr (kF16) return __half_as_ushort(__float2half_rn(x));
  else return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}
template <bool kF16>
__device__ __forceinline__ float from_16(uint16_t w) {
  if constexpr (kF16) return __half2float(__ushort_as_half(w));
  else return __bfloat162float(__ushort_as_bfloat16(w));
}

// Write one row of a query or key operand (row 0 .. 7 where query rows are
// alike); the caller orders the writes before the MMAs (fence_proxy_async, then
// a barrier).
template <bool kF16>
__device__ __forceinline__ void slope_fill_q(uint8_t* at, int row, float slope, float scale) {
  uint16_t w[3];
  float rest = slope_linear(slope, scale) ? 0.5f * (slope / scale) : 0.f;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    w[i] = to_16<kF16>(rest);
    rest -= from_16<kF16>(w[i]);
  }
  reinterpret_cast<uint4*>(at)[row] = make_uint4(w[0] | (static_cast<uint32_t>(w[1]) << 16), w[2], 0u, 0u);
}
template <bool kF16>
__device__ __forceinline__ void slope_fill_k(uint8_t* at, int row) {
  const uint32_t e = to_16<kF16>(static_cast<float>(row));
  reinterpret_cast<uint4*>(at)[row] = make_uint4(e | (e << 16), e, 0u, 0u);
}

// Which side of a tile's rows its keys k0 .. k0 + 127 lie on: 1 before or at
// (j <= p), -1 behind or at, 0 both.  p0: position of the tile's first row of
// 128; `left`: no row of the tile sees a key behind its position.
__device__ __forceinline__ int slope_side(int k0, int p0, bool left) {
  if (left || k0 + 127 <= p0) return 1;
  return k0 >= p0 + 127 ? -1 : 0;
}

// Bias by distance in shared memory, in base-2 units: entry j - p + R + kRelPad
// holds table[map[clamp(j - p)]][h] * log2 e.  The pad lets a warp's 32 rows
// index a block of 64 keys that overlaps (-R, R) without clamping.
constexpr int kRelPad = 95;
__host__ __device__ constexpr int rel_entries(int R) { return 2 * (R + kRelPad) + 1; }

template <bool kF16>
__device__ __forceinline__ float load_16(const uint16_t* p) {
  const uint16_t w = __ldg(p);
  if constexpr (kF16) return __half2float(__ushort_as_half(w));
  else return __bfloat162float(__ushort_as_bfloat16(w));
}

// Fills bias[] with n threads (x0: 0 .. n - 1); a bucket outside [0, num) adds
// nothing.  lo, hi: the least and greatest bias this thread wrote.
template <bool kF16>
__device__ __forceinline__ void rel_fill(float* bias, const RelArgs& r, int H, int h, int x0, int n, float& lo,
                                         float& hi) {
  lo = INFINITY;
  hi = -INFINITY;
  for (int x = x0; x < rel_entries(r.range); x += n) {
    const int at = min(max(x - kRelPad, 0), 2 * r.range);
    const int bucket = __ldg(r.map + at);
    float v = 0.f;
    if (bucket >= 0 && bucket < r.num)
      v = load_16<kF16>(static_cast<const uint16_t*>(r.table) + static_cast<long long>(bucket) * H + h);
    v *= kModLog2e;
    bias[x] = v;
    lo = v == v ? fminf(lo, v) : -INFINITY;  // NaN: no bound holds
    hi = v == v ? fmaxf(hi, v) : INFINITY;
  }
}

}  // namespace osattn
