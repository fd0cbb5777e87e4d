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
enum ScoreMode : int { kModPlain = 0, kModCap = 1, kModSlopes = 2, kModCapSlopes = 3, kModRel = 4 };
__host__ __device__ constexpr bool mode_cap(int m) { return m == kModCap || m == kModCapSlopes; }
__host__ __device__ constexpr bool mode_slopes(int m) { return m == kModSlopes || m == kModCapSlopes; }
__host__ __device__ constexpr bool mode_rel(int m) { return m == kModRel; }

// Mask plan: per 128-row query tile {smallest lo, largest hi, largest lo,
// smallest hi} (the first two over the rows that see a key, 0 and 0 if none
// does), [B][tiles]; then per query row {lo, hi}, [B][Nq], {0, 0} for a row
// that sees nothing.
struct PlanView {
  const int4* tiles;  // null: every row sees [0, Nkv)
  const int2* rows;
};

__device__ __forceinline__ int4 plan_tile(const PlanView& pv, int b, int n_tiles, int tile, int Nkv) {
  if (!pv.tiles) return make_int4(0, Nkv, 0, Nkv);
  return pv.tiles[static_cast<long long>(b) * n_tiles + tile];
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
// one reciprocal; the error of r (about 2^-23 relative, r <= 1) moves the
// logit by at most 2 cap 2^-23, 1e-5 at cap 50, while the one-instruction
// tanh (relative error 2^-11) would move it by 0.02.  E = inf gives r = 0.
// c1 = 2 scale log2(e) / cap.
__device__ __forceinline__ float cap_r(float s, float c1) { return rcp_approx(1.f + ex2_approx(s * c1)); }

// Bias by distance in shared memory, in base-2 units: entry j - p + R + kRelPad
// holds table[map[clamp(j - p)]][h] * log2 e.  The pad lets a thread index a
// whole 128-key tile that overlaps (-R, R) without clamping.
constexpr int kRelPad = 255;
__host__ __device__ constexpr int rel_entries(int R) { return 2 * (R + kRelPad) + 1; }

template <bool kF16>
__device__ __forceinline__ float load_16(const uint16_t* p) {
  const uint16_t w = __ldg(p);
  if constexpr (kF16) return __half2float(__ushort_as_half(w));
  else return __bfloat162float(__ushort_as_bfloat16(w));
}

// Fills bias[] with all threads of the block; a bucket outside [0, num) adds
// nothing.
template <bool kF16>
__device__ __forceinline__ void rel_fill(float* bias, const RelArgs& r, int H, int h) {
  for (int x = threadIdx.x; x < rel_entries(r.range); x += blockDim.x) {
    const int at = min(max(x - kRelPad, 0), 2 * r.range);
    const int bucket = __ldg(r.map + at);
    float v = 0.f;
    if (bucket >= 0 && bucket < r.num)
      v = load_16<kF16>(static_cast<const uint16_t*>(r.table) + static_cast<long long>(bucket) * H + h);
    bias[x] = v * kModLog2e;
  }
}

}  // namespace osattn
