// bwd_mod_tcgen05.cuh - gradients of the modified-score attention forward
// (fwd_mod_tcgen05.cuh) on the tcgen05 tensor cores.  Built for sm_103a; bf16
// or fp16, d = 64 or 128.
//
// With P = e^{y - LSE} on the keys a row sees, dP = dO V^T, D = rowsum(dO O):
//   dY = P (dP - D)               (gradient of the modified score)
//   dS = dY (1 - tanh^2)          (capped scores; dS = dY otherwise)
//   dQ = scale dS K,  dK = scale sum dS^T Q,  dV = sum P^T dO,
// the sums of dK and dV running over the query heads that share the key head,
// and dTable[k][h] = sum of dY over the pairs whose distance has bucket k.
//
// Launches, in order on one stream:
//   dq_kernel    one CTA per 128-row query tile; K and V tiles stream.  Also
//                writes D, without a cap corrected by the row's sum of dY (for
//                dK and dTable; 2 % of a step, and bf16 gradients of a learned
//                bias are off by 0.0015 to 0.0017 of their size, the rounding
//                of the result, in place of 0.003 to 0.004).
//   dkdv_kernel  one CTA per 128-key tile of a key head; the query tiles of
//                every head of its group that can see those keys stream, so
//                the sums over heads stay in tensor memory and nothing is
//                added by atomics: results do not depend on the order of CTAs.
//                Where key tiles are few, a cluster of 2, 4 or 8 CTAs shares
//                one's (head, query tile) pairs and adds its fp32 sums through
//                distributed shared memory in rank order (dkdv_split.h; B1 H8 kv2
//                1078 d64 capped, no mask: whole step 173 -> 84 us).
//                With a learned bias also the sums of dY by distance, here and
//                not in dq_kernel since there is shared memory to spare (there
//                it cost a K slot, 0.35 us a tile at d = 128).
//   rel_reduce   folds the partial sums by distance into the table's buckets.
// P and dS are rounded to 16 bits as MMA operands (the tensor core's operand
// width, half a step of the outputs' type each), everything is summed in fp32.
// D is formed from the 16-bit O that the caller has: a row's dY then miss their
// sum of 0 by dO times O's rounding, as much again in dQ as the rounding of dS
// (bf16: 0.0027 to 0.003 of its size together; dK 0.0024).
//
// CTA layout (384 threads): warps 0-7 elementwise in two warpgroups, group g
// taking columns 64g .. 64g + 63 of every score tile, one tile row a thread;
// warp 8 TMA producer; warp 9 issues the MMAs; 10 and 11 fill the warpgroup
// whose registers the others take (216 for the elementwise warps: 2 % faster
// than the 168 of an even share, which spill).  Tensor memory, dkdv:
// [0, 128) S^T, [128, 256) dP^T, then dV and dK, at d = 64 a second S^T; dq: two S buffers, dP, dQ.
//
// Masked places hold anything: their P and dY are selected to 0, never
// multiplied, and rows of K (dq) or of Q and dO (dkdv) that take part in no
// pair are zeroed in shared memory before they enter a product.
//
// What bounds it: the elementwise work, by issue and latency, as in the
// forward pass: 1.2 us a 128 x 128 tile in dq_kernel and 1.8 in dkdv_kernel
// at d = 128 without masks, where the 3 and 4 products take 0.75 and 1.0.
// Measured (dq, dkdv), bf16, kernel times:
//   B2 H16 kv4 4096 d128 window 1024 cap 50    131, 177 us
//   B1 H16 8192 d128 documents of about 700    114, 136 us
//   B1 H16 4096 d128 learned bias, no mask     169, 232 us (1220 and 1190 TFLOP/s
//     as executed; 860 together for the 5 products that the mathematics asks for)
//   B8 H12 512 d64 learned bias                 28,  48 us;  table sums 5 us
//   B4 H8 kv2 381 d64 fp16 prefix                8,  14 us
//   B4 H16 2048 d128 causal: plain 116, 136; cap 135, 172; slopes 124, 156; cap and
//     slopes 158, 207 us;  d64: 88, 101; 111, 139; 97, 120; 133, 170 us
#pragma once

#include <cmath>
#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dkdv_split.h"
#include "mod_common.cuh"
#include "mod_internal.h"
#include "sm100_ptx.cuh"
#include "softmax_tile.cuh"
#include "tc_attn_mma.cuh"

namespace osattn {
namespace bwdmod {

constexpr int kT = 128;
constexpr int kThreads = 384;
constexpr int kProdWarp = 8, kMmaWarp = 9;
constexpr uint32_t kCols = 512;

enum : uint32_t { kSiteLoad = 61, kSiteMma = 62, kSiteElem = 63, kSiteEpi = 64, kSiteSync = 65 };

// Sums of dY by distance: entry distance + R + kSumPad, padded so that a whole
// 128 x 128 tile that overlaps (-R, R) is indexed without clamping.
constexpr int kSumPad = 255;
__host__ __device__ constexpr int sum_entries(int R) { return 2 * (R + kSumPad) + 1; }

template <int HD, int MODE>
struct Cfg {
  static constexpr int kTileBytes = kT * HD * 2;
  // table of learned biases, or the slope operands
  static constexpr int kTableBytes = mode_rel(MODE) ? (rel_entries(kMaxRelRange) * 4 + 15) / 16 * 16
                                                    : (MODE == kModSlopes ? kSlopeRowsBytes + 4 * kSlopeQBytes : 0);
  // dkdv: K, V, kStages stages of (Q_i, dO_i), per stage LSE, D, lo, hi, then
  // the table, the sums by distance and the warps' diagonal strips
  static constexpr int kStages = HD == 128 ? 2 : 4;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kDkdvRows = 2 * kTileBytes + kStages * kStageBytes;
  static constexpr int kDkdvTable = kDkdvRows + kStages * kT * 16;
  static constexpr int kDkdvSums = kDkdvTable + kTableBytes;
  static constexpr int kSumBytes = mode_rel(MODE) ? (sum_entries(kMaxRelRange) * 4 + 15) / 16 * 16 : 0;
  static constexpr int kStripBytes = mode_rel(MODE) ? 2 * 8 * 96 * 4 : 0;
  static constexpr int kDkdvRegion = kDkdvSums + kSumBytes + kStripBytes;
  // dq: Q, dO, kKSlots K tiles, kVSlots V tiles (K_j is read until dQ_j, V_j
  // until dP_j), then the table: at d = 128 a range above kSmallRel
  // (kModRelWide) takes the third K tile's place.  The slopes' key operand has
  // 64 rows here, used for each half of a tile.
  static constexpr int kKSlots = HD == 128 ? (MODE == kModRelWide ? 2 : 3) : 4;
  static constexpr int kVSlots = HD == 128 ? 2 : 4;
  static constexpr int kDqTable = (2 + kKSlots + kVSlots) * kTileBytes;
  static constexpr int kDqTableBytes =
      MODE == kModSlopes ? kSlopeRowsBytes / 2 + kSlopeQBytes
                         : (MODE == kModRel && HD == 128 ? (rel_entries(kSmallRel) * 4 + 15) / 16 * 16 : kTableBytes);
  static constexpr int kDqRegion = kDqTable + kDqTableBytes;
  static constexpr uint32_t kColAcc0 = 256;       // dV
  static constexpr uint32_t kColAcc1 = 256 + HD;  // dK
  // dkdv: tensor memory has room for a second S^T tile at d = 64; place, column
  // and phase of tile it
  static constexpr bool kTwoS = HD == 64;
  __device__ static constexpr int s_of(int it) { return kTwoS ? it & 1 : 0; }
  __device__ static constexpr uint32_t s_col(int it) { return s_of(it) ? 384u : 0u; }
  __device__ static constexpr uint32_t s_phase(int it) { return static_cast<uint32_t>(kTwoS ? it >> 1 : it) & 1u; }
};

struct __align__(16) Bars {
  uint64_t fixed_full;
  uint64_t full[4];
  uint64_t empty[4];
  uint64_t empty2[4];
  uint64_t s_full[2];
  uint64_t dp_full;
  uint64_t p_full[2];             // of S^T tile 0, 1: a warp may be a tile ahead of another
  uint64_t ds_full;
  uint64_t acc_full;
  uint64_t mma_drain;
  uint64_t d_full;
  uint64_t elem;
  uint64_t staged[2];             // an output tile is in shared memory (dq: 256, dkdv: 128 arrivals)
  uint32_t tmem_base;
  int abort_flag;
  int it_lo, it_hi;
  int side[4];                    // dkdv: slope_side of the stage's query tile, 0 if not linear
  int seen[4];                    // dkdv: bit 0 every query sees every key, bit 1 some query sees none
  float d_part[kT];        // dq: D, added by the two groups (0 + a + b: the order does not matter)
  float far_part[2][8];    // dkdv: sums of dY beyond the range, by warp
};

template <int HD, int MODE>
constexpr int dkdv_smem_bytes() {
  return Cfg<HD, MODE>::kDkdvRegion + static_cast<int>(sizeof(Bars));
}
template <int HD, int MODE>
constexpr int dq_smem_bytes() {
  return Cfg<HD, MODE>::kDqRegion + static_cast<int>(sizeof(Bars));
}

struct Params {
  const float* LSE;
  float* D;
  const uint16_t* O;
  long long o_s[3];
  PlanView plan;
  int H, Hkv, group, Nq, Nkv;
  int q_tiles;      // 128-row query tiles per (b, h)
  int num_tiles;    // this kernel's tiles per head
  int BH;           // this kernel's heads: B * H (dq) or B * Hkv (dkdv)
  int split_log2;   // dkdv: 2^this CTAs (a cluster) share a key tile's query tiles
  uint16_t* dkv[2];        // then: dV, dK
  long long dkv_s[2][3];
  int group_heads;  // heads per last-tile-first (dq) or first-tile-first (dkdv) group of CTAs
  float scale;
  float scale_log2;
  CapArgs cap;
  const float* slopes;
  RelArgs rel;
  float* rel_part;
  int q_offset;
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

template <bool kF16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if constexpr (kF16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

__device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > limit_ns) return;
  }
}

__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t tx_bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(tx_bytes)
               : "memory");
}

// Barrier over a cluster's CTAs, with their shared memory in order.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four floats at `at` (an address of this CTA) in the shared memory of CTA `rank`.
__device__ __forceinline__ void cluster_load4(uint32_t at, int rank, float* v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
      : "r"(at), "r"(rank)
      : "memory");
}

// Barrier over the 256 elementwise threads, bounded like every other wait
// (a warp that gave up elsewhere must not leave the rest waiting).  phase
// counts the barrier's uses; false: give up.
__device__ __forceinline__ bool elem_sync(Bars* bars, uint32_t& phase, const WaitCtl& wc) {
  mbar_arrive(&bars->elem);
  const bool ok = mbar_wait(&bars->elem, phase & 1u, wc, kSiteSync);
  ++phase;
  return __all_sync(0xffffffffu, ok);
}

// The head and the rank by length (0 = longest under a causal mask) of this
// CTA's tile: heads in groups whose streamed tiles fit in L2 together.
__device__ __forceinline__ void unit_of(const Params& p, int unit, int& bh, int& rank) {
  const int nt = p.num_tiles, G = p.group_heads;
  const int g0 = (unit / (G * nt)) * G;
  const int gsize = min(G, p.BH - g0);
  const int r = unit - g0 * nt;
  bh = g0 + r % gsize;
  rank = r / gsize;
}

// NC fp32 tensor-memory columns of one tile row, starting at taddr, times
// `mul`, as 16-bit values into an output tile in shared memory from column
// col0 (zeros when has_acc is false).
template <int NC, bool kF16>
__device__ __forceinline__ void stage_out(uint8_t* tile, int row, int col0, uint32_t taddr, bool has_acc,
                                          float mul) {
#pragma unroll
  for (int ch = 0; ch < NC / 32; ++ch) {
    uint32_t r[32];
    if (has_acc) {
      tmem_ld_32x32b_x32(taddr + ch * 32, r);
      tmem_ld_wait();
      reg_fence32(r);
    } else {
#pragma unroll
      for (int e = 0; e < 32; ++e) r[e] = 0u;
    }
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e)
      pk[e] = pack2<kF16>(__uint_as_float(r[2 * e]) * mul, __uint_as_float(r[2 * e + 1]) * mul);
    stage_row32(tile, row, col0 + ch * 32, pk);
  }
}

// Zeroes row `row` of a 128-row tile in shared memory, column block cb only.
__device__ __forceinline__ void zero_row(uint8_t* tile, int cb, int row) {
  uint4* r = reinterpret_cast<uint4*>(tile + cb * kT * 128 + row * 128);
#pragma unroll
  for (int x = 0; x < 8; ++x) r[x] = make_uint4(0u, 0u, 0u, 0u);
}

// P part over the 64 columns of this thread's group at tile column c0:
// P = 2^(x - LSE log2 e) with x the modified score; kMask selects 0 where
// vis(column) is false.  nl2of4(column): -LSE log2 e of 4 columns, with the
// constant part of the bias.  kBias adds bias(column), score by score.
// kWriteP writes the 16-bit P over columns c0 .. c0 + 31.  On return pr holds
// what dS is made of: P, times 1 - tanh^2 where scores are capped.  (A cap
// takes the polynomial where the 32 scores at hand allow it, see CapArgs.)
template <bool kF16, int MODE, bool kWriteP, bool kMask, bool kBias, typename Vis, typename L2of4,
          typename Bias>
__device__ __forceinline__ void p_part(uint32_t s_addr, int c0, const Params& p, Vis&& vis, L2of4&& nl2of4,
                                       Bias&& bias, float (&pr)[64]) {
  constexpr bool kCap = mode_cap(MODE);
  Chunk sa, sb;
  float ta = 0.f, tb = 0.f;
  if constexpr (kCap) tmem_ld_absmax_32(s_addr + c0, sa, ta);
  else tmem_ld_32x32b_x32(s_addr + c0, sa);
  tmem_ld_wait();
  reg_fence32(sa);
  asm volatile("" : "+f"(ta));
  if constexpr (kCap) tmem_ld_absmax_32(s_addr + c0 + 32, sb, tb);
  else tmem_ld_32x32b_x32(s_addr + c0 + 32, sb);
  const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
  auto half = [&](Chunk& sv, float size, int h) {
    uint32_t pk[16];
    bool small = true, tiny = false;
    if constexpr (kCap) {
      if constexpr (kMask) {  // masked scores, which may hold anything, take no part in the choice
#pragma unroll
        for (int e = 0; e < 32; ++e) sv[e] = vis(c0 + 32 * h + e) ? sv[e] : 0u;
        size = fmaxf(chunk_max(sv), -chunk_min(sv));
      }
      small = __all_sync(0xffffffffu, size <= p.cap.s_max);
      tiny = __all_sync(0xffffffffu, size <= 0.5f * p.cap.s_max);
    }
    auto finish = [&](int x, uint64_t a2, uint64_t f2) {  // entries x, x + 1 of the half: exponent, factor
      const int col = c0 + 32 * h + x;
      if constexpr (kBias) a2 = f2_add(a2, f2_pack(bias(col), bias(col + 1)));
      float a0, a1;
      f2_unpack(a2, a0, a1);
      float e0 = ex2_approx(a0), e1 = ex2_approx(a1);
      if constexpr (kMask) {
        e0 = vis(col) ? e0 : 0.f;
        e1 = vis(col + 1) ? e1 : 0.f;
      }
      if constexpr (kWriteP) pk[x / 2] = pack2<kF16>(e0, e1);
      if constexpr (kCap) f2_unpack(f2_mul(f2_pack(e0, e1), f2), e0, e1);
      pr[32 * h + x] = e0;
      pr[32 * h + x + 1] = e1;
    };
    auto direct = [&](auto degree) {
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const float4 L = nl2of4(c0 + 32 * h + 4 * g);
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
          const int x = 4 * g + u;
          const uint64_t s2 = pair_of(sv, x), n2 = u == 0 ? f2_pack(L.x, L.y) : f2_pack(L.z, L.w);
          if constexpr (kCap) {
            const CapArgs& a = p.cap;
            const uint64_t w = f2_mul(s2, s2);
            uint64_t q;
            if constexpr (decltype(degree)::value == 2)
              q = f2_fma(f2_fma(f2_pack(a.q[2], a.q[2]), w, f2_pack(a.q[1], a.q[1])), w, f2_pack(a.q[0], a.q[0]));
            else
              q = f2_fma(f2_fma(f2_fma(f2_pack(a.k[3], a.k[3]), w, f2_pack(a.k[2], a.k[2])), w,
                                f2_pack(a.k[1], a.k[1])),
                         w, f2_pack(a.k[0], a.k[0]));
            const uint64_t y = f2_mul(q, s2);  // cap2 tanh
            finish(x, f2_add(y, n2), f2_fma(f2_mul(y, y), f2_pack(-a.inv2, -a.inv2), f2_pack(1.f, 1.f)));
          } else {
            finish(x, f2_fma(s2, c2, n2), 0ull);
          }
        }
      }
    };
    if (kCap && tiny) {
      direct(std::integral_constant<int, 2>{});
    } else if (!kCap || small) {
      direct(std::integral_constant<int, 3>{});
    } else {
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const float4 L = nl2of4(c0 + 32 * h + 4 * g);
#pragma unroll
        for (int u = 0; u < 4; u += 2) {
          const int x = 4 * g + u;
          const float r0 = cap_r(__uint_as_float(sv[x]), p.cap.c1), r1 = cap_r(__uint_as_float(sv[x + 1]), p.cap.c1);
          const uint64_t r = f2_pack(r0, r1), n2 = u == 0 ? f2_pack(L.x, L.y) : f2_pack(L.z, L.w);
          const uint64_t y = f2_fma(r, f2_pack(-2.f * p.cap.cap2, -2.f * p.cap.cap2), f2_pack(p.cap.cap2, p.cap.cap2));
          // 1 - tanh^2 = 4 r (1 - r)
          const uint64_t f = f2_mul(f2_mul(r, f2_pack(4.f, 4.f)), f2_fma(r, f2_pack(-1.f, -1.f), f2_pack(1.f, 1.f)));
          finish(x, f2_add(y, n2), f);
        }
      }
    }
    if constexpr (kWriteP) tmem_st_32x32b_x16(s_addr + c0 + 16 * h, pk);
  };
  half(sa, ta, 0);
  tmem_ld_wait();
  reg_fence32(sb);
  asm volatile("" : "+f"(tb));
  half(sb, tb, 1);
}

// P of a group that no row of the warp sees: zeros.
template <bool kWriteP>
__device__ __forceinline__ void p_none(uint32_t s_addr, int c0, float (&pr)[64]) {
#pragma unroll
  for (int x = 0; x < 64; ++x) pr[x] = 0.f;
  if constexpr (kWriteP) {
    uint32_t z[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) z[e] = 0u;
    tmem_st_32x32b_x32(s_addr + c0, z);
  }
}

// dS part over the same 64 columns of the dP tile: dS = pr (dP - D), in 16
// bits over columns c0 .. c0 + 31; ndof4(column): -D of 4 columns.  kMask: a
// masked place (pr = 0) gives 0 whatever dP and D are.  kKeep: pr returns dS.
// kSum: sum2 gets the row's fp32 dS added, as two partial sums.
template <bool kF16, bool kMask, bool kKeep, bool kSum, typename Dof4>
__device__ __forceinline__ void ds_part(uint32_t dp_addr, int c0, Dof4&& ndof4, float (&pr)[64], uint64_t& sum2) {
  uint32_t dva[32], dvb[32];
  tmem_ld_32x32b_x32(dp_addr + c0, dva);
  tmem_ld_wait();
  reg_fence32(dva);
  tmem_ld_32x32b_x32(dp_addr + c0 + 32, dvb);
  auto chunk = [&](const uint32_t(&dv)[32], int ch) {
    uint32_t gk[16];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      const float4 D = ndof4(c0 + 32 * ch + 4 * g);
      const int x = 32 * ch + 4 * g;
      const uint64_t d01 = f2_add(
          f2_pack(__uint_as_float(dv[4 * g]), __uint_as_float(dv[4 * g + 1])), f2_pack(D.x, D.y));
      const uint64_t d23 = f2_add(
          f2_pack(__uint_as_float(dv[4 * g + 2]), __uint_as_float(dv[4 * g + 3])), f2_pack(D.z, D.w));
      float gr[4];
      f2_unpack(f2_mul(f2_pack(pr[x], pr[x + 1]), d01), gr[0], gr[1]);
      f2_unpack(f2_mul(f2_pack(pr[x + 2], pr[x + 3]), d23), gr[2], gr[3]);
      if constexpr (kMask) {
#pragma unroll
        for (int u = 0; u < 4; ++u) gr[u] = pr[x + u] == 0.f ? 0.f : gr[u];
      }
      if constexpr (kKeep) {
#pragma unroll
        for (int u = 0; u < 4; ++u) pr[x + u] = gr[u];
      }
      if constexpr (kSum) sum2 = f2_add(sum2, f2_add(f2_pack(gr[0], gr[1]), f2_pack(gr[2], gr[3])));
      gk[2 * g] = pack2<kF16>(gr[0], gr[1]);
      gk[2 * g + 1] = pack2<kF16>(gr[2], gr[3]);
    }
    tmem_st_32x32b_x16(dp_addr + c0 + 16 * ch, gk);
  };
  chunk(dva, 0);
  tmem_ld_wait();
  reg_fence32(dvb);
  chunk(dvb, 1);
}

// D (128 x N fp32) (+)= A B over 128 inner elements, A the 16-bit operand the
// two warpgroups wrote (elements 0-63 in columns 0-31 of a_tmem, 64-127 in
// 64-95), B an MN-major tile.
template <int N, bool kF16>
__device__ __forceinline__ void mma_groups(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           bool accumulate) {
  constexpr uint32_t id = idesc_f16_f32(128, N, 1, kF16);
  mma_bf16_ts<true>(d_tmem, a_tmem, b_desc, id, accumulate ? 1u : 0u);
#pragma unroll
  for (int kk = 1; kk < 8; ++kk)
    mma_ts_k<1, true>(d_tmem, a_tmem + (kk / 4) * 64 + (kk % 4) * 8,
                      sdesc_add(b_desc, static_cast<uint32_t>((kk * 2048) >> 4)), id);
}

// Whether a learned bias is one value over distances first .. last: -1 (all at
// or below -R), 1 (all at or above R), 0.
__device__ __forceinline__ int far_side(int first, int last, int R) {
  return last <= -R ? -1 : (first >= R ? 1 : 0);
}

// The slope's share of a score tile: one more step of 16 inner elements, q_at
// and k_at the operands.  Transposed tile (128 keys by 128 queries):
template <bool kF16>
__device__ __forceinline__ void add_slope_t(uint32_t s_col, uint32_t q_at, uint32_t k_at, int side) {
  if (side == 0) return;
  mma_ss_k<1, true>(s_col, slope_rows_desc(k_at), slope_q_desc(q_at),
                    idesc_f16_f32(128, 128, 0, kF16) | (side < 0 ? kIdescNegA : 0u));
}
// 128 queries by two halves of 64 keys, each counted from its own first key:
template <bool kF16>
__device__ __forceinline__ void add_slope(uint32_t s_col, uint32_t q_at, uint32_t k_at, int side) {
  if (side == 0) return;
  const uint32_t id = idesc_f16_f32(128, 64, 0, kF16) | (side < 0 ? kIdescNegA : 0u);
  mma_ss_k<1, true>(s_col, slope_q_desc(q_at), slope_rows_desc(k_at), id);
  mma_ss_k<1, true>(s_col + 64, slope_q_desc(q_at), slope_rows_desc(k_at), id);
}

// ------------------------------------------------------------------ dK, dV
template <int HD, bool kF16, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
                const __grid_constant__ CUtensorMap tmdK, const __grid_constant__ CUtensorMap tmdV,
                const Params p) {
  using C = Cfg<HD, MODE>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // see fwd_mod_kernel
    if (threadIdx.x == 0) atomicExch(p.status, 3u /* OSATTN_ERR_CUDA */);
    return;
  }
  uint8_t* sK = smem;
  uint8_t* sV = smem + C::kTileBytes;
  uint8_t* ring = smem + 2 * C::kTileBytes;  // stage s: Q_i at +0, dO_i at +kTileBytes
  float* lse2 = reinterpret_cast<float*>(smem + C::kDkdvRows);  // [stage][query]: -LSE log2 e
  float* dsum = lse2 + C::kStages * kT;                         //   -D
  int* slo = reinterpret_cast<int*>(dsum + C::kStages * kT);    //   lo, hi of the query
  int* shi = slo + C::kStages * kT;
  float* bias_all = reinterpret_cast<float*>(smem + C::kDkdvTable);  // or the slope operands
  [[maybe_unused]] float* sums = reinterpret_cast<float*>(smem + C::kDkdvSums);  // of dY by distance
  [[maybe_unused]] float* strips = reinterpret_cast<float*>(smem + C::kDkdvSums + C::kSumBytes);  // [2][8][96]
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kDkdvRegion);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  int bhk, kt;
  const int part = blockIdx.x & ((1 << p.split_log2) - 1);
  unit_of(p, blockIdx.x >> p.split_log2, bhk, kt);
  const int b = bhk / p.Hkv, hk = bhk % p.Hkv;
  const int k0 = kt * kT;
  // this thread's first query tile of the search below, on its way during the set-up
  int4 entry = static_cast<int>(threadIdx.x) < p.q_tiles ? plan_load(p.plan, b, p.q_tiles, threadIdx.x, p.Nkv)
                                                         : make_int4(0, 0, 0, 0);

  if (threadIdx.x == 0) {
    mbar_init(&bars->fixed_full, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&bars->full[s], 2);  // the dO load's expect-tx, then the Q load's arrival
      mbar_init(&bars->empty[s], 1);
      mbar_init(&bars->empty2[s], 1);
    }
    mbar_init(&bars->s_full[0], 1);
    mbar_init(&bars->s_full[1], 1);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->p_full[0], 256);
    mbar_init(&bars->p_full[1], 256);
    mbar_init(&bars->ds_full, 256);
    mbar_init(&bars->acc_full, 1);
    mbar_init(&bars->mma_drain, 1);
    mbar_init(&bars->elem, 256);
    mbar_init(&bars->staged[0], 128);
    mbar_init(&bars->staged[1], 128);
    bars->abort_flag = 0;
    bars->it_lo = p.q_tiles;
    bars->it_hi = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, kCols);
    tmem_relinquish();
  }
  if constexpr (MODE == kModSlopes) {
    if (threadIdx.x < kT) slope_fill_k<kF16>(reinterpret_cast<uint8_t*>(bias_all), threadIdx.x);
    fence_proxy_async();
  }
  __syncthreads();
  // Query tiles [it_lo, it_hi) hold every row that sees one of these keys.
  for (int q = threadIdx.x; q < p.q_tiles; q += kThreads) {
    if (entry.x < k0 + kT && entry.y > k0) {
      atomicMin(&bars->it_lo, q);
      atomicMax(&bars->it_hi, q + 1);
    }
    if (q + kThreads < p.q_tiles) entry = plan_load(p.plan, b, p.q_tiles, q + kThreads, p.Nkv);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const int it_lo = bars->it_lo;
  const int cnt = max(0, bars->it_hi - it_lo);  // query tiles per head
  // This CTA's share [first, first + n_it) of the key tile's (head, query tile)
  // pairs; with a learned bias it is whole heads, as the sums by distance are
  // a head's.
  const int pairs = cnt * p.group;
  const int first_it = static_cast<int>((static_cast<long long>(pairs) * part) >> p.split_log2);
  const int n_it = static_cast<int>((static_cast<long long>(pairs) * (part + 1)) >> p.split_log2) - first_it;
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{&bars->abort_flag, p.status, p.status + 1, p.wait_limit_ns};

  // 256 x 216 + 128 x 72 = 384 x 168 registers
  if (warp >= kProdWarp) {
    regs_dec<72>();
    if (warp == kProdWarp) {
      int issued = 0;
      if (n_it > 0) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&bars->fixed_full, 2 * C::kTileBytes);
#pragma unroll
          for (int cb = 0; cb < HD / 64; ++cb) {
            tma_load_4d(sK + cb * kT * 128, &tmK, &bars->fixed_full, cb * 64, k0, hk, b);
            tma_load_4d(sV + cb * kT * 128, &tmV, &bars->fixed_full, cb * 64, k0, hk, b);
          }
        }
        // Per-query values of a tile, loaded a tile ahead of their use: the loads
        // depend on nothing, and none waits for a stage.
        struct RowValues {
          float lse[kT / 32], D[kT / 32];
          int2 see[kT / 32];
          PlanTile tile;
        };
        auto load_rows = [&](int it) {
          RowValues v;
          const int h = hk * p.group + (first_it + it) / cnt, qt = it_lo + (first_it + it) % cnt;
          const long long rowbase = (static_cast<long long>(b) * p.H + h) * p.Nq;
#pragma unroll
          for (int r = 0; r < kT / 32; ++r) {
            const int q = qt * kT + lane + 32 * r;
            v.lse[r] = q < p.Nq ? p.LSE[rowbase + q] : -INFINITY;
            v.D[r] = q < p.Nq ? p.D[rowbase + q] : 0.f;
            // (rows past the last see what it sees, with P = 2^-inf: lo and hi keep their order)
            v.see[r] = plan_row(p.plan, b, p.Nq, min(q, p.Nq - 1), p.Nkv);
          }
          v.tile = plan_tile(p.plan, b, p.q_tiles, qt, p.Nkv);
          return v;
        };
        RowValues next = load_rows(0);
        [[maybe_unused]] float slope = 0.f;
        [[maybe_unused]] bool linear = false;
        for (int it = 0; it < n_it; ++it) {
          const int s = it % C::kStages;
          const int head = (first_it + it) / cnt, h = hk * p.group + head;
          const int qt = it_lo + (first_it + it) % cnt, q0 = qt * kT;
          const RowValues now = next;
          if (it + 1 < n_it) next = load_rows(it + 1);
          [[maybe_unused]] float lin = 0.f;  // what a linear slope leaves: lin (k0 - position)
          [[maybe_unused]] int side = 0;
          if constexpr (MODE == kModSlopes) {
            if (it == 0 || qt == it_lo) {
              slope = __ldg(p.slopes + h);
              linear = slope_linear(slope, p.scale);
            }
            if (linear) side = slope_side(k0, q0 + p.q_offset, now.tile.left);
            lin = slope * kModLog2e * static_cast<float>(side);
          }
          float l2[kT / 32], dd[kT / 32];
#pragma unroll
          for (int r = 0; r < kT / 32; ++r) {
            const int q = q0 + lane + 32 * r;
            const bool sees = q < p.Nq && now.see[r].x < now.see[r].y && now.lse[r] != -INFINITY;
            l2[r] = sees ? -(now.lse[r] * kModLog2e) : -INFINITY;
            if constexpr (MODE == kModSlopes)
              if (sees) l2[r] = fmaf(lin, static_cast<float>(k0 - (q + p.q_offset)), l2[r]);
            dd[r] = sees ? -now.D[r] : 0.f;
          }
          uint8_t* st = ring + s * C::kStageBytes;
          bool ok = true;
          if (it >= C::kStages)
            ok = mbar_wait(&bars->empty2[s], static_cast<uint32_t>(it / C::kStages - 1) & 1u, wc, kSiteLoad);
          if (!__all_sync(0xffffffffu, ok)) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&bars->full[s], 2 * C::kTileBytes);
#pragma unroll
            for (int cb = 0; cb < HD / 64; ++cb)
              tma_load_4d(st + C::kTileBytes + cb * kT * 128, &tmdO, &bars->full[s], cb * 64, q0, h, b);
          }
          issued = it + 1;
          if (it >= C::kStages)
            ok = mbar_wait(&bars->empty[s], static_cast<uint32_t>(it / C::kStages - 1) & 1u, wc, kSiteLoad);
          if (!__all_sync(0xffffffffu, ok)) {
            // Q_i will not be loaded: count its bytes and arrival as done
            if (lane == 0) {
              mbar_complete_tx(&bars->full[s], C::kTileBytes);
              mbar_arrive(&bars->full[s]);
            }
            break;
          }
#pragma unroll
          for (int r = 0; r < kT / 32; ++r) {
            const int x = s * kT + lane + 32 * r;
            lse2[x] = l2[r];
            dsum[x] = dd[r];
            slo[x] = now.see[r].x;
            shi[x] = now.see[r].y;
          }
          if constexpr (MODE == kModSlopes) {
            // A head's operand goes to place (head mod 4): the tiles of the head
            // that had it are at least 4 tiles, so at least a ring, back.
            if (it == 0 || qt == it_lo) {
              if (lane < 8)
                slope_fill_q<kF16>(reinterpret_cast<uint8_t*>(bias_all) + kSlopeRowsBytes +
                                       head % 4 * kSlopeQBytes,
                                   lane, slope, p.scale);
              fence_proxy_async();
            }
            if (lane == 0) bars->side[s] = side;
          }
          if (lane == 0)
            bars->seen[s] = (now.tile.lo_max <= k0 && now.tile.hi_min >= k0 + kT ? 1 : 0) | (now.tile.hi_min == 0 ? 2 : 0);
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int cb = 0; cb < HD / 64; ++cb)
              tma_load_4d(st + cb * kT * 128, &tmQ, &bars->full[s], cb * 64, q0, h, b);
            mbar_arrive(&bars->full[s]);  // releases the per-query values above
          }
        }
        if (lane == 0) {
          drain(&bars->fixed_full, 0, wc.limit_ns);
          for (int it = (issued > C::kStages ? issued - C::kStages : 0); it < issued; ++it)
            drain(&bars->full[it % C::kStages], static_cast<uint32_t>(it / C::kStages) & 1u, wc.limit_ns);
        }
      }
    } else if (warp == kMmaWarp) {
      // Order: S^T_0, dP^T_0; then per query tile dV += P^T dO, the next S^T,
      // dK += dS^T Q, the next dP^T; with two S^T tiles the next S^T comes first
      // of all (it waited for P^T to be read: 440 of 2400 cycles a tile at d = 64).
      // The tensor core runs them in issue order.
      if (n_it > 0) {
        const uint64_t kA = sdesc_sw128(smem_u32(sK), 16, 1024);
        const uint64_t vA = sdesc_sw128(smem_u32(sV), 16, 1024);
        auto scores = [&](int it) {
          const int s = it % C::kStages;
          if (!warp_wait(&bars->full[s], static_cast<uint32_t>(it / C::kStages) & 1u, wc, kSiteMma)) return false;
          tc_fence_after_sync();
          const uint32_t col = tmem + C::s_col(it);
          mma_abt<128, HD, kF16, true>(col, kA, sdesc_sw128(smem_u32(ring + s * C::kStageBytes), 16, 1024));
          if constexpr (MODE == kModSlopes)
            add_slope_t<kF16>(col, smem_u32(bias_all) + kSlopeRowsBytes + (first_it + it) / cnt % 4 * kSlopeQBytes,
                              smem_u32(bias_all), bars->side[s]);
          mma_commit<true>(&bars->s_full[C::s_of(it)]);
          return true;
        };
        auto dp = [&](int it) {
          const uint32_t sdo = smem_u32(ring + it % C::kStages * C::kStageBytes + C::kTileBytes);
          mma_abt<128, HD, kF16, true>(tmem + 128, vA, sdesc_sw128(sdo, 16, 1024));
          mma_commit<true>(&bars->dp_full);
        };
        bool ok = warp_wait(&bars->fixed_full, 0, wc, kSiteMma) && scores(0);
        if (ok) dp(0);
        for (int it = 0; ok && it < n_it; ++it) {
          const int s = it % C::kStages;
          const uint32_t sq = smem_u32(ring + s * C::kStageBytes), sdo = sq + C::kTileBytes;
          const bool more = it + 1 < n_it;
          if (C::kTwoS && more) ok = scores(it + 1);
          if (ok) ok = warp_wait(&bars->p_full[C::s_of(it)], C::s_phase(it), wc, kSiteMma);
          if (!ok) break;
          tc_fence_after_sync();
          mma_groups<HD, kF16>(tmem + C::kColAcc0, tmem + C::s_col(it), sdesc_sw128(sdo, kT * 128, 1024), it > 0);
          mma_commit<true>(&bars->empty2[s]);
          if (!C::kTwoS && more) ok = scores(it + 1);
          if (ok) ok = warp_wait(&bars->ds_full, static_cast<uint32_t>(it) & 1u, wc, kSiteMma);
          if (!ok) break;
          tc_fence_after_sync();
          mma_groups<HD, kF16>(tmem + C::kColAcc1, tmem + 128, sdesc_sw128(sq, kT * 128, 1024), it > 0);
          mma_commit<true>(&bars->empty[s]);
          if (more) dp(it + 1);
        }
        if (ok) mma_commit<true>(&bars->acc_full);
        mma_commit<true>(&bars->mma_drain);
        drain(&bars->mma_drain, 0, wc.limit_ns);
        __syncwarp();
      }
    }
  } else {
    regs_inc<216>();
    const int c0 = 64 * (warp >> 2);         // this warpgroup's columns (queries)
    const int row = (warp & 3) * 32 + lane;  // key row of the tile = tensor-memory lane
    const int kabs = k0 + row;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    bool ok = true;
    int h_of = -1;
    [[maybe_unused]] uint32_t sync_phase = 0, near = 0;
    [[maybe_unused]] float far_lo = 0.f, far_hi = 0.f;  // sums of dY at distances <= -R and >= R
    float slope2 = 0.f;
    // Writes the sums of head h by clamped distance, the pads folded into the
    // ends, and clears them.
    [[maybe_unused]] auto flush_sums = [&](int h) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        far_lo += __shfl_xor_sync(0xffffffffu, far_lo, off);
        far_hi += __shfl_xor_sync(0xffffffffu, far_hi, off);
      }
      if (lane == 0) {
        bars->far_part[0][warp] = far_lo;
        bars->far_part[1][warp] = far_hi;
      }
      far_lo = far_hi = 0.f;
      if (!elem_sync(bars, sync_phase, wc)) return false;
      const int R = p.rel.range;
      float* out = p.rel_part + ((static_cast<long long>(b) * p.H + h) * p.num_tiles + kt) * (2 * R + 1);
      for (int x = 1 + static_cast<int>(threadIdx.x); x < 2 * R; x += 256) out[x] = sums[x + kSumPad];
      if (warp < 2) {  // distance -R (warp 0), R (warp 1)
        const float* pad = sums + (warp == 0 ? 0 : 2 * R + kSumPad);
        float v = 0.f;
        for (int x = lane; x <= kSumPad; x += 32) v += pad[x];
        if (lane < 8) v += bars->far_part[warp][lane];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (lane == 0) out[warp == 0 ? 0 : 2 * R] = v;
      }
      if (!elem_sync(bars, sync_phase, wc)) return false;
      for (int x = threadIdx.x; x < sum_entries(R); x += 256) sums[x] = 0.f;
      return true;
    };
    if constexpr (mode_rel(MODE)) {
      for (int x = threadIdx.x; x < sum_entries(p.rel.range); x += 256) sums[x] = 0.f;
      if (n_it == 0) {  // nobody sees these keys: every head's sums are 0
        ok = elem_sync(bars, sync_phase, wc);
        const int heads = p.group >> p.split_log2;
        for (int g = part * heads; ok && g < (part + 1) * heads; ++g) ok = flush_sums(hk * p.group + g);
      }
    }
    int h = 0, qt = 0;
    if (n_it > 0) {
      h = hk * p.group + first_it / cnt;
      qt = it_lo + first_it % cnt;
    }
    for (int it = 0; ok && it < n_it; ++it, ++qt) {
      const int s = it % C::kStages;
      if (qt == bars->it_hi) {
        qt = it_lo;
        ++h;
      }
      const int p0 = qt * kT + p.q_offset;  // position of the tile's first query
      if (h != h_of) {  // uniform over the elementwise warps
        if constexpr (mode_slopes(MODE)) slope2 = p.slopes[h] * kModLog2e;
        if constexpr (mode_rel(MODE)) {
          // the last head's sums, after which everyone is done with its table
          if (h_of >= 0 && !(ok = flush_sums(h_of))) break;
          float least, most;
          rel_fill<kF16>(bias_all, p.rel, p.H, h, threadIdx.x, 256, least, most);
          if (!(ok = elem_sync(bars, sync_phase, wc))) break;
        }
        h_of = h;
      }
      ok = mbar_wait(&bars->s_full[C::s_of(it)], C::s_phase(it), wc, kSiteElem);
      if (ok) ok = mbar_wait(&bars->full[s], static_cast<uint32_t>(it / C::kStages) & 1u, wc, kSiteElem);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after_sync();
      const float4* l2 = reinterpret_cast<const float4*>(lse2 + s * kT);
      const float4* dd = reinterpret_cast<const float4*>(dsum + s * kT);
      const int* lo = slo + s * kT;
      const int* hi = shi + s * kT;
      const int d0 = kabs - p0;  // distance to the tile's first query
      auto vis = [&](int col) { return lo[col] <= kabs && kabs < hi[col]; };
      auto l2of4 = [&](int col) { return l2[col >> 2]; };
      // The group's columns for this warp's rows: all visible, none, or some.
      // lo and hi do not fall from one query to the next that sees a key, so
      // the first and last column decide, in tiles where every query does.
      const int seen = bars->seen[s];
      bool none = false, full = (seen & 1) != 0;
      if (seen == 0) {
        full = __all_sync(0xffffffffu, lo[c0 + 63] <= kabs && kabs < hi[c0]);
        none = __all_sync(0xffffffffu, kabs < lo[c0] || kabs >= hi[c0 + 63]);
      }
      [[maybe_unused]] int side = 0;  // learned bias: distances of the warp's 32 keys to the group's 64 queries
      if constexpr (mode_rel(MODE)) {
        const int first = k0 + 32 * (warp & 3) - p0 - c0 - 63;
        side = far_side(first, first + 94, p.rel.range);
      }
      const uint32_t s_addr = lane_base + C::s_col(it);
      float pr[64];
      auto part = [&](auto mask) {
        constexpr bool kMask = decltype(mask)::value;
        if constexpr (mode_rel(MODE)) {
          const int R = p.rel.range;
          if (side != 0) {
            const float far = bias_all[side < 0 ? 0 : rel_entries(R) - 1];
            p_part<kF16, MODE, true, kMask, true>(s_addr, c0, p, vis, l2of4, [&](int) { return far; }, pr);
          } else {
            const float* bt = bias_all + (d0 + R + kRelPad);
            p_part<kF16, MODE, true, kMask, true>(s_addr, c0, p, vis, l2of4,
                                                  [&](int col) { return bt[-col]; }, pr);
          }
        } else if (mode_slopes(MODE) && (MODE == kModCapSlopes || bars->side[s] == 0)) {
          const float f0 = static_cast<float>(d0);
          p_part<kF16, MODE, true, kMask, true>(
              s_addr, c0, p, vis, l2of4,
              [&](int col) { return -slope2 * fabsf(f0 - static_cast<float>(col)); }, pr);
        } else {
          p_part<kF16, MODE, true, kMask, false>(s_addr, c0, p, vis, l2of4, [](int) { return 0.f; }, pr);
        }
      };
      bool waited = false;
      if (full) {
        part(std::false_type{});
      } else if (none) {
        p_none<true>(s_addr, c0, pr);
      } else {
        part(std::true_type{});
        if (seen & 2) {
          // Queries of this tile that see nothing: their rows of Q and dO
          // must not reach the sums (0 * NaN is NaN).  dP^T, the last other
          // reader of dO, is awaited first.
          ok = mbar_wait(&bars->dp_full, static_cast<uint32_t>(it) & 1u, wc, kSiteElem);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          waited = true;
          uint8_t* st = ring + s * C::kStageBytes;
          if (lo[row] >= hi[row]) {
            // warpgroup 0 clears Q, warpgroup 1 dO
#pragma unroll
            for (int cb = 0; cb < HD / 64; ++cb) zero_row(st + (c0 ? C::kTileBytes : 0), cb, row);
          }
          fence_proxy_async();
        }
      }
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&bars->p_full[C::s_of(it)]);
      if (!waited) {
        ok = mbar_wait(&bars->dp_full, static_cast<uint32_t>(it) & 1u, wc, kSiteElem);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      tc_fence_after_sync();
      auto dof4 = [&](int col) { return dd[col >> 2]; };
      constexpr bool kKeep = mode_rel(MODE);
      uint64_t no_sum = 0;
      if (full)
        ds_part<kF16, false, kKeep, false>(lane_base + 128, c0, dof4, pr, no_sum);
      else
        ds_part<kF16, true, kKeep, false>(lane_base + 128, c0, dof4, pr, no_sum);
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&bars->ds_full);
      if constexpr (mode_rel(MODE)) {
        // A block of 32 keys and 64 queries beyond the range goes to one
        // distance.  Otherwise sums along its diagonals: a running sum moves
        // one lane up with every column, so that it stays on one distance;
        // lane 31 stores the diagonals that end there.  Strip entry u holds
        // distance (32 quarter - c0) + 31 - u within the tile.
        if (side != 0 && !none) {
          float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int x = 0; x < 64; ++x) a[x & 3] += pr[x];
          const float sum = (a[0] + a[1]) + (a[2] + a[3]);
          if (side < 0) far_lo += sum;
          else far_hi += sum;
        }
        if (far_side(k0 - p0 - 127, k0 - p0 + 127, p.rel.range) == 0) {
          const int buf = near++ & 1;
          float* strip = strips + buf * 8 * 96 + warp * 96;
          if (side != 0 || none) {
#pragma unroll
            for (int x = 0; x < 3; ++x) strip[32 * x + lane] = 0.f;
          } else {
            // four runs of 16 columns side by side (one run of 64 waits for
            // each shuffle); what a run has left in lane r would have left
            // lane 31 31 - r columns later
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int x = 0; x < 16; ++x) {
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                acc[u] = __shfl_up_sync(0xffffffffu, acc[u], 1);
                acc[u] = (lane == 0 ? 0.f : acc[u]) + pr[16 * u + x];
                if (lane == 31) strip[16 * u + x] = acc[u];
              }
            }
            if (lane < 31) strip[94 - lane] = acc[3];
#pragma unroll
            for (int u = 2; u >= 0; --u) {
              __syncwarp();
              if (lane < 31) strip[16 * u + 46 - lane] += acc[u];
            }
          }
          if (!(ok = elem_sync(bars, sync_phase, wc))) break;
          // thread u adds distance u - 127 of the tile to the sums
          const int u = threadIdx.x;
          if (u < 2 * kT - 1) {
            float add = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
              const int at = 31 + 32 * (w & 3) - 64 * (w >> 2) - (u - 127);
              if (at >= 0 && at < 95) add += strips[buf * 8 * 96 + w * 96 + at];
            }
            sums[k0 - p0 + (u - 127) + p.rel.range + kSumPad] += add;
          }
        }
      }
    }
    if constexpr (mode_rel(MODE)) {
      if (ok && n_it > 0) ok = flush_sums(h_of);
    }
    // epilogue: warpgroup 0 writes dV, warpgroup 1 dK
    bool has_acc = false;
    if (ok && n_it > 0) {
      ok = mbar_wait(&bars->acc_full, 0, wc, kSiteEpi);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) tc_fence_after_sync();
      has_acc = ok;
    }
    if (ok && p.split_log2 > 0) {
      // fp32 over the tiles, whose last readers are done, for the join below
      const int w = warp >> 2;
      float4* out = reinterpret_cast<float4*>(smem + w * kT * HD * 4) + row * (HD / 4);
      const uint32_t acc = lane_base + (w == 0 ? C::kColAcc0 : C::kColAcc1);
#pragma unroll 1
      for (int ch = 0; ch < HD / 32; ++ch) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(acc + ch * 32, r);
        tmem_ld_wait();
        reg_fence32(r);
#pragma unroll
        for (int x = 0; x < 8; ++x)
          out[(ch * 8 + x) ^ (row & 7)] =
              has_acc ? make_float4(__uint_as_float(r[4 * x]), __uint_as_float(r[4 * x + 1]),
                                    __uint_as_float(r[4 * x + 2]), __uint_as_float(r[4 * x + 3]))
                      : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    } else if (ok) {
      // over V and K, whose last readers are done
      const int w = warp >> 2;
      uint8_t* out = w == 0 ? sV : sK;
      stage_out<HD, kF16>(out, row, 0, lane_base + (w == 0 ? C::kColAcc0 : C::kColAcc1), has_acc,
                          w == 0 ? 1.f : p.scale);
      fence_proxy_async();
      mbar_arrive(&bars->staged[w]);
      if ((warp & 3) == 0) {
        ok = mbar_wait(&bars->staged[w], 0, wc, kSiteEpi);
        if (ok && lane == 0) {
#pragma unroll
          for (int cb = 0; cb < HD / 64; ++cb)
            tma_store_4d(w == 0 ? &tmdV : &tmdK, out + cb * kT * 128, cb * 64, k0, hk, b);
          tma_store_drain();
        }
        __syncwarp();
      }
    }
  }

  __syncwarp();
  if (p.split_log2 > 0) {
    // The sums of the cluster's CTAs, added in rank order; each CTA finishes
    // its share of the rows.  (A CTA whose waits gave up comes here too.)
    cluster_sync();
    const int rows = kT >> p.split_log2;
    for (int x = threadIdx.x; x < 2 * rows * (HD / 8); x += kThreads) {
      const int w = x / (rows * (HD / 8)), c = x % (HD / 8);
      const int row = part * rows + x / (HD / 8) % rows;
      const uint32_t at = smem_u32(smem) + (w * kT + row) * HD * 4;
      float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int r = 0; r < (1 << p.split_log2); ++r) {
        float v[8];
        cluster_load4(at + ((2 * c) ^ (row & 7)) * 16, r, v);
        cluster_load4(at + ((2 * c + 1) ^ (row & 7)) * 16, r, v + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += v[e];
      }
      const float mul = w == 0 ? 1.f : p.scale;
      if (k0 + row < p.Nkv)
        *reinterpret_cast<uint4*>(p.dkv[w] + b * p.dkv_s[w][0] + hk * p.dkv_s[w][1] + (k0 + row) * p.dkv_s[w][2] + 8 * c) =
            make_uint4(pack2<kF16>(a[0] * mul, a[1] * mul), pack2<kF16>(a[2] * mul, a[3] * mul),
                       pack2<kF16>(a[4] * mul, a[5] * mul), pack2<kF16>(a[6] * mul, a[7] * mul));
    }
    cluster_sync();  // the others have read this CTA's sums
  }
  tmem_st_wait();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kCols);
  }
}

// ------------------------------------------------------------------ dQ
constexpr uint32_t kDqColDP = 256, kDqColAcc = 384;

template <int HD, bool kF16, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
    dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmdO,
              const __grid_constant__ CUtensorMap tmdQ, const Params p) {
  using C = Cfg<HD, MODE>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // see fwd_mod_kernel
    if (threadIdx.x == 0) atomicExch(p.status, 3u /* OSATTN_ERR_CUDA */);
    return;
  }
  uint8_t* sQ = smem;
  uint8_t* sdO = smem + C::kTileBytes;
  uint8_t* kring = smem + 2 * C::kTileBytes;
  uint8_t* vring = kring + C::kKSlots * C::kTileBytes;
  float* bias = reinterpret_cast<float*>(smem + C::kDqTable);  // or the slope operands
  Bars* bars = reinterpret_cast<Bars*>(smem + C::kDqRegion);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  int bh, rank;
  unit_of(p, blockIdx.x, bh, rank);
  const int qt = p.num_tiles - 1 - rank;
  const int b = bh / p.H, h = bh % p.H, hk = h / p.group;
  [[maybe_unused]] float slope = 0.f;
  if constexpr (mode_slopes(MODE)) slope = __ldg(p.slopes + h);
  const int q0 = qt * kT;
  const int4 entry = plan_load(p.plan, b, p.q_tiles, qt, p.Nkv);  // on its way during the set-up

  if (threadIdx.x == 0) {
    mbar_init(&bars->fixed_full, 1);
    for (int s = 0; s < C::kKSlots; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int s = 0; s < C::kVSlots; ++s) mbar_init(&bars->empty2[s], 1);
    mbar_init(&bars->s_full[0], 1);
    mbar_init(&bars->s_full[1], 1);
    mbar_init(&bars->dp_full, 1);
    mbar_init(&bars->ds_full, 256);
    mbar_init(&bars->acc_full, 1);
    mbar_init(&bars->mma_drain, 1);
    mbar_init(&bars->d_full, 256);
    mbar_init(&bars->elem, 256);
    mbar_init(&bars->staged[0], 256);
    bars->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, kCols);
    tmem_relinquish();
  }
  if (threadIdx.x < kT) bars->d_part[threadIdx.x] = 0.f;
  [[maybe_unused]] bool linear = false;
  if constexpr (MODE == kModSlopes) {
    linear = slope_linear(slope, p.scale);
    uint8_t* at = reinterpret_cast<uint8_t*>(bias);
    if (threadIdx.x < kT / 2) slope_fill_k<kF16>(at, threadIdx.x);
    if (threadIdx.x < 8) slope_fill_q<kF16>(at + kSlopeRowsBytes / 2, threadIdx.x, slope, p.scale);
    fence_proxy_async();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  const WaitCtl wc{&bars->abort_flag, p.status, p.status + 1, p.wait_limit_ns};
  const PlanTile pt = plan_entry(entry);
  const int kt0 = pt.lo / kT;
  const int n_kt = pt.lo < pt.hi ? (pt.hi + kT - 1) / kT - kt0 : 0;

  // 256 x 216 + 128 x 72 = 384 x 168 registers
  if (warp >= kProdWarp) {
    regs_dec<72>();
    if (warp == kProdWarp) {
      if (lane == 0 && n_kt > 0) {
        mbar_arrive_expect_tx(&bars->fixed_full, 2 * C::kTileBytes);
#pragma unroll
        for (int cb = 0; cb < HD / 64; ++cb) {
          tma_load_4d(sQ + cb * kT * 128, &tmQ, &bars->fixed_full, cb * 64, q0, h, b);
          tma_load_4d(sdO + cb * kT * 128, &tmdO, &bars->fixed_full, cb * 64, q0, h, b);
        }
        int issued = 0;
        for (int j = 0; j < n_kt; ++j) {
          const int a = j % C::kKSlots, v = j % C::kVSlots;
          if (j >= C::kKSlots &&
              !mbar_wait(&bars->empty[a], static_cast<uint32_t>(j / C::kKSlots - 1) & 1u, wc, kSiteLoad))
            break;
          if (j >= C::kVSlots &&
              !mbar_wait(&bars->empty2[v], static_cast<uint32_t>(j / C::kVSlots - 1) & 1u, wc, kSiteLoad))
            break;
          mbar_arrive_expect_tx(&bars->full[a], 2 * C::kTileBytes);
#pragma unroll
          for (int cb = 0; cb < HD / 64; ++cb) {
            tma_load_4d(kring + a * C::kTileBytes + cb * kT * 128, &tmK, &bars->full[a], cb * 64,
                        (kt0 + j) * kT, hk, b);
            tma_load_4d(vring + v * C::kTileBytes + cb * kT * 128, &tmV, &bars->full[a], cb * 64,
                        (kt0 + j) * kT, hk, b);
          }
          issued = j + 1;
        }
        drain(&bars->fixed_full, 0, wc.limit_ns);
        for (int j = (issued > C::kKSlots ? issued - C::kKSlots : 0); j < issued; ++j)
          drain(&bars->full[j % C::kKSlots], static_cast<uint32_t>(j / C::kKSlots) & 1u, wc.limit_ns);
      }
    } else if (warp == kMmaWarp) {
      // Order: S_0, dP_0; then per key tile j: S_{j+1}, dQ += dS_j K_j, dP_{j+1}.
      if (n_kt > 0) {
        const uint64_t qA = sdesc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dA = sdesc_sw128(smem_u32(sdO), 16, 1024);
        [[maybe_unused]] auto slope_step = [&](uint32_t s_col, int j) {
          add_slope<kF16>(s_col, smem_u32(bias) + kSlopeRowsBytes / 2, smem_u32(bias),
                          linear ? slope_side((kt0 + j) * kT, q0 + p.q_offset, pt.left) : 0);
        };
        bool ok = warp_wait(&bars->fixed_full, 0, wc, kSiteMma);
        if (ok) ok = warp_wait(&bars->full[0], 0, wc, kSiteMma);
        if (ok) {
          tc_fence_after_sync();
          mma_abt<128, HD, kF16, true>(tmem, qA, sdesc_sw128(smem_u32(kring), 16, 1024));
          if constexpr (MODE == kModSlopes) slope_step(tmem, 0);
          mma_commit<true>(&bars->s_full[0]);
          mma_abt<128, HD, kF16, true>(tmem + kDqColDP, dA, sdesc_sw128(smem_u32(vring), 16, 1024));
          mma_commit<true>(&bars->dp_full);
          mma_commit<true>(&bars->empty2[0]);
        }
        for (int j = 0; ok && j < n_kt; ++j) {
          const int a = j % C::kKSlots, a1 = (j + 1) % C::kKSlots, v1 = (j + 1) % C::kVSlots;
          const uint32_t sk = smem_u32(kring + a * C::kTileBytes);
          const uint32_t nk = smem_u32(kring + a1 * C::kTileBytes);
          const uint32_t nv = smem_u32(vring + v1 * C::kTileBytes);
          const bool more = j + 1 < n_kt;
          if (more) {
            ok = warp_wait(&bars->full[a1], static_cast<uint32_t>((j + 1) / C::kKSlots) & 1u, wc, kSiteMma);
            if (!ok) break;
            tc_fence_after_sync();
            mma_abt<128, HD, kF16, true>(tmem + 128 * ((j + 1) & 1), qA, sdesc_sw128(nk, 16, 1024));
            if constexpr (MODE == kModSlopes) slope_step(tmem + 128 * ((j + 1) & 1), j + 1);
            mma_commit<true>(&bars->s_full[(j + 1) & 1]);
          }
          ok = warp_wait(&bars->ds_full, static_cast<uint32_t>(j) & 1u, wc, kSiteMma);
          if (!ok) break;
          tc_fence_after_sync();
          mma_groups<HD, kF16>(tmem + kDqColAcc, tmem + kDqColDP, sdesc_sw128(sk, kT * 128, 1024), j > 0);
          mma_commit<true>(&bars->empty[a]);
          if (more) {
            mma_abt<128, HD, kF16, true>(tmem + kDqColDP, dA, sdesc_sw128(nv, 16, 1024));
            mma_commit<true>(&bars->dp_full);
            mma_commit<true>(&bars->empty2[v1]);
          }
        }
        if (ok) mma_commit<true>(&bars->acc_full);
        mma_commit<true>(&bars->mma_drain);
        drain(&bars->mma_drain, 0, wc.limit_ns);
        __syncwarp();
      }
    }
  } else {
    regs_inc<216>();
    const int c0 = 64 * (warp >> 2);         // this warpgroup's columns (keys)
    const int row = (warp & 3) * 32 + lane;  // query row of the tile = tensor-memory lane
    const int q = q0 + row;
    const bool in = q < p.Nq;
    const int2 see = plan_row(p.plan, b, p.Nq, q, p.Nkv);
    const bool row_live = see.x < see.y;
    const long long rix = static_cast<long long>(bh) * p.Nq + q;
    const int p0 = q0 + p.q_offset;
    const float slope2 = slope * kModLog2e;
    float l2 = -INFINITY;  // -LSE log2 e
    // D of this row: warpgroup g takes columns g d/2 .. (g + 1) d/2 - 1, O
    // from global memory (loaded now), dO from the resident tile
    constexpr int kHalfD = HD / 2, kNv = kHalfD / 8;
    const int g = warp >> 2;
    uint4 ov[kNv];
#pragma unroll
    for (int v = 0; v < kNv; ++v) ov[v] = make_uint4(0u, 0u, 0u, 0u);
    if (row_live) {
      const float L = p.LSE[rix];
      l2 = (L == -INFINITY) ? -INFINITY : -(L * kModLog2e);
      const uint4* orow = reinterpret_cast<const uint4*>(
          p.O + b * p.o_s[0] + h * p.o_s[1] + static_cast<long long>(q) * p.o_s[2] + g * kHalfD);
#pragma unroll
      for (int v = 0; v < kNv; ++v) ov[v] = orow[v];
    }
    float4 dv4 = make_float4(0.f, 0.f, 0.f, 0.f);  // -D
    // A row's dY sum to 0 but for the error that D has from O's rounding to 16
    // bits: the sum is what D lacks.  dQ is done by then, dK and the table's
    // gradient take the right D.  (Capped scores: pr has the cap's factor in it.)
    constexpr bool kFixD = !mode_cap(MODE);
    [[maybe_unused]] uint64_t rest2 = 0;
    if (n_kt == 0 && g == 0 && in) p.D[rix] = 0.f;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    [[maybe_unused]] uint32_t sync_phase = 0;
    bool ok = true;
    if constexpr (mode_rel(MODE)) {  // while the first loads and products run
      float least, most;
      rel_fill<kF16>(bias, p.rel, p.H, h, threadIdx.x, 256, least, most);
      ok = elem_sync(bars, sync_phase, wc);
    }
    for (int j = 0; ok && j < n_kt; ++j) {
      ok = mbar_wait(&bars->s_full[j & 1], static_cast<uint32_t>(j >> 1) & 1u, wc, kSiteElem);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after_sync();
      const int kx = (kt0 + j) * kT;
      const int d0 = kx - (q + p.q_offset);
      // the row's visible keys of the group, as bits
      const int from = see.x - kx - c0, to = see.y - kx - c0;
      bool none = false, full = pt.lo_max <= kx && pt.hi_min >= kx + kT;
      if (!full) {
        full = __all_sync(0xffffffffu, from <= 0 && to >= 64);
        none = __all_sync(0xffffffffu, max(from, 0) >= min(to, 64));
      }
      const uint32_t bits[2] = {bit_range(from, to), bit_range(from - 32, to - 32)};
      auto vis = [&](int col) { return (bits[(col - c0) >> 5] & (1u << ((col - c0) & 31))) != 0u; };
      float nl = l2;
      [[maybe_unused]] int sside = 0;
      if constexpr (MODE == kModSlopes) {
        sside = linear ? slope_side(kx, p0, pt.left) : 0;
        nl = fmaf(slope2 * static_cast<float>(sside), static_cast<float>(d0 + c0), nl);
      }
      [[maybe_unused]] int side = 0;  // learned bias: distances of the warp's 32 queries to the group's 64 keys
      if constexpr (mode_rel(MODE)) {
        const int first = kx + c0 - p0 - 32 * (warp & 3) - 31;
        side = far_side(first, first + 94, p.rel.range);
        if (side != 0) nl += bias[side < 0 ? 0 : rel_entries(p.rel.range) - 1];
      }
      const float4 l2v = make_float4(nl, nl, nl, nl);
      auto l2of4 = [&](int) { return l2v; };
      const uint32_t s_addr = lane_base + 128 * (j & 1);
      float pr[64];
      auto part = [&](auto mask) {
        constexpr bool kMask = decltype(mask)::value;
        if constexpr (mode_rel(MODE)) {
          if (side != 0) {
            p_part<kF16, MODE, false, kMask, false>(s_addr, c0, p, vis, l2of4, [](int) { return 0.f; }, pr);
          } else {
            const float* bt = bias + (d0 + p.rel.range + kRelPad);
            p_part<kF16, MODE, false, kMask, true>(s_addr, c0, p, vis, l2of4,
                                                   [&](int col) { return bt[col]; }, pr);
          }
        } else if (mode_slopes(MODE) && sside == 0) {
          const float f0 = static_cast<float>(d0);
          p_part<kF16, MODE, false, kMask, true>(
              s_addr, c0, p, vis, l2of4,
              [&](int col) { return -slope2 * fabsf(f0 + static_cast<float>(col)); }, pr);
        } else {
          p_part<kF16, MODE, false, kMask, false>(s_addr, c0, p, vis, l2of4, [](int) { return 0.f; }, pr);
        }
      };
      if (full)
        part(std::false_type{});
      else if (none)
        p_none<false>(s_addr, c0, pr);
      else
        part(std::true_type{});
      if (kx < pt.lo || min(kx + kT, p.Nkv) > pt.hi) {
        // keys of this tile that no row sees: zero their rows of K_j, which
        // dQ += dS_j K_j reads after ds_full (S_j, the other reader, is done)
        if (kx + row < pt.lo || kx + row >= pt.hi) {
          uint8_t* ks = kring + (j % C::kKSlots) * C::kTileBytes;
          if (HD == 128) zero_row(ks, g, row);
          else if (g == 0) zero_row(ks, 0, row);
        }
        fence_proxy_async();
      }
      if (j == 0) {
        // the half dot product of D over this warpgroup's columns of the
        // swizzled dO tile, then both halves through shared memory
        ok = mbar_wait(&bars->fixed_full, 0, wc, kSiteElem);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        float sum = 0.f;
#pragma unroll
        for (int v = 0; v < kNv; ++v) {
          const int col = g * kHalfD + v * 8;
          const uint4 gv = *reinterpret_cast<const uint4*>(
              sdO + (col / 64) * kT * 128 + row * 128 + ((((col % 64) / 8) ^ (row & 7)) * 16));
          const uint32_t ow[4] = {ov[v].x, ov[v].y, ov[v].z, ov[v].w};
          const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = unpack16<kF16>(ow[e]), y = unpack16<kF16>(gw[e]);
            sum = fmaf(x.x, y.x, fmaf(x.y, y.y, sum));
          }
        }
        atomicAdd(&bars->d_part[row], sum);
        mbar_arrive(&bars->d_full);
        ok = mbar_wait(&bars->d_full, 0, wc, kSiteElem);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const float D = row_live ? bars->d_part[row] : 0.f;
        dv4 = make_float4(-D, -D, -D, -D);
        if (g == 0 && in) p.D[rix] = D;
      }
      ok = mbar_wait(&bars->dp_full, static_cast<uint32_t>(j) & 1u, wc, kSiteElem);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after_sync();
      auto dof4 = [&](int) { return dv4; };
      if (full)
        ds_part<kF16, false, false, kFixD>(lane_base + kDqColDP, c0, dof4, pr, rest2);
      else
        ds_part<kF16, true, false, kFixD>(lane_base + kDqColDP, c0, dof4, pr, rest2);
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&bars->ds_full);
    }
    bool has_acc = false;
    if (ok && n_kt > 0) {
      ok = mbar_wait(&bars->acc_full, 0, wc, kSiteEpi);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) tc_fence_after_sync();
      has_acc = ok;
    }
    if constexpr (kFixD) {
      if (ok && n_kt > 0) {
        float r0, r1;
        f2_unpack(rest2, r0, r1);
        if (g == 1) bars->d_part[row] = r0 + r1;  // everyone has D: dS was complete
        ok = elem_sync(bars, sync_phase, wc);
        if (ok && g == 0 && row_live) p.D[rix] = (r0 + r1 + bars->d_part[row]) - dv4.x;
      }
    }
    if (ok) {
      // over Q, whose last reader is done
      stage_out<HD / 2, kF16>(sQ, row, c0 * HD / 128, lane_base + kDqColAcc + c0 * HD / 128, has_acc, p.scale);
      fence_proxy_async();
      mbar_arrive(&bars->staged[0]);
      if (warp == 0) {
        ok = mbar_wait(&bars->staged[0], 0, wc, kSiteEpi);
        if (ok && lane == 0) {
#pragma unroll
          for (int cb = 0; cb < HD / 64; ++cb) tma_store_4d(&tmdQ, sQ + cb * kT * 128, cb * 64, q0, h, b);
          tma_store_drain();
        }
        __syncwarp();
      }
    }
  }

  __syncwarp();
  tmem_st_wait();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    __syncwarp();
    tc_fence_after_sync();
    tmem_dealloc(tmem, kCols);
  }
}

// The table's gradient: one block per head.  Each warp sums a share of the
// key tiles' partials over batch entries and tiles, lanes along the distances;
// the warps' sums are added in order, then each warp sums the distances of its
// buckets.  Bound by latency: 2 R + 1 floats a tile (5 us for B8 H12 512).
template <bool kF16>
__global__ void __launch_bounds__(1024) rel_reduce_kernel(const float* __restrict__ part,
                                                          uint16_t* __restrict__ out, RelArgs rel, int B,
                                                          int H, int tiles) {
  constexpr int kX = 4;  // blocks of 32 distances a warp takes at a time
  __shared__ float warp_sum[32][32 * kX];
  __shared__ float sums[2 * kMaxRelRange + 1];
  __shared__ int map[2 * kMaxRelRange + 1];
  const int h = blockIdx.x, n = 2 * rel.range + 1, rows = B * tiles;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int x = threadIdx.x; x < n; x += 1024) map[x] = rel.map[x];
  for (int x0 = 0; x0 < n; x0 += 32 * kX) {
    float a[kX];
#pragma unroll
    for (int u = 0; u < kX; ++u) a[u] = 0.f;
#pragma unroll 4
    for (int r = warp; r < rows; r += 32) {
      const int b = r / tiles, t = r - b * tiles;
      const float* src = part + ((static_cast<long long>(b) * H + h) * tiles + t) * n + x0 + lane;
#pragma unroll
      for (int u = 0; u < kX; ++u)
        if (x0 + lane + 32 * u < n) a[u] += src[32 * u];
    }
#pragma unroll
    for (int u = 0; u < kX; ++u) warp_sum[warp][32 * u + lane] = a[u];
    __syncthreads();
    if (threadIdx.x < 32 * kX && x0 + threadIdx.x < n) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < 32; ++w) v += warp_sum[w][threadIdx.x];
      sums[x0 + threadIdx.x] = v;
    }
    __syncthreads();
  }
  for (int k = warp; k < rel.num; k += 32) {
    float v = 0.f;
    for (int x = lane; x < n; x += 32) v += map[x] == k ? sums[x] : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (lane == 0)
      out[static_cast<long long>(k) * H + h] = static_cast<uint16_t>(pack2<kF16>(v, 0.f) & 0xffffu);
  }
}

// The setmaxnreg split hands out exactly 384 x 168 registers; a build with
// another launch count would wait forever in setmaxnreg.inc and is refused.
constexpr int kLaunchRegs = 168;

template <int HD, bool kF16, int MODE>
cudaError_t set_attrs() {
  constexpr int kDkdvMode = MODE == kModRelWide ? kModRel : MODE;
  static_assert(dkdv_smem_bytes<HD, kDkdvMode>() <= 232448 && dq_smem_bytes<HD, MODE>() <= 232448,
                "shared memory per CTA");
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, dkdv_kernel<HD, kF16, kDkdvMode>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncGetAttributes(&fa, dq_kernel<HD, kF16, MODE>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  e = cudaFuncSetAttribute(dkdv_kernel<HD, kF16, kDkdvMode>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       dkdv_smem_bytes<HD, kDkdvMode>());
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(dq_kernel<HD, kF16, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              dq_smem_bytes<HD, MODE>());
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
cudaError_t launch_mode(const ModArgs& a, const Params& pq, const Params& pk, unsigned gq, unsigned gk,
                        const BwdModMaps& m) {
  // dQ first: it writes D, which the dK/dV kernel reads
  dq_kernel<HD, kF16, MODE><<<gq, kThreads, dq_smem_bytes<HD, MODE>(), a.stream>>>(m.q, m.k, m.v, m.g, m.dq, pq);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  constexpr int kDkdvMode = MODE == kModRelWide ? kModRel : MODE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gk);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = dkdv_smem_bytes<HD, kDkdvMode>();
  cfg.stream = a.stream;
  cudaLaunchAttribute cluster;
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = 1u << pk.split_log2;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = pk.split_log2 > 0 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, dkdv_kernel<HD, kF16, kDkdvMode>, m.q, m.k, m.v, m.g, m.dk, m.dv, pk);
  if (e != cudaSuccess || !mode_rel(MODE)) return e;
  rel_reduce_kernel<kF16><<<a.H, 1024, 0, a.stream>>>(a.rel_part, static_cast<uint16_t*>(a.dRel), a.rel,
                                                      a.B, a.H, pk.num_tiles);
  return cudaGetLastError();
}

template <int HD, bool kF16>
cudaError_t launch(const ModArgs& a, const BwdModMaps& m) {
  Params p = {};
  for (int i = 0; i < 3; ++i) p.o_s[i] = a.o_s[i];
  p.LSE = a.LSE;
  p.D = a.D;
  p.O = static_cast<const uint16_t*>(a.O_in);
  p.q_tiles = (a.Nq + kT - 1) / kT;
  p.plan.tiles = static_cast<const int4*>(a.plan);
  p.plan.rows = a.plan ? reinterpret_cast<const int2*>(p.plan.tiles + static_cast<long long>(a.B) * p.q_tiles)
                       : nullptr;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.group = a.H / a.Hkv;
  p.Nq = a.Nq;
  p.Nkv = a.Nkv;
  p.scale = a.scale;
  p.scale_log2 = a.scale * kModLog2e;
  p.cap = make_cap(a.scale, a.softcap, kF16);
  p.slopes = a.slopes;
  p.rel = a.rel;
  p.rel_part = a.rel_part;
  p.q_offset = a.q_offset;
  p.status = a.status;
  p.wait_limit_ns = a.wait_limit_ns;
  // heads whose streamed tiles take about 32 MB of L2 together
  auto group = [&](long long rows, long long bh) {
    const long long gh = (32ll << 20) / (2ll * rows * a.d * 2);
    return static_cast<int>(gh < 1 ? 1 : (gh > bh ? bh : gh));
  };
  Params pk = p, pq = p;
  pk.BH = a.B * a.Hkv;
  pk.num_tiles = (a.Nkv + kT - 1) / kT;
  pk.group_heads = group(static_cast<long long>(a.Nq) * p.group, pk.BH);
  pq.BH = a.B * a.H;
  pq.num_tiles = p.q_tiles;
  pq.group_heads = group(a.Nkv, pq.BH);
  pk.split_log2 = dkdv_split(static_cast<long long>(pk.num_tiles) * pk.BH, a.num_sms,
                        static_cast<long long>(p.q_tiles) * p.group, a.rel.table ? p.group : 8);
  pk.dkv[0] = static_cast<uint16_t*>(a.dV);
  pk.dkv[1] = static_cast<uint16_t*>(a.dK);
  for (int i = 0; i < 3; ++i) {
    pk.dkv_s[0][i] = a.dv_s[i];
    pk.dkv_s[1][i] = a.dk_s[i];
  }
  const long long gk = static_cast<long long>(pk.num_tiles) * pk.BH << pk.split_log2;
  const long long gq = static_cast<long long>(pq.num_tiles) * pq.BH;
  if (gk > 0x7fffffffLL || gq > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned uq = static_cast<unsigned>(gq), uk = static_cast<unsigned>(gk);
  switch (mod_score_mode(a)) {
    case kModCap: return launch_mode<HD, kF16, kModCap>(a, pq, pk, uq, uk, m);
    case kModSlopes: return launch_mode<HD, kF16, kModSlopes>(a, pq, pk, uq, uk, m);
    case kModCapSlopes: return launch_mode<HD, kF16, kModCapSlopes>(a, pq, pk, uq, uk, m);
    case kModRel:
      if constexpr (HD == 128)
        if (a.rel.range > kSmallRel) return launch_mode<HD, kF16, kModRelWide>(a, pq, pk, uq, uk, m);
      return launch_mode<HD, kF16, kModRel>(a, pq, pk, uq, uk, m);
    default: return launch_mode<HD, kF16, kModPlain>(a, pq, pk, uq, uk, m);
  }
}

}  // namespace bwdmod
}  // namespace osattn
