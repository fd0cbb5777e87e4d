// cache_append.cu - new keys and values into a paged cache: osattn_cache_append
// (osattn.h).  Keys, and the queries that come with them, are rotated on the way;
// the pages hold 16-bit values, or e4m3 with a scale for each block of tokens and
// head.
//
// A scale is a power of two, the least 2^e with every magnitude of its block at
// most 448 2^e.  e4m3 has its own exponent, so a power of two costs no precision
// (a value is within 2^-4 of itself down to 2^-6 of a scale, where subnormals
// start), and a block whose later rows need a greater scale is brought to it by an
// exact factor: only what falls among the subnormals is rounded again.  So a cache
// that grew token by token holds what one written in one call holds, up to those.
//
// Bound: each K, V and Q element read and written once; a step of one token a
// sequence is latency alone.  A thread block takes the rows that a unit (a scale's
// block, or 64 tokens of 16-bit pages) receives of one head: the greatest magnitude
// first, with the rotated values kept in registers, then the codes.  Blocks behind
// them rotate the queries.  Measured (GPU time): 4 ragged prompts of up to 2048 tokens,
// H32 kv8 d128 into e4m3 pages 39 us, 4.1 TB/s; one token of 64 sequences 6.3 us.
#include <cmath>
#include <cstdint>

#include "api_shared.h"
#include "osattn.h"
#include "rotary.cuh"
#include "rotary_internal.h"

namespace osattn {
namespace append {

constexpr unsigned kBadArg = 1u;  // OSATTN_ERR_INVALID_ARG in the status word
constexpr int kThreads = 256;
constexpr int kLeastExp = -100;   // of the scale of a block of zeros
// Sweeps over a block whose values stay in registers: 64 tokens of 128 elements in a thread
// block, 8 in a warp; what lies beyond is read and turned twice.  (4 x 2048 whole tokens, H32 kv8 d128
// into e4m3 pages: blocks of 64 43 us, 47 with one sweep held and 49 with four; of 128 43, 45 and 43;
// 64 sequences of 16 tokens 14.4 us, 14.4 and 13.0.)
constexpr int kHeld = 2;
constexpr int kHalfChunk = 64;    // tokens of a 16-bit unit

struct Params {
  const void* in[2];  // K, V [B, Hkv, T, d]
  long long in_s[2][3];
  void* pages[2];  // [num_pages, Hkv, page, d]
  long long page_s[2][3];
  float* scale[2];  // [num_pages, Hkv, page / block]
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* count;      // or null: T
  const int32_t* positions;  // [B, T] or null: ctx + t
  int B, Hkv, T, num_pages, page, max_pages;
  int block;   // tokens of a unit; those of a scale in e4m3
  int blocks;  // units that the rows of a sequence can touch
  rotary::Turns turns;  // half = 0: keys are not rotated
  int wide;             // a chunk of 8 pairs is two 16-byte vectors of a row
  unsigned int* status;
  // queries
  rotary::Rows q[2];
  int q_chunks, q_groups, q_rows;
  long long q_work;
  unsigned kv_blocks;  // blocks of the grid before the queries'
};

// The place of chunk `slot` (16 elements: two vectors of 8) of a row.
__device__ __forceinline__ void slot_at(const Params& p, int slot, int& at0, int& at1) {
  at0 = 16 * slot;
  at1 = at0 + 8;
  if (p.wide && !p.turns.neighbours && slot < p.turns.half / 8) {
    at0 = 8 * slot;
    at1 = p.turns.half + at0;
  }
}

// Chunk `slot` of a row.
template <class E>
struct Slot {
  rotary::Vec<E, 8> v0, v1;
  int pos;
};

// It in fp32, rotated if it is a key's.
template <class E, int HD>
__device__ __forceinline__ void turn_slot(const Params& p, const uint64_t* turn, const uint16_t* row, int slot, bool key, const Slot<E>& raw,
                                          float* y) {
  raw.v0.to(y);
  raw.v1.to(y + 8);
  const int pos = raw.pos;
  const int half = p.turns.half;
  if (!key || half == 0) return;
  if (p.wide) {
    if (slot >= half / 8) return;
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      rotary::cos_sin(turn[slot * 8 + i], pos, p.turns.amplitude, c[i], s[i]);
    if (p.turns.neighbours) rotary::turn_pairs<8>(y, true, c, s);
    else rotary::turn_pairs<8>(y, false, c, s);
    return;
  }
  // pairs that lie anywhere: each element with the other of its pair, and its own sine and
  // cosine (4 x 2048 tokens, H32 kv8 d128, 24 elements turned: 121 us, where 16 or 32 take 43)
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    const int e = 16 * slot + i;
    if (e >= 2 * half) break;
    const bool second = p.turns.neighbours ? (e & 1) != 0 : e >= half;
    const int pair = p.turns.neighbours ? e >> 1 : (second ? e - half : e);
    const int other = p.turns.neighbours ? e ^ 1 : (second ? pair : pair + half);
    float c, s;
    rotary::cos_sin(turn[pair], pos, p.turns.amplitude, c, s);
    const float x = E::up(row[e]), o = E::up(row[other]);
    const float turned = second ? fmaf(o, s, x * c) : fmaf(x, c, -o * s);
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j == i) y[j] = turned;
  }
}

// Two floats as e4m3 (NaN stays NaN, infinities become 448).
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  return to_e4m3x2(a, b) | to_e4m3x2(c, d) << 16;
}
__device__ __forceinline__ void from_e4m3x4(uint32_t w, float* x) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * i))));
    x[2 * i] = __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
    x[2 * i + 1] = __half2float(__ushort_as_half(static_cast<uint16_t>(h >> 16)));
  }
}

// The scale of a block whose greatest finite magnitude is `amax`: 448 is 1.75 2^8.
__device__ __forceinline__ float scale_of(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, kLeastExp);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Keys and values of one unit: the tokens of a block of one sequence and head that
// are new.  kGroup threads (a warp or a block) share it.  `prepare` has them fill `turn`.
template <class E, int HD, bool kE4m3, int kGroup, class F>
__device__ __forceinline__ void store_unit(const Params& p, const uint64_t* turn, long long unit, F prepare) {
  constexpr int kSlots = HD / 16, kTok = kGroup / kSlots;  // chunks of a row, tokens of a sweep
  const int tid = threadIdx.x % kGroup;
  const int which = static_cast<int>(unit & 1);
  unit >>= 1;
  const long long of_heads = rotary::quotient(unit, p.Hkv);
  const int hk = static_cast<int>(unit - of_heads * p.Hkv), b = static_cast<int>(rotary::quotient(of_heads, p.blocks));
  const int j = static_cast<int>(of_heads - static_cast<long long>(b) * p.blocks);
  const int ctx = __ldg(p.ctx + b);
  const int count = p.count ? min(max(__ldg(p.count + b), 0), p.T) : p.T;
  if (ctx < 0 || ctx > p.max_pages * static_cast<long long>(p.page) - count) {
    if (tid == 0) atomicMax(p.status, kBadArg);
    return;
  }
  const int x0 = (ctx / p.block + j) * p.block;  // the block's first place in the sequence
  const int from = max(ctx, x0), to = min(ctx + count, x0 + p.block);
  if (from >= to) return;
  const int32_t* table = p.table + static_cast<long long>(b) * p.max_pages;
  const uint16_t* in = static_cast<const uint16_t*>(p.in[which]) + b * p.in_s[which][0] + hk * p.in_s[which][1];
  const int slot = tid % kSlots;
  int at0, at1;
  slot_at(p, slot, at0, at1);
  auto fetch = [&](int x, Slot<E>& raw) {
    const uint16_t* row = in + (x - ctx) * p.in_s[which][2];
    raw.v0.load(row + at0);
    raw.v1.load(row + at1);
    raw.pos = p.positions ? __ldg(p.positions + static_cast<long long>(b) * p.T + (x - ctx)) : x;
  };
  auto turned = [&](int x, const Slot<E>& raw, float* y) {
    turn_slot<E, HD>(p, turn, in + (x - ctx) * p.in_s[which][2], slot, which == 0, raw, y);
  };
  auto load = [&](int x, float* y) {
    Slot<E> raw;
    fetch(x, raw);
    turned(x, raw, y);
  };
  if constexpr (!kE4m3) {
    if (which == 0) prepare();
    for (int x = from + tid / kSlots; x < to; x += kTok) {
      const int page = __ldg(table + x / p.page);
      if (page < 0 || page >= p.num_pages) {
        atomicMax(p.status, kBadArg);
        continue;
      }
      float y[16];
      load(x, y);
      uint16_t* dst = static_cast<uint16_t*>(p.pages[which]) + page * p.page_s[which][0] + hk * p.page_s[which][1] +
                      (x % p.page) * p.page_s[which][2];
      rotary::Vec<E, 8> v;
      v.from(y);
      v.store(dst + at0);
      v.from(y + 8);
      v.store(dst + at1);
    }
  } else {
    const int page = __ldg(table + x0 / p.page);  // a block lies in one page
    if (page < 0 || page >= p.num_pages) {
      if (tid == 0) atomicMax(p.status, kBadArg);
      return;
    }
    uint8_t* dst = static_cast<uint8_t*>(p.pages[which]) + page * p.page_s[which][0] + hk * p.page_s[which][1];
    const int row0 = x0 % p.page;
    float* at_scale = p.scale[which] + (static_cast<long long>(page) * p.Hkv + hk) * (p.page / p.block) + row0 / p.block;
    const float had = ctx > x0 ? *at_scale : 0.f;  // older rows of the block have a scale
    float y[kHeld][16], amax = 0.f;
    auto widen = [&](const float* v) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float a = fabsf(v[i]);
        amax = a <= 3.402823466e38f ? fmaxf(amax, a) : amax;
      }
    };
    const int first = from + tid / kSlots;
    {
      Slot<E> raw[kHeld];
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (first + u * kTok < to) fetch(first + u * kTok, raw[u]);
      if (which == 0) prepare();
#pragma unroll
      for (int u = 0; u < kHeld; ++u)
        if (first + u * kTok < to) {
          turned(first + u * kTok, raw[u], y[u]);
          widen(y[u]);
        }
    }
    for (int x = first + kHeld * kTok; x < to; x += kTok) {
      float z[16];
      load(x, z);
      widen(z);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
    if constexpr (kGroup > 32) {
      __shared__ float part[kGroup / 32];
      if ((tid & 31) == 0) part[tid >> 5] = amax;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kGroup / 32; ++i) amax = fmaxf(amax, part[i]);
    } else {
      __syncwarp();
    }
    float scale = scale_of(amax);
    if (had >= scale && had <= 3.402823466e38f) {
      scale = had;
    } else if (ctx > x0) {
      // (the older rows are `had` times their codes, zeros if it is 0; a negative one that the new
      // scale does not reach, an infinite one or NaN leaves nothing of them but NaN)
      const float by = fabsf(had) <= scale ? had / scale : __uint_as_float(0x7fc00000u);
      for (int r = row0 + tid / kSlots; r < row0 + ctx - x0; r += kTok) {
        uint4* q = reinterpret_cast<uint4*>(dst + r * p.page_s[which][2] + 16 * slot);
        uint4 w = *q;
        uint32_t* e = &w.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v[4];
          from_e4m3x4(e[i], v);
          e[i] = to_e4m3x4(v[0] * by, v[1] * by, v[2] * by, v[3] * by);
        }
        *q = w;
      }
    }
    if (tid == 0) *at_scale = scale;
    const float inv = 1.f / scale;
    auto store = [&](int x, const float* v) {
      uint8_t* row = dst + (row0 + x - x0) * p.page_s[which][2];
      const uint2 lo = make_uint2(to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                  to_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
      const uint2 hi = make_uint2(to_e4m3x4(v[8] * inv, v[9] * inv, v[10] * inv, v[11] * inv),
                                  to_e4m3x4(v[12] * inv, v[13] * inv, v[14] * inv, v[15] * inv));
      *reinterpret_cast<uint2*>(row + at0) = lo;
      *reinterpret_cast<uint2*>(row + at1) = hi;
    };
#pragma unroll
    for (int u = 0; u < kHeld; ++u)
      if (first + u * kTok < to) store(first + u * kTok, y[u]);
    for (int x = first + kHeld * kTok; x < to; x += kTok) {
      float z[16];
      load(x, z);
      store(x, z);
    }
  }
}

// (Three blocks an SM: the prompts of 4 x 2048 tokens, H32 kv8 d128 into e4m3 pages, take
// 39 us so, 44 with two and 49 with four.)
template <class E, int HD, bool kE4m3, int kGroup>
__global__ void __launch_bounds__(kThreads, 3) append_kernel(const __grid_constant__ Params p) {
  __shared__ uint64_t turn[HD / 2];
  auto fill = [&] { rotary::fill_turns(turn, p.turns.freqs, p.turns.half); };
  if (blockIdx.x < p.kv_blocks) {
    if constexpr (kGroup == kThreads) {
      // (a unit a block: its keys, or values, which need no angles, are under way before them)
      if (blockIdx.x < 2ll * p.B * p.blocks * p.Hkv) store_unit<E, HD, kE4m3, kGroup>(p, turn, blockIdx.x, fill);
    } else {
      fill();
      const long long unit = static_cast<long long>(blockIdx.x) * (kThreads / kGroup) + threadIdx.x / kGroup;
      if (unit < 2ll * p.B * p.blocks * p.Hkv) store_unit<E, HD, kE4m3, kGroup>(p, turn, unit, [] {});
    }
    return;
  }
  const int local = threadIdx.x / p.q_chunks, chunk = threadIdx.x - local * p.q_chunks;
  const long long w_all = static_cast<long long>(blockIdx.x - p.kv_blocks) * p.q_rows + local;
  const bool works = local < p.q_rows && w_all < p.q_work;
  const long long w = works ? w_all : 0;
  const long long token = rotary::quotient(w, p.q_groups);
  const int group = static_cast<int>(w - token * p.q_groups), b = static_cast<int>(rotary::quotient(token, p.T));
  const int t = static_cast<int>(token - static_cast<long long>(b) * p.T);
  const int pos = p.positions ? __ldg(p.positions + token) : __ldg(p.ctx + b) + t;
  const int heads = works ? p.q[0].heads + p.q[1].heads : 0;
  if (p.wide) rotary::turn_heads<E, 8, 4>(p.turns, turn, p.q, b, t, pos, group, p.q_groups, heads, works ? chunk : 0, HD, fill);
  else rotary::turn_heads<E, 1, 4>(p.turns, turn, p.q, b, t, pos, group, p.q_groups, heads, works ? chunk : 0, HD, fill);
}

template <class E, int HD>
cudaError_t launch(Params& p, bool e4m3, bool queries, int num_sms, cudaStream_t stream) {
  // A warp for each unit where a sequence brings few rows, else a block (H32 kv8 d128 into e4m3
  // pages: 64 sequences of 1 row 6.2 us as warps, 10.3 as blocks, of 16 14.4 and 16.4, of 32 24.6 and
  // 18.5; 8 sequences of 16 10.3 and 6.2, of 8 6.2 either way).
  const bool warps = p.T <= 16;
  const int group = warps ? 32 : kThreads;
  const long long units = 2ll * p.B * p.blocks * p.Hkv;
  const long long kv = (units * group + kThreads - 1) / kThreads;
  long long all = kv;
  if (queries) {
    p.q_chunks = rotary::chunks_of(HD, p.turns.half, p.wide ? 8 : 1);
    p.q_rows = kThreads / p.q_chunks;
    const long long tokens = static_cast<long long>(p.B) * p.T;
    int per = 8;
    while (per > 1 && tokens * ((p.q[0].heads + per - 1) / per) < 4ll * p.q_rows * num_sms) per /= 2;
    p.q_groups = (p.q[0].heads + per - 1) / per;
    p.q_work = tokens * p.q_groups;
    all += (p.q_work + p.q_rows - 1) / p.q_rows;
  }
  if (all > 0x7fffffffLL) return cudaErrorInvalidValue;
  p.kv_blocks = static_cast<unsigned>(kv);
  const unsigned grid = static_cast<unsigned>(all);
  if (e4m3) {
    if (warps) append_kernel<E, HD, true, 32><<<grid, kThreads, 0, stream>>>(p);
    else append_kernel<E, HD, true, kThreads><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (warps) append_kernel<E, HD, false, 32><<<grid, kThreads, 0, stream>>>(p);
    else append_kernel<E, HD, false, kThreads><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace append
}  // namespace osattn

using namespace osattn;

extern "C" int osattn_cache_append(const void* K, const void* V, const void* Q, void* K_pages, void* V_pages,
                                   float* K_scale, float* V_scale, void* Q_out, const int32_t* page_table,
                                   const int32_t* ctx_len, const int32_t* new_len, const int32_t* positions, int B,
                                   int H, int Hkv, int T, int d, int num_pages, int page_size, int max_pages,
                                   int scale_block, const int64_t* k_strides, const int64_t* v_strides,
                                   const int64_t* q_strides, const int64_t* kp_strides, const int64_t* vp_strides,
                                   const int64_t* qo_strides, const osattn_rotation* rotation, int dtype,
                                   int cache_dtype, void* stream) {
  using append::aligned_to;
  if (!K || !V || !K_pages || !V_pages || !page_table || !ctx_len) return OSATTN_ERR_INVALID_ARG;
  if (B < 1 || Hkv < 1 || T < 1 || d < 1 || num_pages < 1 || page_size < 1 || max_pages < 1) return OSATTN_ERR_INVALID_ARG;
  if ((Q != nullptr) != (Q_out != nullptr) || (Q && (H < 1 || !rotation))) return OSATTN_ERR_INVALID_ARG;
  for (const void* p : {K, V, static_cast<const void*>(K_pages), static_cast<const void*>(V_pages)})
    if (!aligned_to(p, 16)) return OSATTN_ERR_INVALID_ARG;
  if (!aligned_to(Q, 16) || !aligned_to(Q_out, 16) || !aligned_to(page_table, 4) || !aligned_to(ctx_len, 4) ||
      !aligned_to(new_len, 4) || !aligned_to(positions, 4) || !aligned_to(K_scale, 4) || !aligned_to(V_scale, 4))
    return OSATTN_ERR_INVALID_ARG;
  if (rotation && check_rotation(rotation, d) != OSATTN_OK) return OSATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return OSATTN_ERR_UNSUPPORTED;
  if (dtype != OSATTN_BF16 && dtype != OSATTN_FP16) return OSATTN_ERR_UNSUPPORTED;
  const bool e4m3 = cache_dtype == OSATTN_E4M3;
  if (!e4m3 && cache_dtype != dtype) return OSATTN_ERR_UNSUPPORTED;
  if (e4m3 && (!K_scale || !V_scale || scale_block < 1 || page_size % scale_block != 0)) return OSATTN_ERR_INVALID_ARG;
  const long long keys = static_cast<long long>(max_pages) * page_size;
  if (keys < T || keys > (1ll << 30)) return OSATTN_ERR_INVALID_ARG;
  append::Params p;
  long long qs[3], qos[3];
  if (api_strides(k_strides, Hkv, T, d, dtype, p.in_s[0]) != OSATTN_OK ||
      api_strides(v_strides, Hkv, T, d, dtype, p.in_s[1]) != OSATTN_OK ||
      api_strides(kp_strides, Hkv, page_size, d, cache_dtype, p.page_s[0]) != OSATTN_OK ||
      api_strides(vp_strides, Hkv, page_size, d, cache_dtype, p.page_s[1]) != OSATTN_OK ||
      (Q && (api_strides(q_strides, H, T, d, dtype, qs) != OSATTN_OK ||
             api_strides(qo_strides, H, T, d, dtype, qos) != OSATTN_OK)))
    return OSATTN_ERR_INVALID_ARG;
  if (Q && Q == Q_out && ((B > 1 && qs[0] != qos[0]) || (H > 1 && qs[1] != qos[1]) || (T > 1 && qs[2] != qos[2])))
    return OSATTN_ERR_INVALID_ARG;  // (a row would be written before another thread has read it)
  ApiDevice dev;
  const int rc = api_device(&dev);
  if (rc != OSATTN_OK) return rc;
  p.in[0] = K;
  p.in[1] = V;
  p.pages[0] = K_pages;
  p.pages[1] = V_pages;
  p.scale[0] = K_scale;
  p.scale[1] = V_scale;
  p.table = page_table;
  p.ctx = ctx_len;
  p.count = new_len;
  p.positions = positions;
  p.B = B;
  p.Hkv = Hkv;
  p.T = T;
  p.num_pages = num_pages;
  p.page = page_size;
  p.max_pages = max_pages;
  p.block = e4m3 ? scale_block : append::kHalfChunk;
  p.blocks = static_cast<int>((static_cast<long long>(T) + p.block - 2) / p.block + 1);
  p.turns = rotary::Turns{nullptr, 0, 0, 1.f, 0};
  if (rotation) p.turns = rotary::Turns{rotation->freqs, rotation->rot / 2, rotation->interleaved ? 1 : 0, rotation->amplitude, 0};
  p.wide = p.turns.half % 8 == 0;
  p.status = dev.status;
  p.q[0] = p.q[1] = rotary::Rows{nullptr, nullptr, 0, 0, 0, 0, 0, 0, 0};
  if (Q) p.q[0] = rotary::Rows{Q, Q_out, qs[0], qs[1], qs[2], qos[0], qos[1], qos[2], H};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool fp16 = dtype == OSATTN_FP16;
  cudaError_t e;
  if (d == 128) e = fp16 ? append::launch<rotary::Fp16, 128>(p, e4m3, Q != nullptr, dev.num_sms, s)
                         : append::launch<rotary::Bf16, 128>(p, e4m3, Q != nullptr, dev.num_sms, s);
  else e = fp16 ? append::launch<rotary::Fp16, 64>(p, e4m3, Q != nullptr, dev.num_sms, s)
                : append::launch<rotary::Bf16, 64>(p, e4m3, Q != nullptr, dev.num_sms, s);
  return e == cudaSuccess ? OSATTN_OK : OSATTN_ERR_CUDA;
}
