// rotary.cu - rotary positions: osattn_rotary (osattn.h), forward and, by the
// negative angles, backward.  Memory-bound: every element is read and written once.
//
// A thread holds 16 bytes of a row and, for halves, the 16 that they pair with; the
// sine and cosine of its pairs serve several heads.  Measured (GPU time): B4 H32 kv8
// N4096 d128 bf16 53 us a call, 6.3 TB/s of reads and writes, 93 % of the measured copy
// rate; a decode step of 8 sequences 6.2 us, a launch's latency.
#include <cmath>
#include <cstdint>

#include "api_shared.h"
#include "osattn.h"
#include "rotary.cuh"
#include "rotary_internal.h"

namespace osattn {
namespace rotary {

struct Params {
  Turns turns;
  Rows x[2];
  const int32_t* positions;  // [N], or [B, N] with pos_b = N, or null
  long long pos_b;
  int offset;  // position of row 0 without them
  int N, d, chunks, groups;
  long long work;  // B N groups
  int heads_first; // groups of heads of a token adjacent, else tokens of a group
  int rows;        // (token, group) pairs of a block
};

constexpr int kThreads = 256;

template <class E, int V>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Params p) {
  __shared__ uint64_t turn[kMaxPairs];
  const int local = threadIdx.x / p.chunks, chunk = threadIdx.x - local * p.chunks;
  const long long w_all = static_cast<long long>(blockIdx.x) * p.rows + local;
  const bool works = local < p.rows && w_all < p.work;
  const long long w = works ? w_all : 0;
  long long token;
  int group;
  if (p.heads_first) {
    token = quotient(w, p.groups);
    group = static_cast<int>(w - token * p.groups);
  } else {
    const long long bg = quotient(w, p.N), n = w - bg * p.N;
    const long long b = quotient(bg, p.groups);
    group = static_cast<int>(bg - b * p.groups);
    token = b * p.N + n;
  }
  const int b = static_cast<int>(quotient(token, p.N));
  const long long n = token - static_cast<long long>(b) * p.N;
  const int at = p.positions ? __ldg(p.positions + b * p.pos_b + n) : p.offset + static_cast<int>(n);
  turn_heads<E, V, sizeof(typename E::T) == 4 ? 2 : 4>(p.turns, turn, p.x, b, n, at, group, p.groups,
                                                       works ? p.x[0].heads + p.x[1].heads : 0, works ? chunk : 0, p.d,
                                                       [&] { fill_turns(turn, p.turns.freqs, p.turns.half); });
}

template <class E, int V>
cudaError_t launch_v(const RotaryArgs& a, Params& p) {
  p.chunks = chunks_of(a.d, a.half, V);
  const int heads = a.x[0].heads + a.x[1].heads;
  p.rows = kThreads / p.chunks;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  // A thread turns its chunk of several heads by the same angles.  Four at a time keep
  // enough loads in flight; fewer where that would leave SMs without a block.
  int per = 4;
  while (per > 1 && tokens * ((heads + per - 1) / per) < 2ll * p.rows * a.num_sms) per /= 2;
  while (per < heads && tokens * ((heads + 2 * per - 1) / (2 * per)) >= 16ll * p.rows * a.num_sms && per < 16) per *= 2;
  p.groups = (heads + per - 1) / per;
  p.work = tokens * p.groups;
  const long long blocks = (p.work + p.rows - 1) / p.rows;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  rotary_kernel<E, V><<<static_cast<unsigned>(blocks), kThreads, 0, a.stream>>>(p);
  return cudaGetLastError();
}

template <class E>
cudaError_t launch_e(const RotaryArgs& a) {
  Params p;
  p.turns = Turns{a.freqs, a.half, a.neighbours, a.amplitude, a.inverse};
  p.x[0] = a.x[0];
  p.x[1] = a.x[1];
  p.positions = a.positions;
  p.pos_b = a.pos_b;
  p.offset = a.offset;
  p.N = a.N;
  p.d = a.d;
  p.heads_first = a.x[0].in_h <= a.x[0].in_n || a.N == 1;
  const int v = vector_of(a, sizeof(typename E::T));
  if constexpr (sizeof(typename E::T) == 2)
    if (v >= 8 && chunks_of(a.d, a.half, 8) <= kThreads) return launch_v<E, 8>(a, p);
  if (v >= 4 && chunks_of(a.d, a.half, 4) <= kThreads) return launch_v<E, 4>(a, p);
  if (v >= 2 && chunks_of(a.d, a.half, 2) <= kThreads) return launch_v<E, 2>(a, p);
  return launch_v<E, 1>(a, p);
}

}  // namespace rotary

int vector_of(const RotaryArgs& a, int bytes) {
  // elements of one access: they have to divide the pairs, what is not turned, and every address
  long long all = a.half | (a.d - 2 * a.half);
  uintptr_t base = 0;
  for (const rotary::Rows& r : a.x) {
    if (r.heads == 0) continue;
    all |= r.in_b | r.in_h | r.in_n | r.out_b | r.out_h | r.out_n;
    base |= reinterpret_cast<uintptr_t>(r.in) | reinterpret_cast<uintptr_t>(r.out);
  }
  int v = 16 / bytes;
  while (v > 1 && (all % v != 0 || base % (static_cast<uintptr_t>(v) * bytes) != 0)) v /= 2;
  return v;
}

cudaError_t launch_rotary(const RotaryArgs& a) {
  if (a.dtype == OSATTN_BF16) return rotary::launch_e<rotary::Bf16>(a);
  if (a.dtype == OSATTN_FP16) return rotary::launch_e<rotary::Fp16>(a);
  return rotary::launch_e<rotary::Fp32>(a);
}

int check_rotation(const osattn_rotation* r, int d) {
  if (!r || !r->freqs || reinterpret_cast<uintptr_t>(r->freqs) % 8 != 0 || r->rot < 2 || r->rot % 2 != 0 || r->rot > d ||
      !std::isfinite(r->amplitude))
    return OSATTN_ERR_INVALID_ARG;
  return OSATTN_OK;
}

namespace {

// Element strides {b, h, row} of a tensor that is read (0: an axis it is repeated
// along) or written; that of an axis of length 1 reaches nothing.
bool row_strides(const int64_t* in, int B, int H, int N, int d, bool written, long long* out) {
  const long long own[3] = {static_cast<long long>(H) * N * d, static_cast<long long>(N) * d, d};
  const int len[3] = {B, H, N};
  for (int i = 0; i < 3; ++i) {
    out[i] = len[i] == 1 ? 0 : (in ? in[i] : own[i]);
    if (out[i] < (written && len[i] > 1 ? 1 : 0) || out[i] >= (1ll << 40)) return false;
  }
  return true;
}

}  // namespace

bool fill_rows(rotary::Rows* r, const void* in, void* out, int B, int heads, int N, int d, const int64_t* is,
               const int64_t* os) {
  long long i[3], o[3];
  if (!row_strides(is, B, heads, N, d, false, i) || !row_strides(os, B, heads, N, d, true, o)) return false;
  *r = rotary::Rows{in, out, i[0], i[1], i[2], o[0], o[1], o[2], heads};
  // In place with other strides a row would be written before another thread has read it.
  return in != out || (i[0] == o[0] && i[1] == o[1] && i[2] == o[2]);
}

}  // namespace osattn

using namespace osattn;

extern "C" int osattn_rotary(const void* Q, const void* K, void* Q_out, void* K_out, int B, int H, int Hkv, int N,
                             int d, const int64_t* q_strides, const int64_t* k_strides, const int64_t* qo_strides,
                             const int64_t* ko_strides, const osattn_rotation* rotation, const int32_t* positions,
                             int batch_positions, int offset, int inverse, int dtype, void* stream) {
  if (!Q || !Q_out || B < 1 || H < 1 || Hkv < 0 || N < 1 || d < 2) return OSATTN_ERR_INVALID_ARG;
  if (Hkv > 0 && (!K || !K_out)) return OSATTN_ERR_INVALID_ARG;
  if (check_rotation(rotation, d) != OSATTN_OK) return OSATTN_ERR_INVALID_ARG;
  if (dtype != OSATTN_BF16 && dtype != OSATTN_FP16 && dtype != OSATTN_FP32) return OSATTN_ERR_UNSUPPORTED;
  if (d > kRotaryMaxDim) return OSATTN_ERR_UNSUPPORTED;
  const uintptr_t size = dtype == OSATTN_FP32 ? 4 : 2;
  for (const void* p : {Q, K, static_cast<const void*>(Q_out), static_cast<const void*>(K_out)})
    if (reinterpret_cast<uintptr_t>(p) % size != 0) return OSATTN_ERR_INVALID_ARG;
  if (positions && reinterpret_cast<uintptr_t>(positions) % 4 != 0) return OSATTN_ERR_INVALID_ARG;
  if (!positions && static_cast<long long>(offset) + N - 1 > 0x7fffffffLL) return OSATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(H) + Hkv > 0x3fffffffLL) return OSATTN_ERR_INVALID_ARG;
  RotaryArgs a;
  if (!fill_rows(&a.x[0], Q, Q_out, B, H, N, d, q_strides, qo_strides)) return OSATTN_ERR_INVALID_ARG;
  a.x[1] = rotary::Rows{nullptr, nullptr, 0, 0, 0, 0, 0, 0, 0};
  if (Hkv > 0 && !fill_rows(&a.x[1], K, K_out, B, Hkv, N, d, k_strides, ko_strides)) return OSATTN_ERR_INVALID_ARG;
  ApiDevice dev;
  const int rc = api_device(&dev);
  if (rc != OSATTN_OK) return rc;
  a.freqs = rotation->freqs;
  a.half = rotation->rot / 2;
  a.neighbours = rotation->interleaved ? 1 : 0;
  a.amplitude = rotation->amplitude;
  a.inverse = inverse ? 1 : 0;
  a.positions = positions;
  a.pos_b = batch_positions ? N : 0;
  a.offset = offset;
  a.B = B;
  a.N = N;
  a.d = d;
  a.dtype = dtype;
  a.num_sms = dev.num_sms;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_rotary(a) == cudaSuccess ? OSATTN_OK : OSATTN_ERR_CUDA;
}
