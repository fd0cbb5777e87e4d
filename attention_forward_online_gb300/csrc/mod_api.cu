// mod_api.cu - entry points of modified-score attention (osattn.h):
// osattn_mask_plan, osattn_fwd_mod and osattn_bwd_mod.  Host checks and
// launches only.
#include <cmath>
#include <cstdint>
#include <mutex>

#include "api_shared.h"
#include "mod_common.cuh"
#include "mod_internal.h"
#include "osattn.h"
#include "osattn_internal.h"

namespace osattn {

namespace fwdmod {
template <int HD, bool kF16>
cudaError_t prepare();
template <int HD, bool kF16>
cudaError_t launch(const ModArgs&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                   const CUtensorMap&);
}  // namespace fwdmod
namespace bwdmod {
template <int HD, bool kF16>
cudaError_t prepare();
template <int HD, bool kF16>
cudaError_t launch(const ModArgs&, const BwdModMaps&);
}  // namespace bwdmod

int mod_score_mode(const ModArgs& a) {
  if (a.rel.table) return kModRel;
  if (a.slopes) return a.softcap > 0.f ? kModCapSlopes : kModSlopes;
  return a.softcap > 0.f ? kModCap : kModPlain;
}

namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int kMaxOffset = 1 << 30;

// Kernel attributes of one (d, element type, direction), once per device.
std::mutex g_prepare_mutex;
bool g_prepared[kApiMaxDevices][8];

int prepare_once(int device, int slot, cudaError_t (*prepare)()) {
  std::lock_guard<std::mutex> lock(g_prepare_mutex);
  if (g_prepared[device][slot]) return OSATTN_OK;
  if (prepare() != cudaSuccess) return OSATTN_ERR_CUDA;
  g_prepared[device][slot] = true;
  return OSATTN_OK;
}

int validate_mod(const void* Q, const void* K, const void* V, const void* O, const float* LSE, int B,
                 int H, int Hkv, int Nq, int Nkv, int d, float scale, const osattn_score* s,
                 const void* plan, int dtype) {
  if (!Q || !K || !V || !O || !LSE) return OSATTN_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || Nq < 1 || Nkv < 1 || d < 1)
    return OSATTN_ERR_INVALID_ARG;
  if (Nq > kMaxOffset || Nkv > kMaxOffset) return OSATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return OSATTN_ERR_INVALID_ARG;
  if (!aligned_to(Q, 16) || !aligned_to(K, 16) || !aligned_to(V, 16) || !aligned_to(O, 16) ||
      !aligned_to(LSE, 4) || (plan && !aligned_to(plan, 16)))
    return OSATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H > 0x7fffffffLL) return OSATTN_ERR_INVALID_ARG;
  if (s) {
    if (!cap_ok(s->softcap)) return OSATTN_ERR_INVALID_ARG;
    if (s->q_offset < -kMaxOffset || s->q_offset > kMaxOffset) return OSATTN_ERR_INVALID_ARG;
    if (s->slopes && !aligned_to(s->slopes, 4)) return OSATTN_ERR_INVALID_ARG;
    if (s->rel_table) {
      if (s->slopes) return OSATTN_ERR_INVALID_ARG;
      if (!s->rel_map || !aligned_to(s->rel_table, 2) || !aligned_to(s->rel_map, 4) || s->rel_num < 1 ||
          s->rel_range < 1)
        return OSATTN_ERR_INVALID_ARG;
      if (s->softcap > 0.f || s->rel_range > kMaxRelRange) return OSATTN_ERR_UNSUPPORTED;
    }
  }
  if (d != 64 && d != 128) return OSATTN_ERR_UNSUPPORTED;
  if (dtype != OSATTN_BF16 && dtype != OSATTN_FP16) return OSATTN_ERR_UNSUPPORTED;
  return OSATTN_OK;
}

void common_args(ModArgs* a, int B, int H, int Hkv, int Nq, int Nkv, int d, float scale,
                 const osattn_score* s, const void* plan, int dtype, void* stream, const ApiDevice& dev) {
  *a = ModArgs{};
  a->B = B;
  a->H = H;
  a->Hkv = Hkv;
  a->Nq = Nq;
  a->Nkv = Nkv;
  a->d = d;
  a->fp16 = dtype == OSATTN_FP16;
  a->scale = scale;
  if (s) {
    a->softcap = s->softcap;
    a->slopes = s->slopes;
    a->q_offset = s->q_offset;
    if (s->rel_table) {
      a->rel.table = s->rel_table;
      a->rel.map = s->rel_map;
      a->rel.num = s->rel_num;
      a->rel.range = s->rel_range;
    }
  }
  a->plan = plan;
  a->stream = static_cast<cudaStream_t>(stream);
  a->status = dev.status;
  a->wait_limit_ns = dev.wait_limit_ns;
  a->num_sms = dev.num_sms;
}

}  // namespace
}  // namespace osattn

using namespace osattn;

extern "C" {

size_t osattn_mask_plan_bytes(int B, int Nq) {
  if (B < 1 || Nq < 1) return 0;
  const size_t tiles = (static_cast<size_t>(Nq) + kPlanTile - 1) / kPlanTile;
  return static_cast<size_t>(B) * (tiles * 16 + static_cast<size_t>(Nq) * 8);
}

int osattn_mask_plan(void* plan, size_t plan_bytes, int B, int Nq, int Nkv, int q_offset, int causal,
                     int window, const int32_t* key_len, const int32_t* prefix_len,
                     const int32_t* doc_ids, void* stream) {
  if (!plan || !aligned_to(plan, 16) || B < 1 || Nq < 1 || Nkv < 1 || Nq > kMaxOffset ||
      Nkv > kMaxOffset || q_offset < -kMaxOffset || q_offset > kMaxOffset || window < 0 ||
      plan_bytes < osattn_mask_plan_bytes(B, Nq))
    return OSATTN_ERR_INVALID_ARG;
  if ((key_len && !aligned_to(key_len, 4)) || (prefix_len && !aligned_to(prefix_len, 4)) ||
      (doc_ids && !aligned_to(doc_ids, 4)) || (prefix_len && !causal))
    return OSATTN_ERR_INVALID_ARG;
  PlanArgs a;
  a.plan = plan;
  a.B = B;
  a.Nq = Nq;
  a.Nkv = Nkv;
  a.q_offset = q_offset;
  a.causal = causal ? 1 : 0;
  a.window = window;
  a.key_len = key_len;
  a.prefix_len = prefix_len;
  a.doc_ids = doc_ids;
  a.stream = static_cast<cudaStream_t>(stream);
  return launch_mask_plan(a) == cudaSuccess ? OSATTN_OK : OSATTN_ERR_CUDA;
}

int osattn_fwd_mod(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int H,
                   int Hkv, int Nq, int Nkv, int d, const int64_t* q_strides,
                   const int64_t* k_strides, const int64_t* v_strides, const int64_t* o_strides,
                   float scale, const osattn_score* score, const void* plan, int dtype, void* stream) {
  int rc = validate_mod(Q, K, V, O, LSE, B, H, Hkv, Nq, Nkv, d, scale, score, plan, dtype);
  if (rc != OSATTN_OK) return rc;
  long long qs[3], ks[3], vs[3], os[3];
  if (api_strides(q_strides, H, Nq, d, dtype, qs) != OSATTN_OK ||
      api_strides(k_strides, Hkv, Nkv, d, dtype, ks) != OSATTN_OK ||
      api_strides(v_strides, Hkv, Nkv, d, dtype, vs) != OSATTN_OK ||
      api_strides(o_strides, H, Nq, d, dtype, os) != OSATTN_OK)
    return OSATTN_ERR_INVALID_ARG;
  ApiDevice dev;
  rc = api_device(&dev);
  if (rc != OSATTN_OK) return rc;
  ModArgs a;
  common_args(&a, B, H, Hkv, Nq, Nkv, d, scale, score, plan, dtype, stream, dev);
  a.LSE = LSE;
  CUtensorMap tq, tk, tv, to;
  if (api_encode_map(&tq, Q, a.fp16, d, Nq, H, B, qs, kBoxRows) != OSATTN_OK ||
      api_encode_map(&tk, K, a.fp16, d, Nkv, Hkv, B, ks, kBoxRows) != OSATTN_OK ||
      api_encode_map(&tv, V, a.fp16, d, Nkv, Hkv, B, vs, kBoxRows) != OSATTN_OK ||
      api_encode_map(&to, O, a.fp16, d, Nq, H, B, os, kBoxRows) != OSATTN_OK)
    return OSATTN_ERR_CUDA;
  const int slot = (d == 128 ? 2 : 0) + a.fp16;
  cudaError_t (*const prep[4])() = {fwdmod::prepare<64, false>, fwdmod::prepare<64, true>,
                                    fwdmod::prepare<128, false>, fwdmod::prepare<128, true>};
  rc = prepare_once(dev.device, slot, prep[slot]);
  if (rc != OSATTN_OK) return rc;
  cudaError_t e;
  switch (slot) {
    case 0: e = fwdmod::launch<64, false>(a, tq, tk, tv, to); break;
    case 1: e = fwdmod::launch<64, true>(a, tq, tk, tv, to); break;
    case 2: e = fwdmod::launch<128, false>(a, tq, tk, tv, to); break;
    default: e = fwdmod::launch<128, true>(a, tq, tk, tv, to); break;
  }
  return e == cudaSuccess ? OSATTN_OK : OSATTN_ERR_CUDA;
}

size_t osattn_bwd_mod_workspace_bytes(int B, int H, int Nq, int Nkv, int rel_range) {
  if (B < 1 || H < 1 || Nq < 1 || Nkv < 1 || rel_range < 0) return 0;
  const size_t rows = static_cast<size_t>(B) * H * Nq;
  const size_t tiles = static_cast<size_t>(B) * H * ((static_cast<size_t>(Nkv) + 127) / 128);
  return (rows + (rel_range ? tiles * (2 * static_cast<size_t>(rel_range) + 1) : 0)) * sizeof(float);
}

int osattn_bwd_mod(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                   const float* LSE, void* dQ, void* dK, void* dV, void* dRel, int B, int H, int Hkv,
                   int Nq, int Nkv, int d, const int64_t* q_strides, const int64_t* k_strides,
                   const int64_t* v_strides, const int64_t* o_strides, const int64_t* do_strides,
                   const int64_t* dq_strides, const int64_t* dk_strides, const int64_t* dv_strides,
                   float scale, const osattn_score* score, const void* plan, int dtype,
                   void* workspace, size_t workspace_bytes, void* stream) {
  int rc = validate_mod(Q, K, V, O, LSE, B, H, Hkv, Nq, Nkv, d, scale, score, plan, dtype);
  if (rc != OSATTN_OK) return rc;
  if (!dO || !dQ || !dK || !dV || !aligned_to(dO, 16) || !aligned_to(dQ, 16) || !aligned_to(dK, 16) ||
      !aligned_to(dV, 16))
    return OSATTN_ERR_INVALID_ARG;
  const bool rel = score && score->rel_table;
  if (rel != (dRel != nullptr) || (dRel && !aligned_to(dRel, 2))) return OSATTN_ERR_INVALID_ARG;
  if (!workspace || !aligned_to(workspace, 16) ||
      workspace_bytes < osattn_bwd_mod_workspace_bytes(B, H, Nq, Nkv, rel ? score->rel_range : 0))
    return OSATTN_ERR_INVALID_ARG;
  const int64_t* in[8] = {q_strides, k_strides, v_strides, o_strides,
                          do_strides, dq_strides, dk_strides, dv_strides};
  long long st[8][3];
  for (int i = 0; i < 8; ++i) {
    const bool kv = i == 1 || i == 2 || i == 6 || i == 7;
    if (api_strides(in[i], kv ? Hkv : H, kv ? Nkv : Nq, d, dtype, st[i]) != OSATTN_OK)
      return OSATTN_ERR_INVALID_ARG;
  }
  ApiDevice dev;
  rc = api_device(&dev);
  if (rc != OSATTN_OK) return rc;
  ModArgs a;
  common_args(&a, B, H, Hkv, Nq, Nkv, d, scale, score, plan, dtype, stream, dev);
  a.O_in = O;
  a.LSE = const_cast<float*>(LSE);
  a.dRel = dRel;
  a.dK = dK;
  a.dV = dV;
  for (int i = 0; i < 3; ++i) {
    a.o_s[i] = st[3][i];
    a.dk_s[i] = st[6][i];
    a.dv_s[i] = st[7][i];
  }
  a.D = static_cast<float*>(workspace);
  a.rel_part = a.D + static_cast<size_t>(B) * H * Nq;
  BwdModMaps maps;
  auto encode = [&](CUtensorMap* map, const void* base, int i, bool kv) {
    return api_encode_map(map, base, a.fp16, d, kv ? Nkv : Nq, kv ? Hkv : H, B, st[i], kBoxRows) == OSATTN_OK;
  };
  if (!encode(&maps.q, Q, 0, false) || !encode(&maps.k, K, 1, true) || !encode(&maps.v, V, 2, true) ||
      !encode(&maps.g, dO, 4, false) || !encode(&maps.dq, dQ, 5, false) || !encode(&maps.dk, dK, 6, true) ||
      !encode(&maps.dv, dV, 7, true))
    return OSATTN_ERR_CUDA;
  const int slot = (d == 128 ? 2 : 0) + a.fp16;
  cudaError_t (*const prep[4])() = {bwdmod::prepare<64, false>, bwdmod::prepare<64, true>,
                                    bwdmod::prepare<128, false>, bwdmod::prepare<128, true>};
  rc = prepare_once(dev.device, 4 + slot, prep[slot]);
  if (rc != OSATTN_OK) return rc;
  cudaError_t e;
  switch (slot) {
    case 0: e = bwdmod::launch<64, false>(a, maps); break;
    case 1: e = bwdmod::launch<64, true>(a, maps); break;
    case 2: e = bwdmod::launch<128, false>(a, maps); break;
    default: e = bwdmod::launch<128, true>(a, maps); break;
  }
  return e == cudaSuccess ? OSATTN_OK : OSATTN_ERR_CUDA;
}

}  // extern "C"
