// tree_api.cu - entry point of tree attention over a paged cache (osattn.h):
// osattn_tree_attn.  Host checks and launches only.
#include <cmath>
#include <cstdint>
#include <mutex>

#include "api_shared.h"
#include "osattn.h"
#include "osattn_internal.h"
#include "tree_internal.h"

namespace osattn {
namespace tree {
template <int HD, bool kF16>
cudaError_t prepare();
template <int HD, bool kF16>
cudaError_t launch(const TreeArgs&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&);
}  // namespace tree

namespace {

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

std::mutex g_prepare_mutex;
bool g_prepared[kApiMaxDevices][4];

int prepare_once(int device, int slot, cudaError_t (*prepare)()) {
  std::lock_guard<std::mutex> lock(g_prepare_mutex);
  if (g_prepared[device][slot]) return OSATTN_OK;
  if (prepare() != cudaSuccess) return OSATTN_ERR_CUDA;
  g_prepared[device][slot] = true;
  return OSATTN_OK;
}

}  // namespace
}  // namespace osattn

using namespace osattn;

extern "C" {

size_t osattn_tree_workspace_bytes(int B, int H, int Hkv, int T, int d) {
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || H / Hkv > kTreeMaxGroup || T < 1 ||
      T > kTreeMaxTokens || d < 1)
    return 0;
  const size_t rows = static_cast<size_t>(2) * kTreeMaxCtas * tree_slot_rows(H / Hkv, T);
  return tree_head_bytes(B) + rows * (static_cast<size_t>(d) + 1) * sizeof(float);
}

int osattn_tree_attn(const void* Q, const void* K_pages, const void* V_pages,
                     const int32_t* page_table, const int32_t* ctx_len, const int64_t* tree_mask,
                     void* O, float* LSE, int B, int H, int Hkv, int T, int d, int num_pages,
                     int page_size, int max_pages, const int64_t* q_strides,
                     const int64_t* k_strides, const int64_t* v_strides, const int64_t* o_strides,
                     float scale, float softcap, const float* slopes, int window, int dtype,
                     void* workspace, size_t workspace_bytes, void* stream) {
  if (!Q || !K_pages || !V_pages || !page_table || !ctx_len || !O || !LSE || !workspace)
    return OSATTN_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || T < 1 || d < 1 || num_pages < 1 || page_size < 1 ||
      max_pages < 1 || window < 0)
    return OSATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !cap_ok(softcap)) return OSATTN_ERR_INVALID_ARG;
  if (!aligned_to(Q, 16) || !aligned_to(K_pages, 16) || !aligned_to(V_pages, 16) || !aligned_to(O, 16) ||
      !aligned_to(LSE, 4) || !aligned_to(page_table, 4) || !aligned_to(ctx_len, 4) ||
      (tree_mask && !aligned_to(tree_mask, 8)) || (slopes && !aligned_to(slopes, 4)) ||
      !aligned_to(workspace, 16))
    return OSATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return OSATTN_ERR_UNSUPPORTED;
  if (dtype != OSATTN_BF16 && dtype != OSATTN_FP16) return OSATTN_ERR_UNSUPPORTED;
  if (T > kTreeMaxTokens || H / Hkv > kTreeMaxGroup) return OSATTN_ERR_UNSUPPORTED;
  // a 128-key tile is made of whole pages, or a page of whole tiles
  if (page_size < 8 || (page_size < 128 ? 128 % page_size : page_size % 128) != 0)
    return OSATTN_ERR_UNSUPPORTED;
  // the drafts have to fit the table, and positions and the list of key tiles 31 bits
  const long long keys = static_cast<long long>(max_pages) * page_size;
  const int group = H / Hkv, tok = tree_tok_tile(group);
  const long long tiles = static_cast<long long>(B) * Hkv * ((T + tok - 1) / tok);
  if (keys < T || keys > (1ll << 30) || tiles > (1ll << 30) / ((keys + 127) / 128))
    return OSATTN_ERR_INVALID_ARG;
  if (workspace_bytes < osattn_tree_workspace_bytes(B, H, Hkv, T, d)) return OSATTN_ERR_INVALID_ARG;
  long long qs[3], ks[3], vs[3], os[3];
  if (api_strides(q_strides, H, T, d, dtype, qs) != OSATTN_OK ||
      api_strides(k_strides, Hkv, page_size, d, dtype, ks) != OSATTN_OK ||
      api_strides(v_strides, Hkv, page_size, d, dtype, vs) != OSATTN_OK ||
      api_strides(o_strides, H, T, d, dtype, os) != OSATTN_OK)
    return OSATTN_ERR_INVALID_ARG;
  ApiDevice dev;
  int rc = api_device(&dev);
  if (rc != OSATTN_OK) return rc;
  TreeArgs a;
  a.O = O;
  for (int i = 0; i < 3; ++i) a.o_s[i] = os[i];
  a.LSE = LSE;
  a.table = page_table;
  a.ctx = ctx_len;
  a.mask = tree_mask;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.T = T;
  a.max_pages = max_pages;
  a.page = page_size;
  a.num_pages = num_pages;
  a.window = window;
  a.scale = scale;
  a.softcap = softcap;
  a.slopes = slopes;
  a.workspace = workspace;
  a.stream = static_cast<cudaStream_t>(stream);
  a.status = dev.status;
  a.wait_limit_ns = dev.wait_limit_ns;
  a.num_sms = dev.num_sms;
  // Q as (d, H, T, B): a box is the heads of one group of tok tokens, which
  // land as rows token * group + head
  const int fp16 = dtype == OSATTN_FP16, box = page_size < 128 ? page_size : 128;
  const long long qm[3] = {qs[0], qs[2], qs[1]};
  CUtensorMap tq, tk, tv;
  if (api_encode_map(&tq, Q, fp16, d, H, T, B, qm, group, tok) != OSATTN_OK ||
      api_encode_map(&tk, K_pages, fp16, d, page_size, Hkv, num_pages, ks, box) != OSATTN_OK ||
      api_encode_map(&tv, V_pages, fp16, d, page_size, Hkv, num_pages, vs, box) != OSATTN_OK)
    return OSATTN_ERR_CUDA;
  const int slot = (d == 128 ? 2 : 0) + fp16;
  cudaError_t (*const prep[4])() = {tree::prepare<64, false>, tree::prepare<64, true>,
                                    tree::prepare<128, false>, tree::prepare<128, true>};
  rc = prepare_once(dev.device, slot, prep[slot]);
  if (rc != OSATTN_OK) return rc;
  cudaError_t e;
  switch (slot) {
    case 0: e = tree::launch<64, false>(a, tq, tk, tv); break;
    case 1: e = tree::launch<64, true>(a, tq, tk, tv); break;
    case 2: e = tree::launch<128, false>(a, tq, tk, tv); break;
    default: e = tree::launch<128, true>(a, tq, tk, tv); break;
  }
  return e == cudaSuccess ? OSATTN_OK : OSATTN_ERR_CUDA;
}

}  // extern "C"
