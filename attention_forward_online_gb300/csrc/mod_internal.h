// mod_internal.h - launch interface of the modified-score attention kernels
// (mask plan, forward, backward) and of tree attention.  Not part of the ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace osattn {

constexpr int kPlanTile = 128;      // query rows per summary entry of a mask plan
constexpr int kMaxRelRange = 1024;  // largest distance range of a learned bias

struct PlanArgs {
  void* plan;
  int B, Nq, Nkv, q_offset;
  int causal, window;
  const int32_t* key_len;     // [B] or null
  const int32_t* prefix_len;  // [B] or null
  const int32_t* doc_ids;     // [B, Nkv] or null
  cudaStream_t stream;
};
cudaError_t launch_mask_plan(const PlanArgs& a);

struct RelArgs {
  const void* table = nullptr;   // [num, H], the element type of Q
  const int32_t* map = nullptr;  // [2 range + 1]
  int num = 0, range = 0;
};

// One modified-score call after host validation.
struct ModArgs {
  int B, H, Hkv, Nq, Nkv, d, fp16;
  float scale, softcap;
  const float* slopes;  // [H] or null
  RelArgs rel;
  const void* plan;  // or null
  int q_offset;
  cudaStream_t stream;
  unsigned int* status;
  uint64_t wait_limit_ns;
  int num_sms;
  float* LSE;  // written by the forward pass, read by the backward pass
  // backward
  const void* O_in;
  long long o_s[3];  // its element strides of the b, h and row axes
  float* D;         // workspace [B, H, Nq]
  float* rel_part;  // workspace [B, H, key tiles, 2 range + 1]
  void* dRel;       // [num, H] or null
  void *dK, *dV;    // [B, Hkv, Nkv, d], and their element strides
  long long dk_s[3], dv_s[3];
};

// Tensor maps of the backward pass; g: dO.
struct BwdModMaps {
  CUtensorMap q, k, v, g, dq, dk, dv;
};

int mod_score_mode(const ModArgs& a);

}  // namespace osattn
