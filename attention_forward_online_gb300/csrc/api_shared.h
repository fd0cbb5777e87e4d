// api_shared.h - host-side helpers of osattn_api.cu that the entry points in
// other files use: per-device state, stride checks and tensor maps.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace osattn {

constexpr int kApiMaxDevices = 64;

struct ApiDevice {
  int device = 0, num_sms = 0;
  unsigned int* status = nullptr;  // device status word [0] and give-up site [1]
  uint64_t wait_limit_ns = 0;
};

// Whether `softcap` is 0 (none) or a cap that the kernels take (NaN is not).
inline bool cap_ok(float softcap) { return softcap == 0.f || (softcap >= 1e-3f && softcap <= 1e4f); }

// The current device, set up for the library's kernels.
int api_device(ApiDevice* out);

// Element strides {b, h, row}: the caller's after the checks of
// osattn_fwd_strided, or those of a contiguous [B, H, N, d] tensor.
int api_strides(const int64_t* in, int H, int N, int d, int dtype, long long* out);

// 4-D tensor map (d, N, H, B) of a 16-bit tensor with those strides: 64 x
// box_rows x box_heads boxes, 128-byte swizzle, zero fill.
int api_encode_map(CUtensorMap* map, const void* base, int fp16, int d, int N, int H, int B,
                   const long long* st, int box_rows, int box_heads = 1);

}  // namespace osattn
