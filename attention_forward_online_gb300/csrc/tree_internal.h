// tree_internal.h - launch interface of tree attention over a paged cache.
// Not part of the ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace osattn {

constexpr int kTreeMaxTokens = 64;  // drafts of a sequence: the bits of a mask
constexpr int kTreeMaxGroup = 128;  // query heads of a key head: the rows of a tile
constexpr int kTreeMaxCtas = 160;   // CTAs of the persistent kernel (one per SM)

// Tokens of a 128-row tile, rows of a partial result.
constexpr int tree_tok_tile(int group) { return 128 / group; }
constexpr int tree_slot_rows(int group, int T) {
  return (T < tree_tok_tile(group) ? T : tree_tok_tile(group)) * group;
}
constexpr size_t tree_head_bytes(int B) { return ((static_cast<size_t>(B) + 1) * 4 + 15) / 16 * 16; }

struct TreeArgs {
  void* O;
  long long o_s[3];
  float* LSE;
  const int32_t* table;  // [B, max_pages]
  const int32_t* ctx;    // [B]
  const int64_t* mask;   // [B, T] or null
  int B, H, Hkv, T;
  int max_pages, page, num_pages, window;
  float scale, softcap;
  const float* slopes;
  void* workspace;
  cudaStream_t stream;
  unsigned int* status;
  uint64_t wait_limit_ns;
  int num_sms;
};

}  // namespace osattn
