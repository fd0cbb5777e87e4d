// tree_e4m3_launch.cuh - which form of attention over e4m3 pages a call takes, and its
// launches: few rows a key head (tree_e4m3_tcgen05.cuh) or many (tree_e4m3_wide.cuh).
#pragma once

#include "tree_e4m3_tcgen05.cuh"
#include "tree_e4m3_wide.cuh"

namespace osattn {
namespace tree8 {

constexpr int kLaunchRegs = 128;  // the kernels' setmaxnreg splits assume it

template <int HD, bool kF16, int NG, int MODE>
cudaError_t set_attrs() {
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, tree_e4m3_kernel<HD, kF16, NG, MODE>);
  if (e != cudaSuccess) return e;
  if (NG > 1 && fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(tree_e4m3_kernel<HD, kF16, NG, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Mem<HD, kF16, NG>::kBytes);
}

template <int HD, bool kF16, int NG>
cudaError_t set_modes() {
  cudaError_t e;
  if ((e = set_attrs<HD, kF16, NG, kModPlain>()) != cudaSuccess) return e;
  if ((e = set_attrs<HD, kF16, NG, kModCap>()) != cudaSuccess) return e;
  if ((e = set_attrs<HD, kF16, NG, kModSlopes>()) != cudaSuccess) return e;
  return set_attrs<HD, kF16, NG, kModCapSlopes>();
}

template <int HD, bool kF16, int MODE>
cudaError_t set_wide() {
  cudaFuncAttributes fa;
  cudaError_t e = cudaFuncGetAttributes(&fa, wide::tree_e4m3_wide_kernel<HD, kF16, MODE>);
  if (e != cudaSuccess) return e;
  if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
  return cudaFuncSetAttribute(wide::tree_e4m3_wide_kernel<HD, kF16, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              wide::Mem<HD, kF16>::kBytes);
}

template <int HD, bool kF16>
cudaError_t prepare() {
  cudaError_t e;
  if ((e = set_modes<HD, kF16, 1>()) != cudaSuccess) return e;
  if ((e = set_modes<HD, kF16, 2>()) != cudaSuccess) return e;
  if ((e = set_wide<HD, kF16, kModPlain>()) != cudaSuccess) return e;
  if ((e = set_wide<HD, kF16, kModCap>()) != cudaSuccess) return e;
  if ((e = set_wide<HD, kF16, kModSlopes>()) != cudaSuccess) return e;
  return set_wide<HD, kF16, kModCapSlopes>();
}

inline Divisor divisor(int d) {
  uint32_t bits = 0;
  while ((1ll << bits) < d) ++bits;
  const uint64_t mul = d == 1 ? 0 : ((1ull << (31 + bits)) + d - 1) / d;  // at most 2^32 - 1
  return Divisor{static_cast<uint32_t>(mul), bits == 0 ? 0 : bits - 1, static_cast<uint32_t>(d)};
}

template <int HD, bool kF16, int NG>
void launch_rows(int grid, const TreeE4m3Args& a, const CUtensorMap& k, const CUtensorMap& v, const Params& p) {
  constexpr int kBytes = Mem<HD, kF16, NG>::kBytes;
  const bool cap = a.softcap > 0.f;
  if (cap && a.slopes) tree_e4m3_kernel<HD, kF16, NG, kModCapSlopes><<<grid, kThreads, kBytes, a.stream>>>(k, v, p);
  else if (cap) tree_e4m3_kernel<HD, kF16, NG, kModCap><<<grid, kThreads, kBytes, a.stream>>>(k, v, p);
  else if (a.slopes) tree_e4m3_kernel<HD, kF16, NG, kModSlopes><<<grid, kThreads, kBytes, a.stream>>>(k, v, p);
  else tree_e4m3_kernel<HD, kF16, NG, kModPlain><<<grid, kThreads, kBytes, a.stream>>>(k, v, p);
}

template <int HD, bool kF16>
void launch_wide(int grid, const TreeE4m3Args& a, const CUtensorMap& k, const CUtensorMap& v, const wide::Params& p) {
  constexpr int kBytes = wide::Mem<HD, kF16>::kBytes;
  const bool cap = a.softcap > 0.f;
  if (cap && a.slopes) wide::tree_e4m3_wide_kernel<HD, kF16, kModCapSlopes><<<grid, kThreads, kBytes, a.stream>>>(k, v, p);
  else if (cap) wide::tree_e4m3_wide_kernel<HD, kF16, kModCap><<<grid, kThreads, kBytes, a.stream>>>(k, v, p);
  else if (a.slopes) wide::tree_e4m3_wide_kernel<HD, kF16, kModSlopes><<<grid, kThreads, kBytes, a.stream>>>(k, v, p);
  else wide::tree_e4m3_wide_kernel<HD, kF16, kModPlain><<<grid, kThreads, kBytes, a.stream>>>(k, v, p);
}

// Behind a main kernel: the combine kernel, which may start before that has ended.
template <int HD, bool kF16, class P>
cudaError_t launch_join(int grid, cudaStream_t stream, const P& p) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long units = static_cast<long long>(p.B) * p.Hkv * p.row_tiles;
  // 16 or more partials a unit, if the units are about alike: 8 warps a row (H32 kv8 d128, one
  // token ctx 700: 14.4 us against 16.3; 16 tokens ctx 32000: 39.7 against 46.7)
  const int ways = grid >= 16 * units ? 8 : 1;
  const long long blocks = units * ((static_cast<long long>(p.tile_rows) * ways + 7) / 8);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute dep;
  dep.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  dep.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &dep;
  cfg.numAttrs = 1;
  return ways == 1 ? cudaLaunchKernelEx(&cfg, tree_e4m3_combine<HD, kF16, 1, P>, p, grid)
                   : cudaLaunchKernelEx(&cfg, tree_e4m3_combine<HD, kF16, 8, P>, p, grid);
}

template <int HD, bool kF16>
cudaError_t launch(const TreeE4m3Args& a, const CUtensorMap& k, const CUtensorMap& v) {
  Params p;
  p.Q = static_cast<const uint16_t*>(a.Q);
  p.q_sb = a.q_s[0];
  p.q_sh = a.q_s[1];
  p.q_sn = a.q_s[2];
  p.O = static_cast<uint16_t*>(a.O);
  p.o_sb = a.o_s[0];
  p.o_sh = a.o_s[1];
  p.o_sn = a.o_s[2];
  p.LSE = a.LSE;
  p.table = a.table;
  p.ctx = a.ctx;
  p.mask = reinterpret_cast<const long long*>(a.mask);
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.scales = a.page / a.block;
  p.by_page = divisor(a.page);
  p.by_block = divisor(a.block);
  p.B = a.B;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.group = a.H / a.Hkv;
  p.T = a.T;
  p.rows = a.T * p.group;
  // The form for few rows up to 16 of them (H32 kv8 d128, 16 rows: B8 ctx 6000 36.5 us, 49
  // in the other form, B64 ctx 4000 112 and 176); then the other, which reads a key once for 128
  // rows (20 rows: B64 ctx 4000 174 us, 193 as two tiles, B8 ctx 6000 48 and 47; B2 H16 kv2
  // ctx 100000 d64, 64 rows: 43, 72 as four tiles).
  const bool many = p.rows > kTreeE4m3FewRows && a.block % wide::kChunk == 0;
  const int most_rows = many ? kTreeE4m3Rows : kTreeE4m3FewRows;
  p.row_tiles = (p.rows + most_rows - 1) / most_rows;
  p.tile_rows = (p.rows + p.row_tiles - 1) / p.row_tiles;
  p.max_pages = a.max_pages;
  p.page = a.page;
  p.num_pages = a.num_pages;
  p.box_rows = a.page < BN ? a.page : BN;
  p.window = a.window;
  p.scale_log2 = a.scale * kLog2e;
  p.cap2 = a.softcap * kLog2e;
  p.inv_cap2 = a.softcap > 0.f ? 1.f / p.cap2 : 0.f;
  const CapArgs cap = make_cap(a.softcap, a.softcap, false);
  for (int i = 0; i < 4; ++i) p.cap_k[i] = cap.k[i];
  p.slopes = a.slopes;
  // Where the heads of a token lie side by side, the CTAs of up to 8 heads take the same
  // keys at the same time: pieces of 128 bytes a head far apart in time cost HBM a third
  // (B64 H32 kv8 ctx 8192 d128: 197 us with one list of all heads, 137 like this, 136 where
  // the rows of a head lie one after the other).
  p.lanes = 1;
  if (a.k_s[1] < a.k_s[2])
    for (int n = 2; n <= 8; ++n)
      if (a.Hkv % n == 0) p.lanes = n;
  p.list_heads = a.Hkv / p.lanes;
  const int grid = (a.num_sms < kTreeMaxCtas ? a.num_sms : kTreeMaxCtas) / p.lanes * p.lanes;
  p.head = static_cast<int*>(a.workspace);
  p.o_part = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + tree_head_bytes(a.B));
  p.lse_part = p.o_part + static_cast<long long>(2) * kTreeMaxCtas * p.tile_rows * HD;
  p.status = a.status;
  p.wait_limit_ns = a.wait_limit_ns;
  if (many) {
    wide::Params w;
    static_cast<Params&>(w) = p;
    w.lead = kTreeE4m3Lead;
    launch_wide<HD, kF16>(grid, a, k, v, w);
    return launch_join<HD, kF16>(grid, a.stream, w);
  }
  if (p.tile_rows <= 8) launch_rows<HD, kF16, 1>(grid, a, k, v, p);
  else launch_rows<HD, kF16, 2>(grid, a, k, v, p);
  return launch_join<HD, kF16>(grid, a.stream, p);
}

}  // namespace tree8
}  // namespace osattn
