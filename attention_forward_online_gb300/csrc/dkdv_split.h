// dkdv_split.h - how many CTAs of the dK/dV kernel share a key tile.  Host code.
#pragma once

namespace osattn {
namespace bwdmod {

// CTAs that share a key tile's (head, query tile) pairs, of which it has at
// most `pairs`, as a power of two: one that divides `of`, leaves a CTA two
// pairs, and makes the kernel shortest if a CTA takes 1 / s of a tile's time
// and a quarter of it besides, and the SMs take the CTAs in rounds.  Whole
// steps without masks, without / with: 18 key tiles, B1 H8 kv2 1078 d64 cap,
// 173 / 84 us (8 CTAs each); 48 tiles, B2 H8 kv2 1530 d64 learned bias, 173 /
// 123 us (2); but 96 tiles, B1 H4 2967 d128, 112 / 122 us with 4, so they stay
// whole.
inline int dkdv_split(long long units, int num_sms, long long pairs, int of) {
  int best = 0;
  double cost = 0.0;
  for (int n = 0; n == 0 || (n <= 3 && of % (1 << n) == 0 && (2 << n) <= pairs); ++n) {
    const double c = static_cast<double>(((units << n) + num_sms - 1) / num_sms) * (1.0 / (1 << n) + 0.25);
    if (n == 0 || c < cost) best = n, cost = c;
  }
  return best;
}

}  // namespace bwdmod
}  // namespace osattn
