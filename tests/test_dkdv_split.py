"""The rule for CTAs that share a key tile of the dK/dV kernel: what its comment
says of the shapes that were measured, and what any choice has to keep."""
import os
import re
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_forward_online_gb300", "csrc")
SMS = 152


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    d = tmp_path_factory.mktemp("split")
    (d / "main.cpp").write_text("""
#include <cstdio>
#include "dkdv_split.h"
int main() {
  long long units, pairs;
  int sms, of;
  while (std::scanf("%lld %d %lld %d", &units, &sms, &pairs, &of) == 4)
    std::printf("%d\\n", osattn::bwdmod::dkdv_split(units, sms, pairs, of));
}
""")
    subprocess.run(["g++", "-std=c++17", "-I", CSRC, "-o", str(d / "split"), str(d / "main.cpp")], check=True)

    def run(cases):
        text = "".join("%d %d %d %d\n" % c for c in cases)
        out = subprocess.run([str(d / "split")], input=text, capture_output=True, text=True, check=True).stdout
        return [1 << int(x) for x in out.split()]

    return run


def shape(B, H, Hkv, N, rel):
    tiles = -(-N // 128)
    return B * Hkv * tiles, SMS, tiles * (H // Hkv), H // Hkv if rel else 8


def test_shapes_of_the_comment(split):
    cases = [shape(1, 8, 2, 1078, False), shape(2, 8, 2, 1530, True), shape(1, 4, 4, 2967, False)]
    assert [c[0] for c in cases] == [18, 48, 96]
    assert split(cases) == [8, 2, 1]
    text = " ".join(re.sub(r"\n// ?", " ", open(os.path.join(CSRC, "dkdv_split.h")).read()).split())
    for words in ("18 key tiles, B1 H8 kv2 1078 d64 cap, 173 / 84 us (8 CTAs each)",
                  "48 tiles, B2 H8 kv2 1530 d64 learned bias, 173 / 123 us (2)", "96 tiles, B1 H4 2967 d128"):
        assert words in text, words


def test_every_choice(split):
    cases = [(u, SMS, p, of) for u in (1, 2, 18, 19, 20, 38, 76, 77, 152, 153, 1000) for p in (1, 2, 3, 4, 7, 16, 17, 400)
             for of in (1, 2, 3, 4, 6, 8, 12)]
    for (units, _, pairs, of), n in zip(cases, split(cases)):
        assert n in (1, 2, 4, 8) and of % n == 0
        assert n == 1 or 2 * n <= pairs  # a CTA has two pairs at least
