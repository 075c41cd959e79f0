"""Division by a number that the host knows, on which the attention's indexes rest, against exact
division: its constants as the header makes them, its product as the kernels take it."""
import os
import subprocess

from hybrid_gated_deltanet_delta_gb300 import build as gdn_build

SOURCE = r"""
#include <stdio.h>
#include "gdn_kv4_attn.h"

static uint32_t quotient(gdn::kv4::Divisor d, uint32_t n) {
  const uint32_t high = (uint32_t)((uint64_t)d.m * n >> 32);
  return (high + n) >> d.s;  // 32 bits: must not wrap
}

static long bad = 0, seen = 0;

static void check(uint32_t d, uint64_t n) {
  if (n >= (1ull << 31)) return;
  ++seen;
  if (quotient(gdn::kv4::Divisor(d), (uint32_t)n) != n / d) ++bad;
}

int main() {
  const uint64_t top = (1ull << 31) - 1;
  uint64_t x = 88172645463325252ull;
  auto next = [&] { x ^= x << 13; x ^= x >> 7; x ^= x << 17; return x; };
  auto with = [&](uint32_t d) {
    for (uint64_t n = 0; n < 4; ++n) check(d, n), check(d, top - n);
    const uint64_t q = top / d;  // around multiples: the first ones, the last ones, others
    for (uint64_t k = 0; k < 48; ++k) {
      const uint64_t at = (k < 8 ? k : k < 16 ? q - (k - 8) : next() % (q + 1)) * d;
      for (int o = -1; o <= 1; ++o)
        if (at + o <= top) check(d, at + o);
      check(d, next() % (top + 1));
    }
  };
  for (uint32_t d = 1; d <= 5000; ++d) with(d);
  for (int s = 1; s < 31; ++s)
    for (int o = -2; o <= 2; ++o)
      if ((int64_t)(1ll << s) + o > 0) with((1u << s) + o);
  for (int o = 0; o < 3; ++o) with((uint32_t)top - o);
  for (int i = 0; i < 5000; ++i) with(1 + next() % top);
  for (uint64_t n = 0; n <= 1 << 20; ++n) check(7, n), check(24, n), check(96, n), check(1664, n);
  printf("%ld %ld\n", bad, seen);
}
"""


def test_divisor_is_exact(tmp_path):
    src, exe = tmp_path / "divisor.cpp", tmp_path / "divisor"
    src.write_text(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(gdn_build._nvcc()))), "include")
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-I", gdn_build.INCLUDE, "-I", gdn_build.CSRC,
                           "-I", cuda, str(src), "-o", str(exe)])
    bad, seen = map(int, subprocess.check_output([str(exe)]).split())
    assert bad == 0 and seen > 2_000_000
