"""The exact quotients that the prefix attention shares its work out with, on
the host: the same header, compiled as plain C++."""
import shutil
import subprocess

import pytest

from sparse_kv_verification_gb300 import build

SOURCE = r"""
#include <cstdint>
#include <cstdio>
#include "quotient.h"
using namespace dustin;
static uint64_t s = 88172645463325252ull;
static uint32_t rnd() { s ^= s << 13; s ^= s >> 7; s ^= s << 17; return (uint32_t)(s >> 20); }
static long bad, bad_wide, tried;
static void one(long long x, long long d) {
  if (x < 0 || x >= 1 << 30 || d < 1 || d > 0x7fffffff) return;
  ++tried;
  if (x / d < 1 << 22 && quotient((int)x, (int)d) != x / d) ++bad;
  if (quotient_wide((int)x, (int)d) != x / d) ++bad_wide;
}
int main() {
  for (int i = 0; i < 4000000; ++i) {
    const int d = 1 + (int)(rnd() >> (1 + rnd() % 31));
    const int x = (int)(rnd() >> (2 + rnd() % 30));
    one(x, d);
    // At and beside multiples, where an estimate errs.
    const long long m = (long long)(x / d) * d;
    for (int e = -1; e <= 1; ++e) one(m + e, d);
  }
  for (int d = 1; d <= 200; ++d)          // whole lines over few CTAs
    for (long long x = (1 << 30) - 1000; x < 1 << 30; ++x) one(x, d);
  std::printf("%ld %ld %ld\n", tried, bad, bad_wide);
}
"""


def test_quotients_are_exact(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    src = tmp_path / "quotient.cpp"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-O2", "-std=c++17", "-I" + build.CSRC, str(src), "-o", str(tmp_path / "q")],
                   check=True)
    tried, bad, bad_wide = map(int, subprocess.run([str(tmp_path / "q")], check=True,
                                                   capture_output=True, text=True).stdout.split())
    assert tried > 10 ** 7 and bad == 0 and bad_wide == 0
