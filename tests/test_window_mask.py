"""The bits of the windowed kernels' masks, on the host: against the definition, and without a difference that leaves 32 bits."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "pagedattention_kv_cache_paged_gb300", "csrc")

SOURCE = r"""
#include "window_mask.h"
#include <cstdio>
#include <vector>

int main() {
  const int64_t top = 2147483647, longest = 2147483648LL - 4096;
  const std::vector<int64_t> bounds = {-1, 0, 1, 30, 31, 32, 63, 64, 95, 200, 4095, 1000000, longest - 1};
  const std::vector<int64_t> windows = {1, 2, 31, 32, 33, 100, 4096, 1000000, longest - 1, longest, top - 1, top};
  const std::vector<int64_t> sinks = {0, 1, 31, 32, 33, 64, 100, 1000000, top};
  long n = 0;
  for (int64_t b : bounds)
    for (int64_t w : windows)
      for (int64_t s : sinks)
        for (int64_t at : {int64_t(0), int64_t(32), int64_t(64), int64_t(96), b - 64, b - 31, b, b + 1, b + 64, b - w - 40,
                           b - w + 1, b - w + 20, s - 20, s, longest - 32, longest + 96}) {
          if (at < 0 || at > longest + 96) continue;
          const int k0 = (int)at, low = pa::window_low((int)b, (int)w);
          const uint32_t got = pa::window_seen32((int)b, low, (int)s, k0);
          for (int c = 0; c < 32; ++c, ++n) {
            const int64_t j = at + c;
            const bool want = j <= b && (j > b - w || j < s);
            if (want != (((got >> c) & 1u) != 0)) {
              std::printf("bound %lld window %lld sinks %lld key %lld\n", (long long)b, (long long)w, (long long)s, (long long)j);
              return 2;
            }
          }
        }
  std::printf("%ld\n", n);
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a C++ compiler")
def test_bits_of_a_mask(tmp_path):
    (tmp_path / "mask.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC,
                    str(tmp_path / "mask.cpp"), "-o", str(tmp_path / "mask")], check=True)
    r = subprocess.run([str(tmp_path / "mask")], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    assert int(r.stdout) > 100_000


def test_the_kernel_takes_its_mask_from_there():
    with open(os.path.join(CSRC, "window_umma.cu")) as f:
        source = f.read()
    assert "window_low(bound, a.window)" in source and "window_seen32(bound, low, a.sinks, k0)" in source
