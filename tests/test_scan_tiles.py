"""Host check of the tile counts that the recurrence's kernels work out in 32 bits, at the
longest sequences that the entry points take.  No GPU."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "chunked_gated_delta_bwd_amd", "csrc", "layer", "gdr_layer.h")

PROGRAM = r"""
#include "%s"
#include <cstdio>
int main() {
  const long long top = (1LL << 31) - 1;
  const int tiles[] = {64, 128, 256};
  const long long nears[] = {0, 64, 128, 256, 512, 1LL << 24, 1LL << 30, top - 256, top - 128, top};
  for (int tile : tiles)
    for (long long near : nears)
      for (long long d = -3; d <= 3; ++d) {
        const long long len = near + d;
        if (len < 0 || len > top) continue;
        const long long want = len ? (len + tile - 1) / tile : 1, got = gdr::scan_tiles(int(len), tile);
        if (got != want) {
          printf("%%lld tokens, tiles of %%d: %%lld, expected %%lld\n", len, tile, got, want);
          return 1;
        }
      }
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_tiles_of_the_longest_sequences(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM % HEADER)
    # signed overflow wraps here as it does in the kernels, so that it shows in the count
    subprocess.run(["g++", "-std=c++17", "-O1", "-fwrapv", str(src), "-o", str(exe)], check=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout
