"""Where the tile kernel of the MXFP4 products finds its weights: every lane's 16 bytes of every stage lie
in the wave's own rows, and hold the block that the stage means wherever there is one.  A host program
goes over the offsets (csrc/fp4_places.h) that the kernel computes; no GPU needed."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include "fp4_places.h"
using namespace mxfp4;

static int check(int N, int KB, int sub_tiles) {
  const int panel = 4 * sub_tiles * 32;
  for (int n0 = 0; n0 < N; n0 += panel)
    for (int wave = 0; wave < 4; wave++) {
      const int n = n0 + wave * sub_tiles * 32;
      const int first = fp4_wave_first(n, N), rows = fp4_wave_rows(n, N, sub_tiles * 32);
      if (first < 0 || rows < 1 || rows > sub_tiles * 32 || first + rows > N) return 1;
      if (n < N && first != n) return 2;
      for (int s = 0; s <= (KB - 1) / 8 + 2; s++)
        for (int t = 0; t < sub_tiles; t++)
          for (int i = 0; i < 4; i++)
            for (int lane = 0; lane < 64; lane++) {
              const int upper = i & 1, v = i >> 1, q = lane >> 4;
              const long long at = (long long)fp4_row_at(t, upper, lane, rows, KB) + fp4_block_at(s, v, lane, KB);
              if (at < 0 || at % 16 || at + 16 > (long long)rows * KB * 16) return 3;
              const int row = 32 * t + 16 * upper + lane % 16, block = 8 * s + 4 * v + q;
              if (row < rows && at / (KB * 16) != row) return 4;
              if (block < KB && at / 16 % KB != block) return 5;
              if (block >= KB && s <= (KB - 1) / 8 && at / 16 % KB != KB - 1) return 6;
            }
    }
  return 0;
}

int main() {
  const int widths[] = {1, 2, 5, 31, 32, 33, 63, 64, 65, 127, 130, 255, 256, 257, 300, 545, 5760};
  for (int sub_tiles = 1; sub_tiles <= 2; sub_tiles++)
    for (int N : widths)
      for (int KB = 1; KB <= 100; KB++) {
        if (N == 5760 && KB != 90) continue;
        const int bad = check(N, KB, sub_tiles);
        if (bad) {
          std::printf("N %d, K %d, %d sub-tiles: %d\n", N, 32 * KB, sub_tiles, bad);
          return 1;
        }
      }
  // the largest K: the offsets of 64 rows stay below 2^31
  const int KB = (1 << 21) - 1;
  const long long at = (long long)fp4_row_at(1, 1, 63, 64, KB) + fp4_block_at(1 << 20, 1, 63, KB);
  if (fp4_row_at(1, 1, 63, 64, KB) != 63LL * KB * 16 || at + 16 != 64LL * KB * 16) return 1;
  std::puts("ok");
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_every_lane_reads_its_own_rows(tmp_path):
    src, exe = tmp_path / "places.cpp", tmp_path / "places"
    src.write_text(PROGRAM)
    csrc = os.path.join(ROOT, "mxfp4_mixture_experts_amd", "csrc")
    built = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-fsanitize=undefined", "-fno-sanitize-recover=undefined",
                            "-I", csrc, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert built.returncode == 0, built.stderr
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.strip() == "ok", out.stdout + out.stderr
