"""The blocks that the layer norm is launched with, at every width (host code, compiled and run on the CPU)."""

import shutil
import subprocess

import pytest

from collective_datapath_reduce_gb300 import _build

PROBE = r"""
#include <stdio.h>
#include "ops_norm.cuh"
using namespace pl;
template <typename T>
int check() {
  int bad = 0;
  for (uint64_t width = 1; width <= 20000; ++width)
    for (int aligned = 0; aligned <= (width % V16<T> == 0); ++aligned)
      for (int n = 1; n <= 3; ++n) {
        auto go = [&](auto lie, auto nv, int tpr) {
          constexpr Lie L = decltype(lie)::value;
          constexpr int NV = decltype(nv)::value, N = L == Lie::kSingle ? 1 : V16<T>;
          const Ring r = ring_of<T>(L, width, tpr, n);
          const int threads = tpr * r.groups;
          const bool warps = threads % 32 == 0 && threads <= kMostThreads && (tpr >= 32 ? tpr % 32 == 0 : 32 % tpr == 0);
          const bool fits = r.groups >= 1 && r.stages >= 2 && r.stages <= 5 && r.smem() <= kSmem && r.groups * 2 * width * 4 <= kSmem;
          const bool covers = (uint64_t)tpr * NV * N >= width && (L != Lie::kWhole || (uint64_t)tpr * NV * N == width) &&
                              r.granules * 16 >= width * sizeof(T) + (L == Lie::kSingle ? 16 - sizeof(T) : 0);
          // a group of several warps has a named barrier of its own beside the block's
          const bool barriers = tpr <= 32 || r.groups <= 15;
          if (!(warps && fits && covers && barriers)) {
            if (bad++ < 20) printf("%d-byte width %d aligned %d matrices %d: %d threads, %d a row, %u bytes\n", (int)sizeof(T), (int)width, aligned, n, threads, tpr, r.smem());
          }
          return PL_OK;
        };
        const bool held = width <= (aligned ? (sizeof(T) == 2 ? 12288 : 8192) : 8192);
        with_shape<T>(aligned, width, go, [&] {
          if (held && bad++ < 20) printf("width %d aligned %d: no shape\n", (int)width, aligned);
          return PL_OK;
        });
      }
  return bad;
}
int main() { return check<float>() + check<bf16>() ? 1 : 0; }
"""


def test_every_width_gets_whole_warps_that_cover_its_rows_and_a_ring_that_fits(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    source, program = tmp_path / "probe.cu", tmp_path / "probe"
    source.write_text(PROBE)
    subprocess.run([_build.nvcc(), *_build.ARCH, *_build.CFLAGS, str(source), "-o", str(program)], check=True, capture_output=True)
    r = subprocess.run([str(program)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
