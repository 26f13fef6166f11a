"""The block reduction of the norm ring kernels, on the host: which shared-memory words its lanes read.

A sum of N values over W warps keeps a set of partials per value and warp.  When it adds them up, each of them has
to be read by one lane, and no lane may read anything else: what lies behind a set belongs to the next sum, which
faster warps may be writing, or to other data.
"""
import os
import subprocess

import pytest

from packed_mm_rope_b200 import build

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "norm.cuh"

template <int G, int N>
int check() {
  using S = h3::norm::BlockSum<G, N>;
  constexpr int SET = S::SIZE / 2;
  int reads[SET] = {}, wrong = 0;
  for (int g = 0; g < (N + S::PER - 1) / S::PER; ++g)
    for (int lane = 0; lane < 32; ++lane) {
      const int at = S::source(g, lane);
      if (at == -1) continue;
      if (at < 0 || at >= SET) ++wrong;
      else ++reads[at];
      // the lanes of value v are those whose sum its shuffles form and broadcast
      if (at / S::WP != g * S::PER + lane / S::WP || at % S::WP != lane % S::WP) ++wrong;
    }
  for (int i = 0; i < SET; ++i)
    if (reads[i] != (i / S::WP < N && i % S::WP < S::W ? 1 : 0)) ++wrong;
  std::printf("%d %d %d\n", G, N, wrong);
  return wrong;
}

int main() {
  int wrong = 0;
  wrong += check<256, 1>() + check<256, 2>() + check<256, 4>();      // forward: rows per step
  wrong += check<480, 1>() + check<480, 2>() + check<480, 4>();
  wrong += check<224, 2>() + check<224, 4>();                        // backward: two sums per row
  return wrong != 0;
}
"""


def test_block_sum_reads_its_own_partials_alone(tmp_path):
    try:
        nvcc = build.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    source = tmp_path / "sum.cu"
    source.write_text(PROGRAM)
    exe = str(tmp_path / "sum")
    r = subprocess.run([nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-I", build.CSRC, "-I",
                        os.path.join(build.ROOT, "include"), str(source), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and len(r.stdout.split()) == 24, r.stdout + r.stderr
