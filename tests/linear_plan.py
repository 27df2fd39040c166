"""The expert product's choice of a kernel, for the tests: its host code (csrc/linear_plan.h, plain C++) compiled
and asked on the CPU."""
import functools
import os
import shutil
import subprocess
import tempfile
from collections import namedtuple

import combine_grouped_gemm_amd as moe

CSRC = os.path.join(os.path.dirname(moe.library_path()), "csrc")
KINDS = ("few", "64", "128", "320", "32")
Plan = namedtuple("Plan", "kind split tile_rows fits groups threads")

_MAIN = r"""
#include <cstdio>
#include "linear_plan.h"
int main() {
  int rows, K, N, E, f32, gated;
  while (std::scanf("%d %d %d %d %d %d", &rows, &K, &N, &E, &f32, &gated) == 6) {
    const moe::LinPlan p = moe::lin_plan(rows, K, gated ? 2 * N : N, E, f32 != 0);
    long long groups = 0;
    moe::LinShape s{0, 0, 0};
    if (p.kind != moe::LIN_FEW) {
      s = moe::lin_shape(p.kind, f32 != 0, gated != 0);
      groups = moe::lin_tile_groups(rows, E, N, p.tile_rows > 0 ? p.tile_rows : s.rows, s.cols, p.split);
    }
    std::printf("%d %d %d %d %lld %d\n", p.kind, p.split, p.tile_rows,
                int(moe::lin_fits(rows, K, N, E, f32 != 0, gated != 0)), groups, s.threads);
  }
}
"""


@functools.lru_cache(maxsize=None)
def _program() -> str:
    folder = tempfile.mkdtemp(prefix="linear_plan_")
    source, binary = os.path.join(folder, "main.cpp"), os.path.join(folder, "main")
    with open(source, "w") as f:
        f.write(_MAIN)
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, source, "-o", binary],
                   check=True, capture_output=True, text=True)
    return binary


def plans(sizes) -> list:
    """A Plan for each (rows, K, N, E, f32, gated); few: a launch of the few-rows kernel (groups 0)."""
    text = "".join("%d %d %d %d %d %d\n" % tuple(int(v) for v in s) for s in sizes)
    out = subprocess.run([_program()], input=text, check=True, capture_output=True, text=True).stdout.split("\n")[:-1]
    rows = [[int(v) for v in line.split()] for line in out]
    assert len(rows) == len(sizes)
    return [Plan(KINDS[r[0]], r[1], r[2], bool(r[3]), r[4], r[5]) for r in rows]
