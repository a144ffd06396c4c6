"""Which kernels a training step of the cross entropy takes (``csrc/dense_plan.hpp``,
compiled here for the host): the shapes of the precision tests must reach all of
them, whatever the tile costs are tuned to."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

import loss_precision as lp

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "selective_ssm_parameter_amd", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <string.h>
#include "dense_plan.hpp"
using namespace swimba;
int main() {
  int M, D, V;
  char ty[8];
  while (scanf("%d %d %d %7s", &M, &D, &V, ty) == 4) {
    const bool bf = !strcmp(ty, "bf16");
    auto say = [&](const char* n, const Runs& r) {
      printf("%s-%d%s ", n, r.tile, r.splits > 1 ? "-runs" : "");
    };
    printf("z-%d ", xent_tile(bf, M, V, D));
    say("dx", runs_of(bf, bf ? 2 : 0, false, M, D, (V + 7) / 8 * 8));
    say("dw", runs_of(bf, bf ? 2 : 0, true, V, D, M));
    printf("\n");
  }
}
"""
TILES = {"bf16": (256256, 256192, 128128, 64064, 32064), "f32": (128128, 64064, 32064)}
Z_TILES = {"bf16": (256256, 128128, 64128), "f32": (128128, 64128, 32128)}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_kernel_is_reached(dtype, tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    one = [s for s in lp.STEPS if s[0] * s[2] < 1 << 27]  # (in one piece of the vocabulary)
    got = set(subprocess.run([str(exe)], input="\n".join(f"{m} {d} {v} {dtype}" for m, d, v in one),
                             capture_output=True, text=True, check=True).stdout.split())
    want = {f"z-{t}" for t in Z_TILES[dtype]} | {f"dx-{t}" for t in TILES[dtype]} \
        | {f"dw-{t}" for t in TILES[dtype]}
    large = [t for t in TILES[dtype] if t >= 128000 or t == 32064]
    want |= {f"{p}-{t}-runs" for p in ("dx", "dw") for t in large}
    assert want <= got, sorted(want - got)
