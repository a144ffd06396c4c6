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
Z_TILES = {"bf16": (256256, 128128, 64128), "f32": (128128, 32128)}



def ask(tmp_path, shapes):
    """The program's answers, a line per (tokens, d_model, vocabulary, type)."""
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    return subprocess.run([str(exe)], input="\n".join(f"{m} {d} {v} {t}" for m, d, v, t in shapes),
                          capture_output=True, text=True, check=True).stdout.splitlines()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_kernel_is_reached(dtype, tmp_path):
    one = [s for s in lp.STEPS if s[0] * s[2] < 1 << 27]  # (in one piece of the vocabulary)
    got = {k for line in ask(tmp_path, [(*s, dtype) for s in one]) for k in line.split()}
    want = {f"z-{t}" for t in Z_TILES[dtype]} | {f"dx-{t}" for t in TILES[dtype]} \
        | {f"dw-{t}" for t in TILES[dtype]}
    large = [t for t in TILES[dtype] if t >= 128000 or t == 32064]
    want |= {f"{p}-{t}-runs" for p in ("dx", "dw") for t in large}
    assert want <= got, sorted(want - got)


# us of a float32 forward and backward by the tile of z, as measured on an MI355X:
# (tokens, d_model, vocabulary): {tile: us}
MEASURED = {
    (999, 480, 10007): {128128: 456, 64128: 439, 32128: 403},
    (4096, 768, 32768): {128128: 6465, 64128: 7117, 32128: 6824},
    (500, 1024, 5000): {128128: 271, 64128: 275, 32128: 241},
    (2048, 256, 20000): {128128: 766, 64128: 869, 32128: 865},
    (64, 256, 500): {128128: 65, 64128: 49, 32128: 40},
    (246, 480, 832): {128128: 102, 64128: 69, 32128: 52},
    (128, 1024, 30000): {128128: 381, 64128: 366, 32128: 362},
    (1, 1000, 20000): {128128: 262, 64128: 189, 32128: 161},
    (1500, 128, 3000): {128128: 101, 64128: 101, 32128: 102},
    (300, 64, 50000): {128128: 152, 64128: 201, 32128: 173},
    (3000, 512, 5000): {128128: 576, 64128: 631, 32128: 627},
    (777, 1600, 2500): {128128: 381, 64128: 395, 32128: 275},
    (100, 2000, 700): {128128: 304, 64128: 174, 32128: 117},
    (9000, 96, 2000): {128128: 236, 64128: 259, 32128: 221},
    (16384, 64, 10000): {128128: 953, 64128: 1554, 32128: 1240},
    (2500, 800, 12000): {128128: 1790, 64128: 1957, 32128: 1865},
}


def test_planned_float32_tile_is_near_the_best_measured(tmp_path):
    """Each at most 8 % longer than the best, 1 % on average."""
    lines = ask(tmp_path, [(*s, "f32") for s in MEASURED])
    over = [t[int(line.split()[0][2:])] / min(t.values()) - 1
            for line, t in zip(lines, MEASURED.values())]
    assert max(over) <= 0.08 and sum(over) / len(over) <= 0.01, list(zip(MEASURED, over))
