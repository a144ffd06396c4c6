"""How the convolution and the single-token scan divide their work
(``csrc/ssm_plan.hpp``, compiled here for the host): the shapes of the long-run tests
must reach what large workloads reach."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

import ssm_runs

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "selective_ssm_parameter_amd", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include "ssm_plan.hpp"
using namespace swimba;
int main() {
  int B, T, C, ld, bf;
  while (scanf("%d %d %d %d %d", &B, &T, &C, &ld, &bf) == 5) {
    const int f = vec_of(vec_fwd(bf), C, ld, 0), b = vec_of(vec_bwd(bf), C, ld, ld);
    printf("%d %d %d %d %d\n", f, run_length(B, T, C / f, kFwdThreads), b,
           run_length(B, T, C / b, kBwdThreads), step_sequences(B, C));
  }
}
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    """(batch, tokens, channels, row stride, bf16) -> vector and run forward, vector and run
    backward, sequences a thread of one token."""
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    src, exe = d / "plan.cpp", d / "plan"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-I", CSRC, "-o", str(exe), str(src)], check=True)

    def run(*args):
        out = subprocess.run([str(exe)], input=" ".join(map(str, args)), capture_output=True,
                             text=True, check=True).stdout
        return [int(v) for v in out.split()]

    return run


def stride(C, pad, dtype):
    per = 8 if dtype == "bf16" else 4
    return -(-(C + pad) // per) * per


def test_long_runs_in_both_directions(ask):
    forms = set()
    for B, T, C, dtype, _, _, _, _, pad in ssm_runs.CONV:
        vf, rf, vb, rb, _ = ask(B, T, C, stride(C, pad, dtype), int(dtype == "bf16"))
        assert rf >= 24 and rb >= 24 and T % rf and T % rb, (B, T, C, rf, rb)
        forms |= {("forward", dtype, vf), ("backward", dtype, vb)}
        forms |= {("longest", vb)} if rb == 256 else set()
    want = {(d, t, v) for t in ("bf16", "f32") for d, v in (("forward", 1), ("backward", 1))}
    want |= {("forward", "bf16", 8), ("backward", "bf16", 4), ("forward", "f32", 4),
             ("backward", "f32", 2), ("longest", 4)}
    assert want <= forms, want - forms


def test_two_sequences_a_thread(ask):
    for B, C, _, _, _ in ssm_runs.STEP:
        assert B % 2 == 1 and ask(B, 1, C, C, 1)[4] == 2, (B, C)
    assert ask(255, 1, 1024, 1024, 1)[4] == 1
