"""Host-side contract of the layer calls (``include/swimba_layers.h``): every
declared symbol is exported and bound, and bad arguments are refused before
any device work (the pointers passed are never dereferenced)."""
from __future__ import annotations

import ctypes
import os
import re

import pytest
import torch

from selective_ssm_parameter_amd import binding as sb
from selective_ssm_parameter_amd import layers as sl

HEADER = os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "swimba_layers.h")
FAKE, MISALIGNED = 0x1000, 0x1004
BIG = 1 << 50


def lib():
    if not os.path.exists(sb.LIB_PATH):
        pytest.skip("libswimba.so not built")
    return sl.lib()


def dims(batch=2, seqlen=100, d=128, f=192, dtype="bf16"):
    return sl.layer_dims(batch, seqlen, d, f, dtype)


def err():
    return sb.lib().swimba_last_error().decode()


def ref(d):
    return ctypes.byref(d) if d is not None else None


def norm(d, x=FAKE, res=None, w=FAKE, b=FAKE, eps=1e-5, s=None, y=FAKE, mean=None, rstd=None):
    return lib().swimba_layer_norm(ref(d), x, res, w, b, eps, s, y, mean, rstd, None)


def norm_b(d, s=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, dy=FAKE, dyt=1, dres=None, dx=FAKE, dw=FAKE,
           db=FAKE, ws=FAKE, nb=BIG):
    return lib().swimba_layer_norm_backward(ref(d), s, w, mean, rstd, dy, dyt, dres, dx, dw, db,
                                            ws, nb, None)


def scan(d, x=FAKE, f=FAKE, o=FAKE, ld=192, lens=None, h0=None, y=FAKE, h=None, carry=None,
         ws=FAKE, nb=BIG):
    return lib().swimba_gated_scan(ref(d), x, f, o, ld, lens, h0, y, h, carry, ws, nb, None)


def scan_b(d, x=FAKE, f=FAKE, o=FAKE, ld=192, lens=None, carry=FAKE, dy=FAKE, dh=None, dx=FAKE,
           df=FAKE, do=FAKE, ldd=192, dh0=None, ws=FAKE, nb=BIG):
    return lib().swimba_gated_scan_backward(ref(d), x, f, o, ld, lens, carry, dy, dh, dx, df, do,
                                            ldd, dh0, ws, nb, None)


def step(d, x=FAKE, f=FAKE, o=None, ld=192, hp=FAKE, h=FAKE, y=FAKE):
    return lib().swimba_gated_step(ref(d), x, f, o, ld, hp, h, y, None)


def proj(d, x=FAKE, w=FAKE, act=0, z=None, h=FAKE):
    return lib().swimba_gated_project(ref(d), x, w, act, z, h, None)


def proj_b(d, x=FAKE, w=FAKE, dh=FAKE, act=0, dx=FAKE, dw=FAKE, ws=FAKE, nb=BIG):
    return lib().swimba_gated_project_backward(ref(d), x, w, dh, act, dx, dw, ws, nb, None)


def out_b(d, y=FAKE, w=FAKE, do=FAKE, dy=FAKE, dw=FAKE, ws=FAKE, nb=BIG):
    return lib().swimba_output_project_backward(ref(d), y, w, do, dy, dw, ws, nb, None)


ALL = [norm, norm_b, scan, scan_b, proj, proj_b, out_b]


def test_exports_every_declared_symbol():
    L = lib()
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    syms = set(re.findall(r"\b(swimba_[a-z_]+)\s*\(", text))
    assert syms == set(sl.EXPORTS)
    for s in syms:
        assert hasattr(L, s)
    # the two headers declare different symbols
    assert not syms & set(sb.EXPORTS)


@pytest.mark.parametrize("call", ALL + [step])
def test_dims_are_checked(call):
    lib()
    assert call(None) == -1 and "dims is NULL" in err()
    assert call(dims(batch=-1)) == -2
    bad = dims()
    bad.dtype = 7
    assert call(bad) == -2
    bad = dims()
    bad.reserved = 1
    assert call(bad) == -2
    assert call(dims(d=(1 << 20) + 8, f=8, seqlen=1)) == -2


def test_norm_refusals():
    lib()
    d = dims()
    for kw in ("x", "w", "y"):
        assert norm(d, **{kw: None}) == -1
    assert norm(d, res=FAKE) == -1 and "sum is NULL" in err()
    for kw in ("x", "res", "w", "b", "y", "mean", "rstd"):
        assert norm(d, **{kw: MISALIGNED}) == -5, kw
    for eps in (-1e-6, float("nan"), float("inf")):
        assert norm(d, eps=eps) == -2
    assert norm(dims(d=32769)) == -3
    assert norm(dims(batch=1 << 13, seqlen=1 << 13, d=512)) == -2  # 2^26 rows of a wave each
    assert norm(dims(seqlen=0), x=None, w=None, y=None) == 0
    need = sl.layer_workspace_size(d, sl.LAYER_NORM_BACKWARD)
    assert need > 0
    for kw in ("s", "w", "mean", "rstd", "dy", "dx", "dw"):
        assert norm_b(d, **{kw: None}) == -1, kw
    for kw in ("s", "w", "mean", "rstd", "dy", "dres", "dx", "dw", "db", "ws"):
        assert norm_b(d, **{kw: MISALIGNED}) == -5, kw
    assert norm_b(d, dyt=2) == -3 and norm_b(dims(dtype="f32"), dyt=1) == -3
    assert norm_b(d, nb=need - 1) == -4 and norm_b(d, ws=None, nb=0) == -4
    assert norm_b(dims(seqlen=0), dw=None) == -1


def test_scan_refusals():
    lib()
    d = dims(seqlen=300)
    need = sl.layer_workspace_size(d, sl.LAYER_GATED_SCAN)
    assert need > 0 and sl.lib().swimba_gated_scan_carry_size(ref(d)) == 2 * 3 * 192 * 4
    # a sequence of one chunk needs no workspace
    assert sl.layer_workspace_size(dims(seqlen=128), sl.LAYER_GATED_SCAN) == 0
    for kw in ("x", "f", "y"):
        assert scan(d, **{kw: None}) == -1, kw
    for kw in ("x", "f", "o", "lens", "h0", "y", "h", "carry", "ws"):
        assert scan(d, **{kw: MISALIGNED}) == -5, kw
    assert scan(d, ld=191) == -2 and scan(d, ld=-1) == -2 and scan(d, ld=1 << 22) == -2
    assert scan(d, nb=need - 1) == -4 and scan(d, ws=None, nb=0) == -4
    assert scan(dims(batch=0), x=None, f=None, y=None) == 0
    assert scan(dims(batch=1 << 24, seqlen=1), ld=192) == -2  # more workgroups than a launch has
    assert scan(dims(batch=1 << 30, seqlen=0), h=FAKE) == -2
    need = sl.layer_workspace_size(d, sl.LAYER_GATED_SCAN_BACKWARD)
    for kw in ("x", "f", "carry", "dy", "dx", "df", "do"):
        assert scan_b(d, **{kw: None}) == -1, kw
    for kw in ("x", "f", "o", "lens", "carry", "dy", "dh", "dx", "df", "dh0", "ws", "do"):
        assert scan_b(d, **{kw: MISALIGNED}) == -5, kw
    assert scan_b(d, ld=100) == -2 and scan_b(d, ldd=100) == -2
    assert scan_b(d, nb=need - 1) == -4
    assert step(dims()) == -2 and "seqlen must be 1" in err()
    d1 = dims(seqlen=1)
    for kw in ("x", "f", "hp", "h", "y"):
        assert step(d1, **{kw: None}) == -1, kw
    for kw in ("x", "f", "o", "hp", "h", "y"):
        assert step(d1, **{kw: MISALIGNED}) == -5, kw
    assert step(d1, ld=8) == -2 and step(d1, ld=1 << 22) == -2
    assert step(dims(batch=0, seqlen=1), x=None) == 0


def test_projection_refusals():
    lib()
    d = dims()
    for kw in ("x", "w", "h"):
        assert proj(d, **{kw: None}) == -1, kw
    for kw in ("x", "w", "z", "h"):
        assert proj(d, **{kw: MISALIGNED}) == -5, kw
    assert proj(d, act=2) == -2 and proj(d, act=-1) == -2
    for call in (proj, proj_b, out_b):
        assert call(dims(d=100)) == -3 and call(dims(f=100)) == -3
        assert call(dims(d=4)) == -3
    # w_in of 2 x 2^16 rows of 2^13 bf16 values: 2 GiB
    big = dims(d=1 << 13, f=1 << 16)
    assert proj(big) == -2 and "2 GiB" in err()
    assert proj_b(big) == -2
    assert out_b(dims(d=1 << 15, f=1 << 15)) == -2
    assert proj(dims(seqlen=0), x=None, w=None, h=None) == 0
    need = sl.layer_workspace_size(d, sl.LAYER_GATED_PROJECT_BACKWARD)
    assert need >= 200 * 2 * 192 * 2
    for kw in ("x", "w", "dh", "dx", "dw"):
        assert proj_b(d, **{kw: None}) == -1, kw
    for kw in ("x", "w", "dh", "dx", "dw", "ws"):
        assert proj_b(d, **{kw: MISALIGNED}) == -5, kw
    assert proj_b(d, nb=need - 1) == -4 and proj_b(d, act=9) == -2
    for kw in ("y", "w", "do", "dy", "dw"):
        assert out_b(d, **{kw: None}) == -1, kw
        assert out_b(d, **{kw: MISALIGNED}) == -5, kw
    long = dims(batch=8, seqlen=2048)
    need = sl.layer_workspace_size(long, sl.LAYER_OUTPUT_PROJECT_BACKWARD)
    assert need > 0 and out_b(long, nb=need - 1) == -4


def test_workspace_of_invalid_dims():
    lib()
    bad = dims(batch=-1)
    assert all(sl.layer_workspace_size(bad, c) == 0 for c in range(5))
    assert all(sl.layer_workspace_size(dims(seqlen=0), c) == 0 for c in range(5))
    assert sl.layer_workspace_size(dims(), 99) == 0
    assert sl.lib().swimba_gated_scan_carry_size(ref(bad)) == 0


def test_size_queries_keep_the_last_error():
    lib()
    assert norm(None) == -1 and "dims is NULL" in err()
    for bad in (dims(batch=-1), dims(d=(1 << 20) + 8, f=8, seqlen=1)):
        assert sl.layer_workspace_size(bad, sl.LAYER_NORM_BACKWARD) == 0
        assert sl.lib().swimba_gated_scan_carry_size(ref(bad)) == 0
        assert "dims is NULL" in err()


def test_binding_checks_row_strides():
    lib()
    wide = torch.zeros(4, 30)
    (a, b, c), ld = sl._rows(-1, wide[:, :8], wide[:, 8:16], None)
    assert ld == 30 and b - a == 32 and c is None
    with pytest.raises(ValueError, match="one row stride"):
        sl._rows(-1, wide[:, :8], torch.zeros(4, 8))
    with pytest.raises(ValueError, match="unit stride"):
        sl._rows(-1, torch.zeros(8, 4).t())
    with pytest.raises(ValueError, match="contiguous"):
        sl._ptrs(-1, wide[:, :8])
    with pytest.raises(ValueError, match="current device"):
        sl._ptrs(0, wide)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        sl.swimba_layer_norm_backward(dims(), None, None, None, None,
                                      torch.zeros(2, dtype=torch.float16), None, None, None, None,
                                      None)
