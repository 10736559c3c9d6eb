"""CPU-only checks of ep_matmul_split: when columns are split and over how many
blocks, what workspace that takes, and the refusals of its calls."""
import ctypes
import random

import pytest

import matmul_paths as P
from combine_get_dispatch_layout_amd import ep, moe
from test_matmul_abi import PTR, _w


def size(w, rows, act=0):
    out = ctypes.c_int64(-1)
    assert moe._lib().ep_matmul_workspace_size(ctypes.byref(w), rows, act, ctypes.byref(out)) == ep.EP_OK
    return out.value


def test_choice():
    """Few tiles and many steps of 128 columns, and nothing else."""
    assert P.splits(64, 7168, 4096) == 4 and P.splits(33, 16384, 4096) == 4
    assert P.splits(64, 7168, 256) == 7 and P.splits(1, 131056, 16) == 32
    for rows, cols, out in ((0, 7168, 4096), (1, 7168, 4096), (64, 2048, 2048), (256, 7168, 4096), (4096, 7168, 4096)):
        assert P.splits(rows, cols, out) == 1
    rng = random.Random(5)
    seen = set()
    for _ in range(5000):
        act = rng.randint(0, 1)
        rows, cols = int(2 ** rng.uniform(0, 14)), 16 * int(2 ** rng.uniform(0, 12.9))
        out = 2 * int(2 ** rng.uniform(0, 12))
        n = P.splits(rows, cols, out, act)
        steps, tiles = (cols + 127) // 128, (rows + 63) // 64 * ((out + 63) // 64)
        assert n == 1 or (2 <= n <= 32 and n * tiles <= 256 and steps >= 8 * n), (rows, cols, out, act, n)
        need = size(_w(rows=out, cols=cols), rows, act)
        assert need == (4 * n * rows * out if n > 1 else 0) and need <= 4 << 20
        seen.add(n)
    assert len(seen) > 8


@pytest.mark.parametrize("bad", [dict(format=moe.EP_WEIGHT_BF16), dict(num_experts=2), dict(cols=120), dict(group=32),
                                 dict(rows=0)])
def test_size_refusals(bad):
    out = ctypes.c_int64()
    f = moe._lib().ep_matmul_workspace_size
    assert f(ctypes.byref(_w(**bad)), 1, 0, ctypes.byref(out)) == ep.EP_ERR_INVALID_ARG
    w = _w()
    assert f(None, 1, 0, ctypes.byref(out)) == ep.EP_ERR_INVALID_ARG
    assert f(ctypes.byref(w), 1, 0, None) == ep.EP_ERR_INVALID_ARG
    assert f(ctypes.byref(w), -1, 0, ctypes.byref(out)) == ep.EP_ERR_INVALID_ARG
    assert f(ctypes.byref(w), 1, 2, ctypes.byref(out)) == ep.EP_ERR_INVALID_ARG
    assert f(ctypes.byref(_w(rows=33)), 1, 1, ctypes.byref(out)) == ep.EP_ERR_INVALID_ARG


def test_call_refusals():
    f = moe._lib().ep_matmul_split

    def call(w=_w(rows=256, cols=7168), x=PTR, xs=PTR, n=64, act=0, y=PTR, ws=PTR, have=1 << 30):
        return f(None if w is None else ctypes.byref(w), x, xs, n, act, y, ws, have, None)
    need = size(_w(rows=256, cols=7168), 64)
    assert need > 0
    for bad in (dict(w=None), dict(w=_w(num_experts=2)), dict(x=None), dict(x=PTR + 8), dict(xs=None), dict(xs=PTR + 2),
                dict(n=-1), dict(act=3), dict(y=None), dict(y=PTR + 1)):
        assert call(**bad) == ep.EP_ERR_INVALID_ARG
    for bad in (dict(ws=None), dict(ws=PTR + 128), dict(have=need - 1), dict(have=0), dict(have=-1)):
        assert call(**bad) == ep.EP_ERR_WORKSPACE
    assert call(x=None, xs=None, n=0, y=None, ws=None, have=0) == ep.EP_OK      # no rows
