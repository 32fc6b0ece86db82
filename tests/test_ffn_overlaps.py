"""Outputs of the block norm that overlap its inputs or one another are refused on
the host (made-up addresses: no GPU is needed, and a call that passes the checks
has no rows' worth of work to do with them)."""
import ctypes

import pytest

ARG = 1
BASE = 0x100000


@pytest.fixture(scope="module")
def L():
    from dynamic_approximate_gemv_b200 import build
    build.build()
    import dynamic_approximate_gemv_b200 as E
    return E.lib()


def call(L, **kw):
    """rows 4, dim 64, binary16, each array a page of its own unless kw says otherwise."""
    from dynamic_approximate_gemv_b200.ffn import _NormArgs
    base = dict(rows=4, dim=64, dtype=1, weight_dtype=1, h_dtype=1, post_kind=0, pre_kind=1, eps=1e-5,
                weight_offset=0.0, residual_scale=1.0, branch_scale=1.0, x=BASE, x_stride=64, y=BASE + 0x1000,
                y_stride=64, x_out=BASE + 0x2000, x_out_stride=64, h_out=BASE + 0x3000, h_stride=64)
    base.update(kw)
    return L.effort_block_norm(ctypes.byref(_NormArgs(**base)), None)


ROW = 128  # bytes


@pytest.mark.parametrize("kw", [
    dict(x_out=BASE + 2), dict(x_out=BASE - 2), dict(x_out=BASE + ROW), dict(x_out=BASE + 3 * ROW + ROW - 2),
    dict(x_out=BASE, x_out_stride=65), dict(x_out=BASE + 0x1000 + ROW), dict(h_out=BASE + 2), dict(h_out=BASE, h_dtype=0),
    dict(h_out=BASE + 0x2000), dict(h_out=BASE + 0x2000 + 4), dict(h_out=BASE, x_out=BASE),
    dict(gate=BASE + 0x2000, gate_stride=64), dict(gate=BASE + 0x2000 + ROW, gate_stride=0),
    dict(gate=BASE + 0x3000, gate_stride=64), dict(pre_weight=BASE + 0x3000 + 2 * ROW),
    dict(pre_bias=BASE + 0x2000 - 2), dict(q_out=BASE, q_stride=64, q_scales=BASE + 0x5000, q_scales_stride=1),
    dict(q_out=BASE + 0x4000, q_stride=64, q_scales=BASE + 0x1000, q_scales_stride=1),
    dict(q_out=BASE + 0x4000, q_stride=64, q_scales=BASE + 0x4000 + 252, q_scales_stride=1),
    dict(q_out=BASE + 0x3000, q_stride=64, q_scales=BASE + 0x5000, q_scales_stride=1),
    # interleaved rows that reach one element into one another
    dict(x_stride=128, x_out=BASE + 2 * 63, x_out_stride=128),
    dict(x_stride=128, x_out=BASE + 2 * (128 + 65), x_out_stride=128),
    # rows of different strides that meet further down
    dict(x_stride=100, x_out=BASE + 2 * 64, x_out_stride=130),
])
def test_refused(L, kw):
    assert call(L, **kw) == ARG


@pytest.mark.parametrize("kw", [
    dict(), dict(x_out=BASE), dict(x_out=BASE + 0x1000), dict(h_out=BASE), dict(h_out=BASE + 0x1000, x_out=BASE),
    dict(x_out=BASE + 4 * ROW), dict(x_out=BASE - 4 * ROW), dict(y=BASE), dict(y=BASE, x_out=BASE),
    dict(x_stride=128, x_out=BASE + ROW, x_out_stride=128), dict(x_stride=128, x_out=BASE - ROW, x_out_stride=128),
    dict(x_stride=192, x_out=BASE + ROW, x_out_stride=192, h_out=BASE + 2 * ROW, h_stride=192),
    # rows 0 and 1 of x lie around rows of another stride that never meet them
    dict(rows=2, x_stride=1000, x_out=BASE + 2 * 64, x_out_stride=300),
    dict(rows=1, x_out=BASE, x_out_stride=9999), dict(rows=1, x_out=BASE + ROW),
])
def test_accepted(L, kw):
    """None of these is an argument error.  (They are checked without a device: with
    one they would run on made-up addresses.)"""
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses, for hosts without a device")
    assert call(L, **kw) != ARG


def test_against_sets_of_bytes(L):
    """x and x_out placed at random: refused exactly where they share a byte (and are not the same array)."""
    import random

    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses, for hosts without a device")
    rng = random.Random(5)
    refused = 0
    for _ in range(3000):
        rows, dim = rng.randint(1, 6), rng.randint(1, 12)
        sx = dim + rng.choice([0, 1, 5, dim, 2 * dim, 40])
        so = sx if rng.random() < 0.5 else dim + rng.randint(0, 50)
        at = 2 * rng.randint(-(rows + 1) * max(sx, so), (rows + 1) * max(sx, so))
        mine = {2 * (r * sx + i) for r in range(rows) for i in range(dim)}
        theirs = {at + 2 * (r * so + i) for r in range(rows) for i in range(dim)}
        same = at == 0 and (rows == 1 or sx == so)
        want = bool(mine & theirs) and not same
        got = call(L, rows=rows, dim=dim, x=BASE, x_stride=sx, x_out=BASE + at, x_out_stride=so, y=None, h_out=None)
        assert (got == ARG) == want, (rows, dim, sx, so, at)
        refused += want
    assert 500 < refused < 2500
