"""The block norm against its definition in 64 bits."""
import pytest
import torch

import ffn_reference as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dynamic_approximate_gemv_b200 import build
    build.build()
    import dynamic_approximate_gemv_b200 as E
    return E


def draw(rows, dim, dt, seed=0, scale=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(rows, dim, generator=g, device="cuda")).to(dt)


def check(E, rows, dim, dt, post, pre, gate, weights=True, bias=False, off=0.0, a=0.75, b=1.25, eps=1e-5,
          out_dtype=None, quantize=False, with_y=True, wdt=None, seed=0):
    dt = DT[dt]
    wdt = dt if wdt is None else DT[wdt]
    x = draw(rows, dim, dt, seed)
    y = draw(rows, dim, dt, seed + 1) + 0.25 if with_y else None
    g = {None: None, "one": draw(1, dim, dt, seed + 2, 1.0), "row": draw(rows, dim, dt, seed + 2, 1.0)}[gate]
    vec = lambda k: (1 + 0.2 * torch.randn(dim, device="cuda", generator=torch.Generator("cuda").manual_seed(k))).to(wdt)  # noqa: E731
    pw, w = (vec(5) if weights and post else None), (vec(6) if weights and pre else None)
    pb, bb = (vec(7) if bias and post else None), (vec(8) if bias and pre else None)
    r = E.block_norm(x, y, post=post, post_weight=pw, post_bias=pb, gate=g, residual_scale=a, branch_scale=b, pre=pre,
                     pre_weight=w, pre_bias=bb, eps=eps, weight_offset=off, out_dtype=out_dtype and DT[out_dtype],
                     quantize=quantize)
    (v, dv), (h, dh) = R.block_norm(x, y, post, pre, g, a, b, pw, pb, w, bb, off, eps)
    R.assert_close(r.x, v, dv, "x")
    if quantize:
        R.check_quantised(r.q, r.scales, h, dh)
    else:
        R.assert_close(r.h, h, dh, "h")
    return r


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [1, 2, 7, 64, 127, 128, 129, 1000, 4096, 5003, 14336])
def test_widths(E, dim, dt):
    check(E, 3, dim, dt, "rms", "rms", "row")
    check(E, 3, dim, dt, "rms", "rms", None, quantize=True)


@pytest.mark.parametrize("dim", [16384, 16392, 20001, 32768, 40960])
def test_widest(E, dim):
    check(E, 2, dim, "bf16", "layer", "layer", "one", bias=True)
    check(E, 2, dim, "f32", "rms", "rms", "row", quantize=True)


@pytest.mark.parametrize("post", [None, "rms", "layer"])
@pytest.mark.parametrize("pre", [None, "rms", "layer"])
@pytest.mark.parametrize("gate", [None, "one", "row"])
def test_forms(E, post, pre, gate):
    check(E, 5, 520, "bf16", post, pre, gate, bias=True, off=1.0)
    check(E, 5, 520, "f16", post, pre, gate, quantize=True, wdt="f32")
    check(E, 5, 521, "f32", post, pre, gate, weights=False, out_dtype="f16")


@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_out_types(E, dt, out):
    check(E, 4, 264, dt, "rms", "rms", "one", out_dtype=out, wdt=out)


def test_without_a_branch(E):
    check(E, 4, 100, "bf16", None, "rms", None, with_y=False, a=0.5)
    x = draw(4, 100, torch.float16)
    r = E.block_norm(x)
    assert r.x is x  # nothing was added or scaled
    _, (h, dh) = R.block_norm(x, None, None, "rms", None, 1.0, 1.0, None, None, None, None, 0.0, 1e-5)
    R.assert_close(r.h, h, dh)


@pytest.mark.parametrize("rows", [0, 1, 2, 149, 1500, 4099])
def test_rows(E, rows):
    if rows:
        check(E, rows, 136, "bf16", "rms", "rms", "row", quantize=True)
        check(E, rows, 136, "f16", "rms", "layer", "row")
    else:
        r = E.block_norm(torch.empty(0, 136, device="cuda"), quantize=True)
        assert r.q.shape == (0, 136) and r.scales.shape == (0, 2)


def test_one_dimension(E):
    x, y = draw(1, 4096, torch.float32), draw(1, 4096, torch.float32, 1)
    r1 = E.block_norm(x[0], y[0], post="rms")
    r2 = E.block_norm(x, y, post="rms")
    assert r1.x.shape == (4096,) and torch.equal(r1.h, r2.h[0]) and torch.equal(r1.x, r2.x[0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strides_and_what_lies_between_rows(E, dt):
    dt = DT[dt]
    m, n = 9, 133
    wide = draw(m, 200, dt)
    x, y = wide[:, 3:3 + n], draw(m, 150, dt, 1)[:, 1:1 + n]
    xo, ho = torch.full((m, 160), 7.0, device="cuda", dtype=dt), torch.full((m + 2, 140), 7.0, device="cuda", dtype=dt)
    r = E.block_norm(x, y, post="layer", x_out=xo[:, 1:1 + n], h_out=ho[:m, :n])
    (v, dv), (h, dh) = R.block_norm(x, y, "layer", "rms", None, 1.0, 1.0, None, None, None, None, 0.0, 1e-5)
    R.assert_close(r.x, v, dv)
    R.assert_close(r.h, h, dh)
    assert bool((xo[:, 0] == 7).all() and (xo[:, 1 + n:] == 7).all())
    assert bool((ho[:m, n:] == 7).all() and (ho[m:] == 7).all())


def test_in_place(E):
    x, y = draw(33, 1024, torch.bfloat16), draw(33, 1024, torch.bfloat16, 1)
    ref = E.block_norm(x, y, post="rms")
    x2, y2 = x.clone(), y.clone()
    r = E.block_norm(x2, y2, post="rms", x_out=x2, h_out=y2)
    assert r.x is x2 and torch.equal(x2, ref.x) and torch.equal(y2, ref.h)


def test_zero_rows_and_constant_rows(E):
    x = torch.zeros(4, 300, device="cuda")
    x[2] = 5.0
    r = E.block_norm(x, pre="rms", quantize=True)
    assert bool((r.q.float()[0] == 0).all()) and bool((r.scales[0] == 0).all())
    h = E.block_norm(x, pre="layer").h
    assert bool((h.abs() < 1e-3).all())  # (5 - 5) / sqrt(eps) in every column, up to the mean's rounding
    h0 = E.block_norm(x[2:3], pre="rms", eps=0.0).h
    assert torch.allclose(h0, torch.ones_like(h0), rtol=8 * R.U32)


def test_tiny_blocks_quantise_to_zero(E):
    x = torch.full((1, 256), 1e-44, device="cuda")
    x[:, 128:] = 1.0
    q, s = E.quantize_e4m3(x)
    assert float(s[0, 0]) == 0.0 and bool((q.float()[:, :128] == 0).all())
    assert bool((q.float()[:, 128:] == 448).all())


def test_nonfinite_rows_stay_their_own(E):
    x = draw(8, 512, torch.float32)
    ref = E.block_norm(x, pre="rms", quantize=True)
    bad = x.clone()
    bad[2, 200] = float("nan")
    bad[5, 300] = float("inf")
    r = E.block_norm(bad, pre="rms", quantize=True)
    keep = [0, 1, 3, 4, 6, 7]
    assert torch.equal(r.q[keep].view(torch.uint8), ref.q[keep].view(torch.uint8))
    assert torch.equal(r.scales[keep], ref.scales[keep])
    assert not torch.isfinite(r.scales[2]).any()
    q, s = E.quantize_e4m3(bad)
    assert torch.isnan(s[2, 1]) and torch.isinf(s[5, 2])
    assert torch.isfinite(s[2, 0]) and torch.isfinite(s[5, 3])


def test_huge_and_small_values(E):
    x = draw(2, 640, torch.float32) * 1e15
    _, (h, dh) = R.block_norm(x, None, None, "rms", None, 1.0, 1.0, None, None, None, None, 0.0, 1e-5)
    R.assert_close(E.block_norm(x).h, h, dh)
    x = draw(2, 640, torch.float32) * 1e-12
    _, (h, dh) = R.block_norm(x, None, None, "rms", None, 1.0, 1.0, None, None, None, None, 0.0, 1e-5)
    R.assert_close(E.block_norm(x).h, h, dh + 2.0 ** -100)


def test_quantise_alone_matches_torch_rounding(E):
    x = draw(37, 1000, torch.bfloat16, 4)
    q, s = E.quantize_e4m3(x)
    assert q.stride(0) % 16 == 0
    R.check_quantised(q, s, x.double(), torch.zeros(37, 1000, dtype=torch.float64, device="cuda"))
    # the scale is one division, the value another: bit for bit (by a tensor: torch
    # multiplies by the reciprocal where the divisor is a number)
    pad = torch.nn.functional.pad(x.float(), (0, 24)).reshape(37, 8, 128)
    assert torch.equal(s, pad.abs().amax(2) / torch.full_like(s, 448.0))
    t = (pad / s[..., None]).reshape(37, -1)[:, :1000].to(torch.float8_e4m3fn)
    assert torch.equal(q.contiguous().view(torch.uint8), t.view(torch.uint8))


def test_other_stream_and_graph(E):
    x, y = draw(64, 2048, torch.bfloat16), draw(64, 2048, torch.bfloat16, 1)
    ref = E.block_norm(x, y, post="rms", quantize=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        r = E.block_norm(x, y, post="rms", quantize=True)
    s.synchronize()
    assert torch.equal(r.x, ref.x) and torch.equal(r.scales, ref.scales)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = E.block_norm(x, y, post="rms", quantize=True)
    x.copy_(y)
    want = E.block_norm(x, y, post="rms", quantize=True)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(r.x, want.x) and torch.equal(r.q.view(torch.uint8), want.q.view(torch.uint8))


def test_binding_refuses(E):
    x = draw(4, 64, torch.float32)
    bad = [
        (ValueError, lambda: E.block_norm(x, post="rms")),
        (ValueError, lambda: E.block_norm(x, gate=x)),
        (ValueError, lambda: E.block_norm(x, x[:3])),
        (TypeError, lambda: E.block_norm(x, x.half())),
        (ValueError, lambda: E.block_norm(x, pre="batch")),
        (ValueError, lambda: E.block_norm(x.T)),
        (ValueError, lambda: E.block_norm(x, pre_weight=x[0, :63])),
        (ValueError, lambda: E.block_norm(x, pre=None, pre_weight=x[0])),
        (ValueError, lambda: E.block_norm(x, x, gate=x[:2])),
        (ValueError, lambda: E.block_norm(x, quantize=True, out_dtype=torch.float16)),
        (TypeError, lambda: E.block_norm(x, out_dtype=torch.float64)),
        (TypeError, lambda: E.block_norm(x.double())),
        (E.EffortError, lambda: E.block_norm(x, eps=-1.0)),
        (E.EffortError, lambda: E.block_norm(x[:1].expand(4, 64))),
        (E.EffortError, lambda: E.block_norm(torch.zeros(1, 40961, device="cuda"))),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()
