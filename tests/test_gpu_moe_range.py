"""The mixture of experts where its inputs or scales lie far from 1: a result in
range is not lost on the way."""
import pytest
import torch

import ffn_reference as R
import moe_precision as MP

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dynamic_approximate_gemv_b200 import build
    build.build()
    import dynamic_approximate_gemv_b200 as E
    return E


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def check(E, x, std1, std3, std2, i=256, f=192, e=2, bits=False):
    """One call with e4m3 weights of these standard deviations, by their scales alone,
    within the bound of ffn_reference or (bits: of positive weights) the closer one of moe_precision."""
    draw = (lambda *a: randn(*a).abs()) if bits else randn
    w, s = zip(*(R.quantise_weights(0.02 * draw(k, e, *d)) for k, d in enumerate([(i, f), (i, f), (f, i)])))
    s = tuple(t * (std / 0.02) for t, std in zip(s, (std1, std3, std2)))
    layer = E.MoeLayer(*w, scales=s)
    w64 = [R.dequantise_weights(q, t) for q, t in zip(w, s)]
    ids = torch.arange(e, device="cuda", dtype=torch.int32).repeat(len(x), 1)
    gates = torch.full((len(x), e), 0.5, device="cuda")
    out = layer(x, ids=ids, gates=gates)[0]
    ref, tol = MP.moe(x, *w64, ids, gates, out.dtype, "e4m3") if bits else R.moe(x, *w64, ids, gates, out.dtype)
    assert float(ref.abs().max()) < 1e30
    R.assert_close(out, ref, tol)
    layer.close()


@pytest.mark.parametrize("mag", [1e-29, 1e-31, 1e-32, 1e-33, 1e-35])
def test_tiny_x_under_large_scales(E, mag):
    """The hidden activations' scale comes from the norm of x, however small x is."""
    check(E, mag * randn(9, 3, 256), 1e-12 / mag, 1e-12 / mag, 1e10)


@pytest.mark.parametrize("std1,std3,std2", [(1e-24, 1e14, 1e9), (1e14, 1e-24, 1e9), (1e20, 1e-10, 1e-10),
                                            (1e-10, 1e20, 1e-10), (1e-25, 1e25, 1.0), (1e25, 1e-25, 1.0)])
def test_opposite_scales(E, std1, std3, std2):
    """One of w1 and w3 with squares below or above fp32's range, the result within it."""
    check(E, randn(9, 3, 256), std1, std3, std2)


@pytest.mark.parametrize("mag", [1e30, 1e36])
def test_large_x_under_small_scales(E, mag):
    check(E, mag * randn(9, 3, 256), 0.05 / mag, 0.05 / mag, 0.05)


@pytest.mark.parametrize("mag,std1,std3,std2", [(1e-18, 0.02, 0.02, 1e-3), (1e-19, 0.2, 0.2, 1e-3), (1e-31, 1e-7, 1e30, 1e30),
                                                (1e-31, 1e30, 1e-7, 1e30)])
def test_tiny_products_keep_their_bits(E, mag, std1, std3, std2):
    """Hidden activations near the bottom of fp32's range, or a or b there: no factor
    on the way becomes a subnormal number that has lost bits.  (All positive, so that
    nothing cancels and the bound is relative to the result.)"""
    check(E, mag * randn(9, 3, 256).abs(), std1, std3, std2, bits=True)
