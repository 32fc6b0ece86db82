"""The feed-forward operators at the limits of their sizes: arrays whose offsets
pass 32 bits, the longest and widest matrices, the most pairs."""
import pytest
import torch

import ffn_reference as R
import test_gpu_block_norm as N
import test_gpu_fp8 as P
import test_gpu_moe as M

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dynamic_approximate_gemv_b200 import build
    build.build()
    import dynamic_approximate_gemv_b200 as E
    return E


@pytest.mark.parametrize("quantize", [False, True])
@pytest.mark.parametrize("dim", [4096, 4099])
def test_norm_past_32_bits(E, dim, quantize):
    """4.5 G elements: rows on both sides of 2^31 and 2^32 and the last ones are those of a call on them alone."""
    rows = 1_100_003
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(rows, dim, device="cuda", dtype=torch.bfloat16)
    for r in range(0, rows, 100_000):
        x[r:r + 100_000] = torch.randn(min(100_000, rows - r), dim, device="cuda", generator=g)
    got = E.block_norm(x, pre="layer", quantize=quantize)
    for at in (0, 2 ** 31 // dim - 1, 2 ** 32 // dim - 1, rows - 3):
        part = x[at:at + 3]
        _, (h, dh) = R.block_norm(part, None, None, "layer", None, 1.0, 1.0, None, None, None, None, 0.0, 1e-5)
        if quantize:
            R.check_quantised(got.q[at:at + 3], got.scales[at:at + 3], h, dh)
        else:
            R.assert_close(got.h[at:at + 3], h, dh)


def test_product_past_32_bits(E):
    rows, i, o = 70_001, 128, 65_536
    wq, ws, q, s = P.operands(rows, i, o)
    out = E.Fp8Matrix(wq, ws).matmul(q, s)
    for at in (0, 2 ** 31 // o - 1, 2 ** 32 // o - 1, rows - 2):
        ref, tol = R.product(q[at:at + 2], s[at:at + 2], wq, ws)
        R.assert_close(out[at:at + 2], ref, tol)


@pytest.mark.parametrize("rows,i,o", [(1, 262144, 100), (9, 262144, 100), (20, 262144, 100), (200, 262144, 130), (1, 60, 262144),
                                      (16, 60, 262144), (40, 60, 262144), (130, 60, 262144)])
def test_product_longest_and_widest(E, rows, i, o):
    P.check(E, rows, i, o, "f32")


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
@pytest.mark.parametrize("i,f", [(40960, 72), (72, 40960)])
def test_mixture_longest(E, kind, i, f):
    c = M.Case(E, 2, i, f, kind)
    x = M.randn(3, 5, i)
    ids = torch.tensor([[0, 1]] * 5, device="cuda", dtype=torch.int32)
    gates = torch.rand(5, 2, device="cuda", generator=M.gen(4))
    c.check(x, ids, gates, c.layer(x, ids=ids, gates=gates)[0])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_mixture_most_pairs(E, kind):
    M.Case(E, 256, 64, 48, kind).run(256, 16, "bf16")
