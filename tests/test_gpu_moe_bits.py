"""How many bits of x, of the hidden activations and of the sums the mixture of
experts keeps (the bound of moe_precision.py), above all beside outliers."""
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


DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def outlier_layer(E, kind, which, e=2, i=256, f=256):
    """Weights with an outlier among their columns (or rows) whose own part of the
    result is nothing: w1's column 5 and w3's column 9 a thousand times the
    others, behind rows of zeros in w2; or inputs 3 and 70 that no weight reads."""
    w = [0.02 * randn(20 + k, e, *d) for k, d in enumerate([(i, f), (i, f), (f, i)])]
    if "w1" in which:
        w[0][:, :, 5::64] *= 1000
        w[2][:, 5::64] = 0
    if "w3" in which:
        w[1][:, :, 9::64] *= 1000
        w[2][:, 9::64] = 0
    if "x" in which:
        for k in (3, 70):
            w[0][:, k] = 0
            w[1][:, k] = 0
    if kind == "e4m3":
        q, s = zip(*(R.quantise_weights(t) for t in w))
        return E.MoeLayer(*q, scales=s), [R.dequantise_weights(a, b) for a, b in zip(q, s)]
    w = [t.to(DT[kind]) for t in w]
    return E.MoeLayer(*w), [t.double() for t in w]


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("which", ["none", "w1", "w1 w3", "x"])
@pytest.mark.parametrize("tokens", [1, 6, 20])
def test_outliers_leave_the_others_their_bits(E, kind, dt, out, which, tokens):
    layer, w64 = outlier_layer(E, kind, which)
    x = randn(31, tokens, 256)
    if "x" in which:
        x[:, [3, 70]] = 2.0e4
    x = x.to(DT[dt])
    ids = torch.arange(2, device="cuda", dtype=torch.int32).repeat(tokens, 1)
    gates = torch.tensor([[0.75, 0.25]], device="cuda").repeat(tokens, 1)
    got = layer(x, ids=ids, gates=gates, out_dtype=DT[out])[0]
    ref, tol = MP.moe(x, *w64, ids, gates, got.dtype, kind)
    R.assert_close(got, ref, tol)


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
def test_small_values_of_a_block_of_x_keep_their_bits(E, kind):
    """fp32 inputs 2^-22 to 2^-26 below their block's largest, which w1 does not read and
    w3 alone reads: b is large and exact, a is all of the small ones."""
    i, f = 256, 64
    w1, w3, w2 = 0.02 * randn(40, 1, i, f), torch.zeros(1, i, f, device="cuda"), 0.02 * randn(41, 1, f, i)
    w1[0, 3::64] = 0
    w3[0, 3] = 2.0 ** -10
    x = randn(32, 4, i) * 2.0 ** -10
    x[:, 3::64] = 2.0 ** 14
    w = [w1, w3, w2]
    if kind == "e4m3":
        q, s = zip(*(R.quantise_weights(t) for t in w))
        layer, w64 = E.MoeLayer(*q, scales=s), [R.dequantise_weights(a, b) for a, b in zip(q, s)]
    else:
        w = [t.to(DT[kind]) for t in w]
        layer, w64 = E.MoeLayer(*w), [t.double() for t in w]
    ids, gates = torch.zeros(4, 1, device="cuda", dtype=torch.int32), torch.ones(4, 1, device="cuda")
    got = layer(x, ids=ids, gates=gates)[0]
    ref, tol = MP.moe(x, *w64, ids, gates, got.dtype, kind)
    R.assert_close(got, ref, tol)


def test_long_sums_of_bf16_weights(E):
    """One large product and then many small ones in a warp's K blocks: a sum that
    truncates at each instruction would drop every small one."""
    i, f = 40960, 8
    w1 = torch.zeros(1, i, f, device="cuda")
    w1[0, :, 0] = 0.9 * 2.0 ** -27
    w1[0, :1024:64, 0] = 1 / 16  # the first K block of each of sixteen warps
    x = torch.ones(1, i, device="cuda")
    x[0, :1024:64] = 16.0
    w3 = torch.zeros(1, i, f, device="cuda")
    w3[0, 1, 0] = 1.0
    w2 = torch.zeros(1, f, i, device="cuda")
    w2[0, 0] = 1.0
    w = [t.bfloat16() for t in (w1, w3, w2)]
    layer = E.MoeLayer(*w)
    ids, gates = torch.zeros(1, 1, device="cuda", dtype=torch.int32), torch.ones(1, 1, device="cuda")
    got = layer(x, ids=ids, gates=gates)[0]
    a = (x.double() @ w[0][0].double())[0, 0]
    ref = a * torch.sigmoid(a)
    # a: four instructions of its K block (10 U each), 40 K blocks of a warp, 16 warps; silu and two roundings 12 U
    rel = float((got.double() - ref).abs().max() / ref)
    assert rel <= (4 * 10 + 40 + 16 + 12) * MP.U, rel / MP.U
