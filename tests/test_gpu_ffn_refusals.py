"""Calls of the feed-forward operators that are refused rather than answered
wrongly, and forms of arguments the other tests leave out."""
import ctypes

import pytest
import torch

import ffn_reference as R

pytestmark = pytest.mark.gpu
ARG = 1


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


@pytest.fixture(scope="module")
def matrix(E):
    return E.Fp8Matrix(*R.quantise_weights(0.05 * randn(1, 256, 128)))


@pytest.fixture(scope="module")
def layer(E):
    return E.MoeLayer(*(0.05 * randn(k, 4, *s).half() for k, s in enumerate([(64, 32), (64, 32), (32, 64)])),
                      router=randn(9, 4, 64))


# -- outputs over inputs

def test_product_out_over_its_inputs_is_refused(E, matrix):
    q, s = E.quantize_e4m3(randn(2, 300, 256))
    over = q.view(torch.float32)  # [300, 64]
    wide = torch.empty(300, 128, device="cuda")
    for bad in (torch.as_strided(over, (150, 128), (128, 1)), torch.as_strided(s, (4, 128), (128, 1))):
        with pytest.raises(E.EffortError) as e:
            matrix.matmul(q[:len(bad)], s[:len(bad)], out=bad)
        assert e.value.status == ARG
    matrix.matmul(q, s, out=wide)


def test_mixture_over_its_own_arguments_is_refused(E, layer):
    x = randn(0, 8, 64)
    buf = torch.zeros(8 * 64 + 64, device="cuda")
    ids = buf[:16].view(torch.int32).view(8, 2)
    gates = buf[16:32].view(8, 2)
    out = buf[24:24 + 512].view(8, 64)
    with pytest.raises(E.EffortError) as e:
        layer(x, ids=ids, gates=gates, out=out)
    assert e.value.status == ARG
    layer(x, ids=ids, gates=gates, out=buf[32:544].view(8, 64))
    # out over x is allowed: x has been read by then
    ref = layer(x, top_k=2)[0]
    assert torch.equal(layer(x, top_k=2, out=x)[0], ref)


def test_norm_out_over_part_of_its_input_is_refused(E):
    wide = randn(1, 9, 200)
    with pytest.raises(E.EffortError) as e:
        E.block_norm(wide[:, :100], wide[:, 100:], x_out=wide[:, 99:199])
    assert e.value.status == ARG
    a, b = wide[:, :100].clone(), wide[:, 100:].clone()
    ref = E.block_norm(a, b)
    r = E.block_norm(wide[:, :100], wide[:, 100:], x_out=wide[:, :100], h_out=wide[:, 100:])
    assert torch.equal(r.x, ref.x) and torch.equal(r.h, ref.h)
