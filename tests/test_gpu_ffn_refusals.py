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


# -- gradients: there is no backward pass, so none is dropped in silence

def test_inputs_that_want_gradients_are_refused(E, matrix, layer):
    x, w = randn(0, 4, 64), randn(1, 64)
    for call in (lambda t: E.block_norm(t), lambda t: E.block_norm(x, t), lambda t: E.block_norm(x, x, gate=t),
                 lambda t: E.block_norm(x, pre_weight=t[0]), lambda t: E.block_norm(x, x, post="layer", post_bias=t[0]),
                 lambda t: E.quantize_e4m3(t), lambda t: layer(t, top_k=1),
                 lambda t: layer(x, ids=torch.zeros(4, 64, device="cuda", dtype=torch.int32)[:, :2].contiguous(),
                                 gates=t[:, :2].contiguous())):
        with pytest.raises(RuntimeError, match="gradient"):
            call(x.clone().requires_grad_())
        with torch.no_grad():
            call(torch.nn.Parameter(x.clone()))
        call(x)
    q, s = E.quantize_e4m3(randn(2, 3, 256))
    with pytest.raises(RuntimeError, match="gradient"):
        matrix.matmul(q, s.clone().requires_grad_())
    with torch.no_grad():
        assert torch.equal(matrix.matmul(q, s.clone().requires_grad_()), matrix.matmul(q, s))


def test_tensors_without_plain_storage_are_refused(E, layer):
    x = randn(0, 4, 3, 64)
    with pytest.raises((TypeError, ValueError)):
        torch.vmap(lambda t: E.block_norm(t).h)(x)
    with pytest.raises((TypeError, ValueError)):
        torch.vmap(lambda t: layer(t, top_k=1)[0])(x)
    with pytest.raises((TypeError, ValueError)):
        E.block_norm(torch._neg_view(x[0]))
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        fake = torch.empty(3, 64, device="cuda")
    with pytest.raises((TypeError, ValueError)):
        E.block_norm(fake)


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


# -- sizes

@pytest.mark.parametrize("k", [-1, 17, 2 ** 31, 2 ** 40])
def test_top_k_is_checked_before_anything_is_made(E, layer, k):
    held = torch.cuda.memory_reserved()
    with pytest.raises(E.EffortError):
        layer(randn(0, 4, 64), top_k=k)
    assert torch.cuda.memory_reserved() <= held + (4 << 20)


def test_too_many_tokens_are_refused_before_anything_is_made(E, layer):
    x = torch.zeros(1, 64, device="cuda").expand(1 << 22, 64)
    held = torch.cuda.memory_reserved()
    with pytest.raises(E.EffortError):
        layer(x, top_k=1)
    assert torch.cuda.memory_reserved() <= held + (4 << 20)


# -- closed handles

def test_closed_handles_are_refused(E):
    m = E.Fp8Matrix(*R.quantise_weights(0.05 * randn(1, 256, 128)))
    layer = E.MoeLayer(*(0.05 * randn(k, 2, 32, 32).half() for k in range(3)), router=randn(9, 2, 32))
    q, s = E.quantize_e4m3(randn(2, 3, 256))
    for h in (m, layer):
        h.close()
        h.close()
    for call in (lambda: m.matmul(q, s), m.info, lambda: layer(randn(0, 4, 32), top_k=1), layer.info):
        with pytest.raises(E.EffortError) as e:
            call()
        assert e.value.status == ARG


# -- types of the matvec entry points, on live handles

def test_matvecs_refuse_bfloat16_vectors(E):
    W = (0.02 * randn(3, 256, 512)).half()
    pm, ws = E.PreparedMatrix(W), E.Workspace(256, 512)
    L, out = E.lib(), torch.empty(512, device="cuda")
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for dtype, v, want in ((0, randn(4, 256), 0), (1, randn(4, 256).half(), 0), (2, randn(4, 256).bfloat16(), ARG),
                           (3, randn(4, 256), ARG), (-1, randn(4, 256), ARG)):
        p = ctypes.c_void_p(v.data_ptr())
        o = ctypes.c_void_p(out.data_ptr())
        assert L.effort_gemv_ex(pm._h, p, dtype, ctypes.c_float(0.5), o, None, None, None, stream) == want
        assert L.effort_gemv_static(pm._h, p, dtype, ctypes.c_float(0.5), o, None, None, None, stream) == want
        handles, zero = (ctypes.c_void_p * 1)(pm._h.value), (ctypes.c_int32 * 1)(0)
        assert L.effort_gemv_batched(ws._h, handles, zero, zero, 1, p, dtype, (ctypes.c_float * 1)(0.5), o, None, None,
                                     stream) == want
        assert L.effort_dense_gemv(ws._h, ctypes.c_void_p(W.data_ptr()), 256, 512, p, dtype, o, stream) == want
    torch.cuda.synchronize()
    ws.close()
    pm.close()


# -- one dimension

def test_one_dimension_with_every_argument(E):
    x, y, g = randn(0, 500), randn(1, 500), randn(2, 500)
    ref = E.block_norm(x[None], y[None], gate=g[None], post="layer", out_dtype=torch.bfloat16)
    xo, ho = torch.empty(500, device="cuda"), torch.empty(500, device="cuda", dtype=torch.bfloat16)
    r = E.block_norm(x, y, gate=g, post="layer", x_out=xo, h_out=ho)
    assert r.x.data_ptr() == xo.data_ptr() and r.h.data_ptr() == ho.data_ptr()
    assert torch.equal(xo, ref.x[0]) and torch.equal(ho, ref.h[0])
    ref = E.block_norm(x[None], y[None], gate=g[None], post="layer", quantize=True)
    r = E.block_norm(x, y, gate=g[None], post="layer", quantize=True)
    assert r.q.shape == (500,) and r.scales.shape == (4,)
    assert torch.equal(r.x, ref.x[0]) and torch.equal(r.scales, ref.scales[0])
    assert torch.equal(r.q.view(torch.uint8), ref.q[0].view(torch.uint8))
