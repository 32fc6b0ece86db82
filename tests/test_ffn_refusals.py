"""Host-side argument checks of the feed-forward operators (block norm, e4m3
product, mixture of experts): every bad call is refused before any device work,
so no GPU is needed."""
import ctypes

import pytest

ARG, NOMEM, UNSUPPORTED = 1, 3, 6
vp = ctypes.c_void_p
FAKE = 0x100000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    from dynamic_approximate_gemv_b200 import build
    build.build()
    import dynamic_approximate_gemv_b200 as E
    return E.lib()


def norm_args(**kw):
    from dynamic_approximate_gemv_b200.ffn import _NormArgs
    base = dict(rows=4, dim=64, dtype=1, weight_dtype=1, h_dtype=1, post_kind=1, pre_kind=1, eps=1e-5,
                weight_offset=0.0, residual_scale=1.0, branch_scale=1.0, x=FAKE, x_stride=64, y=FAKE, y_stride=64,
                x_out=FAKE, x_out_stride=64, h_out=FAKE, h_stride=64)
    base.update(kw)
    return _NormArgs(**base)


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(dim=0), dict(x=None), dict(x=FAKE + 1), dict(y=FAKE + 1), dict(dtype=3), dict(dtype=-1),
    dict(weight_dtype=7), dict(h_dtype=5), dict(post_kind=3), dict(pre_kind=-1), dict(eps=-1.0),
    dict(eps=float("nan")), dict(eps=float("inf")), dict(residual_scale=float("nan")),
    dict(branch_scale=float("inf")), dict(weight_offset=float("nan")), dict(x_stride=63), dict(y_stride=10),
    dict(x_out_stride=63), dict(h_stride=0), dict(gate=FAKE, gate_stride=63), dict(gate=FAKE + 1),
    dict(y=None), dict(y=None, post_kind=0, gate=FAKE), dict(x_out=None, h_out=None), dict(q_out=FAKE, q_stride=64),
    dict(q_scales=FAKE, q_scales_stride=1), dict(q_out=FAKE, q_stride=63, q_scales=FAKE, q_scales_stride=1),
    dict(q_out=FAKE, q_stride=64, q_scales=FAKE, q_scales_stride=0),
    dict(q_out=FAKE, q_stride=64, q_scales=FAKE + 2, q_scales_stride=1), dict(pre_weight=FAKE + 1),
    dict(post_bias=FAKE + 1), dict(h_out=FAKE + 2, h_dtype=0),
])
def test_block_norm_refuses(L, kw):
    assert L.effort_block_norm(ctypes.byref(norm_args(**kw)), None) == ARG


def test_block_norm_limits(L):
    assert L.effort_block_norm(None, None) == ARG
    big = dict(x_stride=50000, y_stride=50000, x_out_stride=50000, h_stride=50000)
    assert L.effort_block_norm(ctypes.byref(norm_args(dim=40961, **big)), None) == UNSUPPORTED
    assert L.effort_block_norm(ctypes.byref(norm_args(rows=(1 << 24) + 1)), None) == UNSUPPORTED
    assert L.effort_block_norm(ctypes.byref(norm_args(rows=0)), None) == 0  # nothing to do, nothing launched


def test_fp8_prepare_refuses(L, monkeypatch):
    h = vp()
    p = L.effort_fp8_prepare
    assert p(None, FAKE, 4, 4, None, ctypes.byref(h)) == ARG
    assert p(FAKE, None, 4, 4, None, ctypes.byref(h)) == ARG
    assert p(FAKE, FAKE + 2, 4, 4, None, ctypes.byref(h)) == ARG
    assert p(FAKE, FAKE, 0, 4, None, ctypes.byref(h)) == ARG
    assert p(FAKE, FAKE, 4, -1, None, ctypes.byref(h)) == ARG
    assert p(FAKE, FAKE, 4, 4, None, None) == ARG
    assert p(FAKE, FAKE, 300000, 4, None, ctypes.byref(h)) == UNSUPPORTED
    assert p(FAKE, FAKE, 262144, 262144, None, ctypes.byref(h)) == UNSUPPORTED
    monkeypatch.setenv("EFFORT_ALLOC_CAP_BYTES", "4096")
    assert p(FAKE, FAKE, 4096, 4096, None, ctypes.byref(h)) == NOMEM
    assert h.value is None


def test_fp8_calls_refuse_null_handles(L):
    assert L.effort_fp8_matmul(None, FAKE, 128, FAKE, 1, 1, 0, FAKE, 4, None) == ARG
    assert L.effort_fp8_get_info(None, None, None, None) == ARG
    assert L.effort_fp8_destroy(None) == ARG


def moe_weights(**kw):
    from dynamic_approximate_gemv_b200.ffn import _MoeWeights
    base = dict(n_experts=4, in_dim=64, hidden_dim=64, weight_kind=0, w1=FAKE, w3=FAKE, w2=FAKE, router=FAKE,
                router_dtype=0)
    base.update(kw)
    return _MoeWeights(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(n_experts=0), ARG), (dict(in_dim=0), ARG), (dict(hidden_dim=-4), ARG), (dict(w1=None), ARG),
    (dict(w3=None), ARG), (dict(w2=None), ARG), (dict(weight_kind=3), ARG), (dict(w1=FAKE + 1), ARG),
    (dict(weight_kind=2), ARG), (dict(s1=FAKE, s3=FAKE, s2=FAKE), ARG),
    (dict(weight_kind=2, s1=FAKE, s3=FAKE, s2=FAKE + 2), ARG), (dict(router_dtype=9), ARG),
    (dict(router=FAKE + 2), ARG), (dict(n_experts=257), UNSUPPORTED), (dict(in_dim=40961), UNSUPPORTED),
    (dict(hidden_dim=40961), UNSUPPORTED),
])
def test_moe_prepare_refuses(L, kw, status):
    h = vp()
    assert L.effort_moe_prepare(ctypes.byref(moe_weights(**kw)), None, ctypes.byref(h)) == status
    assert h.value is None


def test_moe_calls_refuse_null_handles_and_the_cap(L, monkeypatch):
    h, n = vp(), ctypes.c_size_t()
    assert L.effort_moe_prepare(None, None, ctypes.byref(h)) == ARG
    assert L.effort_moe_prepare(ctypes.byref(moe_weights()), None, None) == ARG
    assert L.effort_moe_scratch_bytes(None, 1, 1, ctypes.byref(n)) == ARG
    assert L.effort_moe_forward(None, FAKE, 0, 64, 1, 1, 0, FAKE, FAKE, FAKE, 0, 64, FAKE, 0, None) == ARG
    assert L.effort_moe_get_info(None, None, None, None, None) == ARG
    assert L.effort_moe_destroy(None) == ARG
    monkeypatch.setenv("EFFORT_ALLOC_CAP_BYTES", "4096")
    assert L.effort_moe_prepare(ctypes.byref(moe_weights()), None, ctypes.byref(h)) == NOMEM
    assert h.value is None


def test_matvec_entry_points_refuse_bf16(L):
    """EFFORT_BF16 belongs to the feed-forward operators; the matvec's entry
    points refuse a null handle and an unknown dtype alike with ARG."""
    assert L.effort_gemv_ex(None, FAKE, 2, ctypes.c_float(0.5), FAKE, None, None, None, None) == ARG
    assert L.effort_gemv_batched(None, None, None, None, 1, None, 2, None, None, None, None, None) == ARG


def test_binding_refuses_host_tensors():
    import torch

    import dynamic_approximate_gemv_b200 as E
    with pytest.raises(ValueError):
        E.block_norm(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        E.quantize_e4m3(torch.zeros(2, 8))
    with pytest.raises(ValueError):
        E.Fp8Matrix(torch.zeros(8, 8).to(torch.float8_e4m3fn), torch.ones(1, 1))
    with pytest.raises(ValueError):
        E.MoeLayer(torch.zeros(2, 8, 8).half(), torch.zeros(2, 8, 8).half(), torch.zeros(2, 8, 8).half())

