"""The mixture-of-experts layer against its definition in 64 bits."""
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


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(seed, *shape):
    return torch.randn(*shape, generator=gen(seed), device="cuda")


class Case:
    def __init__(self, E, experts, i, f, kind, seed=0, router_dt=torch.float32, scale=0.02):
        w = [randn(seed + k, *s) * scale for k, s in enumerate([(experts, i, f), (experts, i, f), (experts, f, i)])]
        scales = None
        if kind == "e4m3":
            qs = [R.quantise_weights(t) for t in w]
            w, scales = [q for q, _ in qs], tuple(s for _, s in qs)
            self.w64 = [R.dequantise_weights(q, s) for q, s in qs]
        else:
            w = [t.to(DT[kind]) for t in w]
            self.w64 = [t.double() for t in w]
        self.router = (randn(seed + 3, experts, i) / 8).to(router_dt)
        self.layer = E.MoeLayer(*w, scales=scales, router=self.router)
        self.E, self.experts, self.i = E, experts, i

    def check(self, x, ids, gates, out, what=""):
        ref, tol = R.moe(x, *self.w64, ids, gates, out.dtype)
        R.assert_close(out, ref, tol, what)

    def run(self, tokens, k, dt="f32", out=None, seed=9, **kw):
        x = randn(seed, tokens, self.i).to(DT[dt])
        o, ids, gates = self.layer(x, top_k=k, out_dtype=out and DT[out], **kw)
        want, soft, part = R.route(x, self.router, k)
        assert torch.equal(ids, want)
        g = part if kw.get("gate_mode") == "top_of_softmax" else soft
        R.assert_close(gates, g, g * 64 * R.U32 + 1e-5 * g, "gates")  # logits to 1e-5: |x||w| sums of up to 4096 terms
        self.check(x, ids, gates, o, f"{tokens} tokens, top {k}")
        again = self.layer(x, top_k=k, out_dtype=out and DT[out], **kw)
        assert torch.equal(again[0], o)  # bit for bit
        return x, o


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("out", ["f32", "f16", "bf16"])
def test_types(E, kind, dt, out):
    c = Case(E, 4, 256, 384, kind)
    c.run(5, 2, dt, out)


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("i,f", [(1, 1), (8, 16), (7, 9), (65, 63), (128, 128), (129, 257), (200, 1003), (1000, 120)])
def test_ragged(E, kind, i, f):
    c = Case(E, 5, i, f, kind)
    for tokens in (1, 3, 20):
        c.run(tokens, 2, "f32")
        c.run(tokens, 1, "bf16")


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 130, 256])
def test_tokens(E, kind, tokens):
    Case(E, 3, 192, 160, kind).run(tokens, 2, "f16")


@pytest.mark.parametrize("experts,k", [(1, 1), (2, 2), (16, 16), (64, 6), (255, 8), (256, 16)])
def test_experts_and_top(E, experts, k):
    c = Case(E, experts, 64, 48, "bf16")
    c.run(1, k, "bf16")
    c.run(19, k, "f32", gate_mode="top_of_softmax")


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
def test_all_tokens_to_one_expert(E, kind):
    """The longest list one expert can get, through the caller's own routing."""
    c = Case(E, 4, 136, 200, kind)
    x = randn(1, 256, 136)
    ids = torch.full((256, 3), 2, device="cuda", dtype=torch.int32)  # and three times by each token
    gates = torch.rand(256, 3, device="cuda", generator=gen(2))
    out, i2, g2 = c.layer(x, ids=ids, gates=gates)
    assert i2 is ids and g2 is gates
    c.check(x, ids, gates, out)


def test_given_routing_with_padding(E):
    c = Case(E, 4, 100, 72, "f16")
    x = randn(1, 9, 100)
    ids = torch.tensor([[0, 1], [-1, 2], [3, 4], [-1, -1], [1, 1], [99, 2**31 - 1], [-2**31, 0], [2, 3], [0, 3]],
                       device="cuda", dtype=torch.int32)
    gates = torch.rand(9, 2, device="cuda", generator=gen(2)) - 0.3
    x[3] = float("nan")  # padding rows may hold anything
    out = torch.full((11, 104), 7.0, device="cuda")
    c.layer(x, ids=ids, gates=gates, out=out[:9, :100])
    valid = torch.where((ids >= 0) & (ids < 4), ids, -1)
    x2 = x.clone()
    x2[3] = 0
    c.check(x2, valid, gates, out[:9, :100])
    assert bool((out[3, :100] == 0).all() and (out[5, :100] == 0).all())
    assert bool((out[9:] == 7).all() and (out[:, 100:] == 7).all())


def test_ties_go_to_the_lower_expert(E):
    c = Case(E, 8, 64, 64, "f16")
    row = randn(5, 1, 64) / 8
    c.router = row.expand(8, 64).contiguous()
    layer = E.MoeLayer(*(t.half() for t in c.w64), router=c.router)
    _, ids, gates = layer(randn(6, 4, 64), top_k=3)
    assert torch.equal(ids, torch.tensor([[0, 1, 2]] * 4, device="cuda", dtype=torch.int32))
    assert torch.allclose(gates, torch.full_like(gates, 1 / 3), rtol=4 * R.U32)


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
def test_nonfinite_tokens_stay_their_own(E, kind):
    c = Case(E, 4, 160, 96, kind)
    x = randn(1, 12, 160)
    ids = torch.randint(0, 4, (12, 2), device="cuda", generator=gen(3), dtype=torch.int32)
    gates = torch.rand(12, 2, device="cuda", generator=gen(4)) + 0.1
    ref = c.layer(x, ids=ids, gates=gates)[0]
    bad = x.clone()
    bad[3, 17] = float("nan")
    bad[8, 20] = float("inf")
    out = c.layer(bad, ids=ids, gates=gates)[0]
    keep = [t for t in range(12) if t not in (3, 8)]
    assert torch.equal(out[keep], ref[keep])
    assert torch.isnan(out[3]).all() and not torch.isfinite(out[8]).any()
    # and the router with a NaN token: in-range ids, NaN gates, other tokens as before
    o1, i1, g1 = c.layer(x, top_k=2)
    o2, i2, g2 = c.layer(bad, top_k=2)
    assert bool(((i2 >= 0) & (i2 < 4)).all()) and torch.isnan(g2[3]).all()
    assert torch.equal(o1[keep], o2[keep]) and torch.equal(i1[keep], i2[keep])


@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("mag", [1e-12, 1e-3, 3e4, 1e9])
def test_ranges(E, kind, mag):
    """x far from 1: nothing overflows inside where the result is in range."""
    c = Case(E, 2, 256, 128, kind)
    x = randn(1, 3, 256) * mag
    x[:, 0] *= 50
    ids = torch.tensor([[0, 1]] * 3, device="cuda", dtype=torch.int32)
    gates = torch.full((3, 2), 0.5, device="cuda")
    c.check(x, ids, gates, c.layer(x, ids=ids, gates=gates)[0])


@pytest.mark.parametrize("router_dt", ["f32", "f16", "bf16"])
def test_router_types(E, router_dt):
    Case(E, 8, 320, 64, "f16", router_dt=DT[router_dt]).run(6, 2, "bf16")


def test_strides(E):
    c = Case(E, 4, 130, 70, "bf16")
    wide = randn(1, 5, 300).bfloat16()
    x = wide[:, 7:137]
    a = c.layer(x, top_k=2)
    b = c.layer(x.contiguous(), top_k=2)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind,tokens", [("e4m3", 1), ("f16", 16), ("bf16", 3)])
def test_full_size(E, kind, tokens):
    """Two experts of 4096 x 14336."""
    c = Case(E, 2, 4096, 14336, kind)
    c.run(tokens, 1, "bf16")
    if kind == "e4m3":
        c.run(tokens, 2, "f32")


def test_streams_and_graphs(E):
    c = Case(E, 8, 512, 448, "e4m3")
    xs = [randn(20 + k, 5, 512).half() for k in range(4)]
    ref = [c.layer(x, top_k=2)[0] for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [None] * 4
    torch.cuda.synchronize()
    for _ in range(4):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[k] = c.layer(xs[k], top_k=2)[0]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    graphs = []
    for x in xs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = c.layer(x, top_k=2)[0]
        graphs.append((g, o))
    for k, (g, _) in enumerate(graphs):
        with torch.cuda.stream(streams[k]):
            for _ in range(5):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for (_, o), r in zip(graphs, ref))


def test_no_tokens(E):
    c = Case(E, 2, 32, 32, "f16")
    out, ids, gates = c.layer(torch.empty(0, 32, device="cuda"), top_k=2)
    assert out.shape == (0, 32) and ids.shape == (0, 2)


def test_nonfinite_weights_are_refused(E):
    w = [randn(k, 2, 32, 32).half() for k in range(3)]
    w[1][1, 3, 4] = float("inf")
    with pytest.raises(E.EffortError) as e:
        E.MoeLayer(*w)
    assert e.value.status == 4


def test_binding_refuses(E):
    c = Case(E, 4, 64, 32, "f16")
    x = randn(1, 3, 64)
    ids, gates = torch.zeros(3, 2, device="cuda", dtype=torch.int32), torch.zeros(3, 2, device="cuda")
    bad = [
        (ValueError, lambda: c.layer(x)),
        (ValueError, lambda: c.layer(x[:, :63], top_k=1)),
        (ValueError, lambda: c.layer(x, top_k=2, gate_mode="sigmoid")),
        (ValueError, lambda: c.layer(x, ids=ids)),
        (ValueError, lambda: c.layer(x, ids=ids.long(), gates=gates)),
        (ValueError, lambda: c.layer(x, ids=ids[:2], gates=gates[:2])),
        (ValueError, lambda: c.layer(x, top_k=3, ids=ids, gates=gates)),
        (TypeError, lambda: c.layer(x.double(), top_k=1)),
        (TypeError, lambda: c.layer(x, top_k=1, out_dtype=torch.float64)),
        (E.EffortError, lambda: c.layer(x, top_k=5)),
        (E.EffortError, lambda: c.layer(x, top_k=0)),
        (E.EffortError, lambda: c.layer(randn(1, 257, 64), top_k=1)),
        (ValueError, lambda: E.MoeLayer(*(randn(k, 2, 32, 32).half() for k in range(3)))(randn(1, 1, 32), top_k=1)),
    ]
    for kind, call in bad:
        with pytest.raises(kind):
            call()


def test_layer_between_norms(E):
    """Norm, experts, norm with the residual: the run of a decoder block."""
    c = Case(E, 4, 256, 192, "e4m3")
    x = randn(1, 6, 256).bfloat16()
    w = (1 + 0.1 * randn(2, 256)).bfloat16()
    r = E.block_norm(x, pre="rms", pre_weight=w)
    y, ids, gates = c.layer(r.h, top_k=2)
    c.check(r.h, ids, gates, y)
    n = E.block_norm(r.x, y, post="rms", post_weight=w, pre="rms", pre_weight=w, quantize=True)
    (v, dv), (h, dh) = R.block_norm(x, y, "rms", "rms", None, 1.0, 1.0, w, None, w, None, 0.0, 1e-5)
    R.assert_close(n.x, v, dv)
    R.check_quantised(n.q, n.scales, h, dh)
