"""Feed-forward operators: the shapes at which the kernels change, and the ways
a program may call them (first inside a capture, from several threads)."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import ffn_reference as R
import test_gpu_block_norm as N
import test_gpu_fp8 as P
import test_gpu_moe as M

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dynamic_approximate_gemv_b200 import build
    build.build()
    import dynamic_approximate_gemv_b200 as E
    return E


# -- many rows of the norm go through shared memory, by width
@pytest.mark.parametrize("dim", [264, 512, 1024, 1032, 2048, 3000, 4096, 4104, 8192, 9000, 16384])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_norm_many_rows(E, dim, dt):
    N.check(E, 1200, dim, dt, "rms", "rms", "row", quantize=True)
    N.check(E, 777, dim, dt, "layer", "layer", "one", bias=True, off=1.0)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("wdt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,dim", [(200, 9000), (3, 12288), (5, 5003), (70, 8195)])
def test_norm_long_rows_by_weight_type(E, rows, dim, wdt, dt):
    N.check(E, rows, dim, dt, "rms", "layer", "row", bias=True, wdt=wdt, quantize=True)


@pytest.mark.parametrize("wdt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("form", [(None, "rms", None), ("rms", None, "one"), ("layer", "rms", None)])
def test_norm_many_rows_forms(E, wdt, dt, form):
    N.check(E, 900, 2048, dt, *form, wdt=wdt, bias=True)
    N.check(E, 900, 2048, dt, *form, weights=False, out_dtype="f32")


def test_norm_many_rows_without_a_branch(E):
    N.check(E, 2000, 1024, "bf16", None, "rms", None, with_y=False, a=0.5, quantize=True)
    N.check(E, 2000, 1024, "f16", None, "layer", None, with_y=False, a=1.0)


def test_norm_many_rows_in_place(E):
    x, y = N.draw(1500, 2048, torch.bfloat16), N.draw(1500, 2048, torch.bfloat16, 1)
    ref = E.block_norm(x, y, post="rms")
    r = E.block_norm(x, y, post="rms", x_out=x, h_out=y)
    assert torch.equal(r.x, ref.x) and torch.equal(y, ref.h)


def test_norm_many_rows_nonfinite_rows_stay_their_own(E):
    x = N.draw(800, 1024, torch.float32)
    ref = E.block_norm(x, quantize=True)
    bad = x.clone()
    bad[5, 3], bad[700, 1000] = float("nan"), float("inf")
    r = E.block_norm(bad, quantize=True)
    keep = [i for i in range(800) if i not in (5, 700)]
    assert torch.equal(r.q[keep].view(torch.uint8), ref.q[keep].view(torch.uint8))
    assert torch.equal(r.scales[keep], ref.scales[keep])
    assert not torch.isfinite(r.scales[5]).any()


def test_norm_and_quotients_of_every_size(E):
    """The quantised values are those of the division, for scales from subnormals to large."""
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn(700, 512, device="cuda", generator=g) * torch.logspace(-44, 36, 700, device="cuda")[:, None]
    q, s = E.quantize_e4m3(x)
    amax = x.reshape(700, 4, 128).abs().amax(2)
    assert torch.equal(s, amax / torch.full_like(amax, 448.0))
    d = s.repeat_interleave(128, 1)
    # a subnormal scale is rounded to a multiple of 2^-149, so that a quotient can pass 448: those saturate
    want = torch.where(d == 0, torch.zeros_like(x), x / d).clamp(-448, 448).to(torch.float8_e4m3fn)
    assert torch.equal(q.contiguous().view(torch.uint8), want.view(torch.uint8))


# -- the product's kernels
@pytest.mark.parametrize("rows,i,o", [(2, 2048, 16384), (8, 2048, 16384), (9, 2048, 1024), (16, 512, 4096), (12, 200000, 8),
                                      (7, 200000, 40), (16, 1100, 1900), (31, 130, 20000), (64, 9000, 257), (65, 9000, 257),
                                      (129, 3000, 513), (700, 520, 4000)])
def test_product_shapes(E, rows, i, o):
    P.check(E, rows, i, o, "f32", rows)


@pytest.mark.parametrize("rows", [1, 8, 16, 40, 128, 300])
@pytest.mark.parametrize("o", [1, 16, 17, 64, 127, 255, 256, 1001])
def test_product_narrow(E, rows, o):
    P.check(E, rows, 1500, o, "bf16", o)


@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,o", [(150, 75), (150, 300), (70, 511), (1000, 9000)])
def test_product_writes_its_rows_only(E, rows, o, dt):
    """Rows that start off 16 bytes, with what lies between them left as it was."""
    wq, ws, q, s = P.operands(rows, 500, o)
    m = E.Fp8Matrix(wq, ws)
    ref = m.matmul(q, s, out_dtype=dt)
    wide = torch.full((rows, o + 9), 7.0, device="cuda", dtype=dt)
    m.matmul(q, s, out=wide[:, 3:3 + o])
    assert torch.equal(wide[:, 3:3 + o], ref)
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 3 + o:] == 7).all())


def test_product_scales_off_sixteen_bytes(E):
    """x_scales whose rows start anywhere, with K blocks enough for whole batches."""
    wq, ws, q, s = P.operands(200, 3000, 300)
    m = E.Fp8Matrix(wq, ws)
    ref = m.matmul(q, s)
    wide = torch.full((200, 31), float("nan"), device="cuda")
    wide[:, 3:27] = s
    assert torch.equal(m.matmul(q, wide[:, 3:27]), ref)


# -- the mixture's chunks, shares and sets
@pytest.mark.parametrize("kind", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("experts,i,f,tokens,k", [(2, 256, 4200, 40, 1), (3, 130, 6000, 9, 2), (1, 512, 2100, 100, 1),
                                                  (40, 300, 200, 5, 8), (2, 2000, 70, 12, 2), (16, 64, 64, 60, 4)])
def test_mixture_shapes(E, kind, experts, i, f, tokens, k):
    c = M.Case(E, experts, i, f, kind)
    c.run(tokens, k, "bf16")
    c.run(tokens, k, "f32", out="f16")


def test_one_token_names_experts_twice(E):
    c = M.Case(E, 4, 200, 300, "e4m3")
    x = M.randn(1, 1, 200)
    ids = torch.tensor([[2, 2, 0, 2, -1]], device="cuda", dtype=torch.int32)
    gates = torch.tensor([[0.5, -0.25, 1.0, 2.0, 3.0]], device="cuda")
    c.check(x, ids, gates, c.layer(x, ids=ids, gates=gates)[0])


# -- the ways of calling
FIRST_IN_CAPTURE = """
import sys, torch
sys.path.insert(0, {root!r}); sys.path.insert(0, {root!r} + "/tests")
import dynamic_approximate_gemv_b200 as E
import ffn_reference as R
rows = int(sys.argv[1])
g = torch.Generator("cuda").manual_seed(1)
w = [0.05 * torch.randn(3, *s, device="cuda", generator=g) for s in ((256, 192), (256, 192), (192, 256))]
layer = E.MoeLayer(*(t.half() for t in w), router=torch.randn(3, 256, device="cuda", generator=g))
wq, ws = R.quantise_weights(0.05 * torch.randn(256, 384, device="cuda", generator=g))
m = E.Fp8Matrix(wq, ws)
x = torch.randn(rows, 256, device="cuda", generator=g).bfloat16()
def step():
    r = E.block_norm(x, pre="rms")
    y = layer(r.h, top_k=2)[0]
    n = E.block_norm(r.x, y, post="rms", quantize=True)
    return n.x, m.matmul(n.q, n.scales)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    a = step()
graph.replay()
torch.cuda.synchronize()
b = step()
torch.cuda.synchronize()
assert all(torch.equal(s, t) for s, t in zip(a, b))
assert torch.isfinite(b[1]).all()
print("ok")
"""


@pytest.mark.parametrize("rows", [1, 12, 100, 250])
def test_first_call_of_a_process_inside_a_capture(E, rows):
    p = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE.format(root=ROOT), str(rows)], capture_output=True,
                       text=True, timeout=300)
    assert p.returncode == 0 and "ok" in p.stdout, p.stderr[-2000:]


def test_two_threads_on_one_handle(E):
    wq, ws, q, s = P.operands(20, 2048, 512)
    m = E.Fp8Matrix(wq, ws)
    c = M.Case(E, 4, 256, 256, "f16")
    xs = [M.randn(k, 6, 256) for k in range(2)]
    ref, refs = m.matmul(q, s), [c.layer(x, top_k=2)[0] for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                a, b = m.matmul(q, s), c.layer(xs[k], top_k=2)[0]
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(a, ref) and torch.equal(b, refs[k])):
                    bad.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
