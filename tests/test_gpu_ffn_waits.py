"""Waits inside the feed-forward kernels: they do not count the time of the kernel
before, and one that runs out leaves NaN, never a wrong number.  In child
processes with the debug build, whose environment variables shorten the waits
and let them run out (every one of them ends by itself)."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

HEAD = """
import os, sys, torch
sys.path.insert(0, {root!r}); sys.path.insert(0, {root!r} + "/tests")
import dynamic_approximate_gemv_b200 as E
import ffn_reference as R
g = torch.Generator("cuda").manual_seed(1)
randn = lambda *s: torch.randn(*s, device="cuda", generator=g)
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dynamic_approximate_gemv_b200 import build
    build.build()


def child(code, *args):
    env = dict(os.environ, EFFORT_DEBUG_LIB="1")
    r = subprocess.run([sys.executable, "-c", HEAD.format(root=ROOT) + code, *map(str, args)], env=env, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]


BEHIND_A_LONG_KERNEL = """
# A kernel of another program's that lets its successor start at once and then takes 0.2 s (its loop is bounded).
# One of its blocks leaves the other SMs to the product, whose waits have 20000 tries: a few ms.
source = r'''
extern "C" __global__ void lingering(long long ns) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  long long t0, t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t0));
  for (int i = 0; i < 1 << 28; ++i) {
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    if (t - t0 > ns) break;
  }
}
'''
lingering = torch.cuda._compile_kernel(source, "lingering")
rows, i, o = map(int, sys.argv[1:])
m = E.Fp8Matrix(*R.quantise_weights(0.05 * randn(i, o)))
q, s = E.quantize_e4m3(randn(rows, i))
ref = m.matmul(q, s, out_dtype=torch.float32)
torch.cuda.synchronize()
os.environ["EFFORT_TEST_WAIT_TRIES"] = "20000"
lingering(grid=(1, 1, 1), block=(32, 1, 1), args=[200_000_000])
out = m.matmul(q, s, out_dtype=torch.float32)
torch.cuda.synchronize()
assert torch.equal(out, ref), torch.isnan(out).float().mean()
print("ok")
"""


@pytest.mark.parametrize("rows,i,o", [(4, 512, 512), (12, 2048, 4096), (40, 1024, 512), (200, 1024, 512), (1300, 512, 2560)])
def test_product_behind_a_long_kernel(rows, i, o):
    child(BEHIND_A_LONG_KERNEL, rows, i, o)


LOST = """
# From the given stage of every block's ring on, 16 bytes are waited for that never come.
rows, i, o, after = map(int, sys.argv[1:])
m = E.Fp8Matrix(*R.quantise_weights(0.05 * randn(i, o)))
q, s = E.quantize_e4m3(randn(rows, i))
ref = m.matmul(q, s, out_dtype=torch.float32)
torch.cuda.synchronize()
os.environ["EFFORT_TEST_WAIT_TRIES"] = "20000"
os.environ["EFFORT_TEST_LOST_COPY"] = str(after)
out = m.matmul(q, s, out_dtype=torch.float32)
torch.cuda.synchronize()
nan = torch.isnan(out)
assert torch.equal(out[~nan], ref[~nan])
print("NaN", float(nan.float().mean()))
assert nan.all() if after == 0 else nan.any()
del os.environ["EFFORT_TEST_WAIT_TRIES"], os.environ["EFFORT_TEST_LOST_COPY"]
assert torch.equal(m.matmul(q, s, out_dtype=torch.float32), ref)
torch.cuda.synchronize()
print("ok")
"""


# few rows on the rings of stream.cuh (alone and in clusters); clusters with joined parts (up to 64 rows, and 128 x 128 tiles), and 128 x 256 tiles of several rounds; `after` is
# below a block's share of K blocks in each
@pytest.mark.parametrize("rows,i,o,after", [(1, 512, 512, 0), (1, 4096, 14336, 0), (1, 4096, 14336, 3), (8, 14336, 4096, 2),
                                            (13, 1000, 500, 0), (3, 40000, 100, 1), (12, 2048, 4096, 0), (12, 2048, 4096, 2), (30, 4096, 300, 1), (64, 4096, 14336, 0),
                                            (64, 4096, 14336, 13), (200, 4091, 1003, 2), (1024, 1024, 4096, 5),
                                            (2000, 2048, 8192, 0), (2000, 2048, 8192, 20)])
def test_product_whose_waits_run_out(rows, i, o, after):
    """Every output is right or NaN, and the next call is right."""
    child(LOST, rows, i, o, after)


LOST_MIXTURE = """
# As above, in the mixture's products: what a lost copy of the first leaves goes through the second.
kind, dt, tokens, after = sys.argv[1], *map(int, sys.argv[2:])
e, i, f = 4, 1024, 1792
w = [0.05 * randn(e, *d) for d in ((i, f), (i, f), (f, i))]
scales = None
if kind == "e4m3":
    w, scales = zip(*(R.quantise_weights(t) for t in w))
else:
    w = [t.to({{"f16": torch.float16, "bf16": torch.bfloat16}}[kind]) for t in w]
layer = E.MoeLayer(*w, scales=scales, router=randn(e, i))
x = randn(tokens, i).to([torch.float32, torch.bfloat16][dt])
ref = layer(x, top_k=2)[0]
torch.cuda.synchronize()
os.environ["EFFORT_TEST_WAIT_TRIES"] = "20000"
os.environ["EFFORT_TEST_LOST_COPY"] = str(after)
out = layer(x, top_k=2)[0]
torch.cuda.synchronize()
nan = torch.isnan(out)
assert torch.equal(out[~nan], ref[~nan])
print("NaN", float(nan.float().mean()))
assert nan.any() and (after or nan.all())
del os.environ["EFFORT_TEST_WAIT_TRIES"], os.environ["EFFORT_TEST_LOST_COPY"]
assert torch.equal(layer(x, top_k=2)[0], ref)
torch.cuda.synchronize()
print("ok")
""".replace("{{", "{").replace("}}", "}")


@pytest.mark.parametrize("kind,dt,tokens,after", [("e4m3", 0, 1, 0), ("e4m3", 1, 7, 1), ("f16", 0, 1, 1), ("f16", 1, 20, 0),
                                                  ("bf16", 0, 40, 2), ("bf16", 1, 3, 0)])
def test_mixture_whose_waits_run_out(kind, dt, tokens, after):
    child(LOST_MIXTURE, kind, dt, tokens, after)


LOST_NORM = """
rows, dim, after = map(int, sys.argv[1:])
x, y = randn(rows, dim).bfloat16(), randn(rows, dim).bfloat16()
call = lambda **kw: E.block_norm(x, y, post="rms", gate=y, pre="layer", **kw)
ref, refq = call(), call(quantize=True)
torch.cuda.synchronize()
os.environ["EFFORT_TEST_WAIT_TRIES"] = "20000"
os.environ["EFFORT_TEST_LOST_COPY"] = str(after)
out, outq = call(), call(quantize=True)
torch.cuda.synchronize()
for a, b in ((out.x, ref.x), (out.h, ref.h), (outq.scales, refq.scales), (outq.q.float(), refq.q.float())):
    nan = torch.isnan(a)
    assert torch.equal(a[~nan], b[~nan]) and nan.any() and (after or nan.all())
    assert not after or not nan.all()
del os.environ["EFFORT_TEST_WAIT_TRIES"], os.environ["EFFORT_TEST_LOST_COPY"]
assert torch.equal(call().h, ref.h)
torch.cuda.synchronize()
print("ok")
"""


@pytest.mark.parametrize("rows,dim,after", [(8000, 1024, 0), (8000, 1024, 1), (2000, 4096, 2), (900, 16384, 3)])
def test_norm_whose_waits_run_out(rows, dim, after):
    child(LOST_NORM, rows, dim, after)
