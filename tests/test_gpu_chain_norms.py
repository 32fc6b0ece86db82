"""The decode chain as the benchmark runs it: its matvecs joined by the library's
norm.  Every norm is compared with 64 bits and every matvec with the oracle, on
the values that the chain itself hands on, and the captured chain gives what
its calls give one by one."""
import os
import sys

import numpy as np
import pytest
import torch

import ffn_reference as R
from dynamic_approximate_gemv_b200 import inputs
from oracle import effort_oracle as O
from test_gpu_chain import checked_gemv

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DIMS = (512, 128, 1792)


@pytest.fixture(scope="module")
def E():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dynamic_approximate_gemv_b200 import build
    build.build()
    import dynamic_approximate_gemv_b200 as E
    return E


class CheckedNorm:
    """The library's block_norm, each call compared with its definition."""

    def __init__(self, E):
        self.E, self.calls = E, 0

    def block_norm(self, v):
        r = self.E.block_norm(v)
        _, (h, dh) = R.block_norm(v[None], None, None, "rms", None, 1.0, 1.0, None, None, None, None, 0.0, 1e-5)
        R.assert_close(r.h, h[0], dh[0])
        self.calls += 1
        return r


class CheckedMatrix:
    def __init__(self, pm, prep):
        self.pm, self.prep, self.calls = pm, prep, 0

    def gemv(self, v, effort):
        self.calls += 1
        return checked_gemv(self.pm, self.prep, v, effort)


def test_chain_with_the_librarys_norm(E):
    sys.path.insert(0, ROOT)
    import bench
    mats, checked = [], []
    for layer in range(2):
        L, C = {}, {}
        for m, (name, a, b) in enumerate(bench.CHAIN_MATS):
            Wn = inputs.weights(DIMS[a], DIMS[b], 1000 * layer + m)
            L[name] = E.PreparedMatrix(torch.from_numpy(Wn).cuda(), 0.8)
            C[name] = CheckedMatrix(L[name], O.Prepared(Wn.view(np.uint16), 0.8))
        mats.append(L)
        checked.append(C)
    try:
        x = torch.from_numpy(inputs.vector(DIMS[0], 9)).cuda()
        norm = CheckedNorm(E)
        want = bench.chain_token(norm, checked, x, 0.25)
        assert norm.calls == 10 and all(c.calls == 1 for C in checked for c in C.values())
        assert torch.equal(bench.chain_token(E, mats, x, 0.25), want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            bench.chain_token(E, mats, x, 0.25)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = bench.chain_token(E, mats, x, 0.25)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del g
    finally:
        for L in mats:
            for pm in L.values():
                pm.close()
