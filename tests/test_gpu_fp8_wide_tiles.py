"""The e4m3 product where a hundred tiles of 128 x 256 and more are to be made:
the kernel of long prompts, with rows, columns and K that end inside a tile."""
import pytest
import torch

import ffn_reference as R
import test_gpu_fp8 as P

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


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,i,o", [(1283, 1000, 2500), (1280, 130, 2560), (12801, 250, 200), (128, 512, 25601),
                                      (1793, 4091, 1793), (1300, 1, 2307), (2049, 1152, 4111)])
def test_ragged(E, rows, i, o, dt):
    P.check(E, rows, i, o, dt, rows)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_nonfinite_rows_stay_their_own(E, dt):
    wq, ws, q, s = P.operands(1400, 400, 2570)
    m = E.Fp8Matrix(wq, ws)
    ref = m.matmul(q, s, out_dtype=DT[dt])
    want, tol = R.product(q, s, wq, ws)
    R.assert_close(ref, want, tol)
    bad = [0, 127, 128, 700, 1399]
    q.view(torch.uint8)[bad[0], 7] = 0x7F
    q.view(torch.uint8)[bad[2], 399] = 0xFF
    s[bad[1], 2], s[bad[3], 0], s[bad[4], 3] = float("inf"), float("nan"), float("-inf")
    out = m.matmul(q, s, out_dtype=DT[dt])
    assert torch.isnan(out[[0, 128, 700]]).all() and not torch.isfinite(out[[127, 1399]]).any()
    keep = [r for r in range(1400) if r not in bad]
    assert torch.equal(out[keep], ref[keep])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_writes_its_rows_only(E, dt):
    """Off 16 bytes and inside a wider array, against 64 bits."""
    wq, ws, q, s = P.operands(1290, 500, 2563)
    want, tol = R.product(q, s, wq, ws)
    wide = torch.full((1292, 2570), 7.0, device="cuda", dtype=DT[dt])
    E.Fp8Matrix(wq, ws).matmul(q, s, out=wide[:1290, 3:2566])
    R.assert_close(wide[:1290, 3:2566], want, tol)
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, 2566:] == 7).all()) and bool((wide[1290:] == 7).all())


def test_one_nonzero_entry(E):
    i, o, rows = 300, 2570, 1290
    for r, k, n in [(0, 0, 0), (127, 127, 255), (128, 128, 256), (1289, 299, 2569), (640, 200, 1279), (129, 17, 128)]:
        wq = torch.zeros(i, o, device="cuda").to(torch.float8_e4m3fn)
        wq.view(torch.uint8)[k, n] = 0x38  # 1.0
        q = torch.zeros(rows, 304, device="cuda", dtype=torch.uint8)
        q[r, k] = 0xC0  # -2.0
        ws = torch.full((3, 21), 0.5, device="cuda")
        s = torch.full((rows, 3), 3.0, device="cuda")
        out = E.Fp8Matrix(wq, ws).matmul(q.view(torch.float8_e4m3fn)[:, :i], s, out_dtype=torch.float32)
        want = torch.zeros(rows, o, device="cuda")
        want[r, n] = -3.0
        assert torch.equal(out, want), (r, k, n)
