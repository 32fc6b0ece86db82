"""The product with e4m3 operands against its definition in 64 bits."""
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


def operands(rows, i, o, seed=0):
    wq, ws = R.quantise_weights(0.02 * torch.randn(i, o, generator=gen(seed), device="cuda"))
    x = torch.randn(rows, -(-i // 16) * 16, generator=gen(seed + 1), device="cuda")
    x = x * (1 + 9 * (torch.rand(x.shape[1], generator=gen(seed + 2), device="cuda") < 0.02))
    pad = torch.nn.functional.pad(x[:, :i], (0, R.blocks(i) * 128 - i)).reshape(rows, -1, 128)
    s = pad.abs().amax(2) / 448
    # what lies between the end of a row and the next one is not read as a value: NaN bytes there
    q = torch.full((rows, -(-i // 16) * 16), 0x7F, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    q[:, :i] = (pad / s[..., None]).reshape(rows, -1)[:, :i].to(torch.float8_e4m3fn)
    return wq, ws, q[:, :i], s


def check(E, rows, i, o, dt="bf16", seed=0):
    wq, ws, q, s = operands(rows, i, o, seed)
    m = E.Fp8Matrix(wq, ws)
    out = m.matmul(q, s, out_dtype=DT[dt])
    ref, tol = R.product(q, s, wq, ws)
    R.assert_close(out, ref, tol, f"{rows}x{i}x{o}")
    assert torch.equal(out, m.matmul(q, s, out_dtype=DT[dt]))  # and again, bit for bit
    return m


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 400])
def test_rows(E, rows):
    check(E, rows, 512, 384, "f32", rows)


@pytest.mark.parametrize("rows", [1, 5, 24, 70, 300])
@pytest.mark.parametrize("i,o", [(1, 1), (16, 8), (15, 3), (127, 129), (128, 128), (129, 127), (1000, 77), (4091, 1003),
                                 (260, 2048), (2500, 130)])
def test_ragged(E, rows, i, o):
    check(E, rows, i, o, "f32", rows + i)


@pytest.mark.parametrize("rows", [1, 12, 40, 200])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_out_types(E, rows, dt):
    check(E, rows, 640, 392, dt)


@pytest.mark.parametrize("rows,i,o", [(1, 4096, 14336), (3, 14336, 4096), (16, 4096, 1024), (60, 4096, 4096),
                                      (513, 4096, 1024), (130, 14336, 1024), (1, 40000, 100), (2, 64, 32768)])
def test_full_sizes(E, rows, i, o):
    check(E, rows, i, o, "f16")


def test_wide_prompt(E):
    check(E, 2048, 1024, 4096, "bf16")


@pytest.mark.parametrize("rows", [1, 20, 150])
def test_strides(E, rows):
    wq, ws, q, s = operands(rows, 272, 200)
    m = E.Fp8Matrix(wq, ws)
    ref = m.matmul(q, s, out_dtype=torch.float32)
    q2 = torch.full((rows, 512), 0x7F, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
    q2[:, 16:288] = q
    s2 = torch.full((rows, 9), float("nan"), device="cuda")
    s2[:, 2:5] = s
    out = torch.full((rows + 3, 203), 7.0, device="cuda")
    m.matmul(q2[:, 16:288], s2[:, 2:5], out=out[:rows, 1:201])
    assert torch.equal(out[:rows, 1:201], ref)
    assert bool((out[rows:] == 7).all() and (out[:, 0] == 7).all() and (out[:, 201:] == 7).all())


@pytest.mark.parametrize("rows", [1, 9, 40, 300])
def test_nonfinite_rows_stay_their_own(E, rows):
    wq, ws, q, s = operands(rows + 2, 400, 264)
    m = E.Fp8Matrix(wq, ws)
    ref = m.matmul(q, s, out_dtype=torch.float32)
    q.view(torch.uint8)[0, 7] = 0x7F
    s[1, 2] = float("inf")
    out = m.matmul(q, s, out_dtype=torch.float32)
    assert torch.isnan(out[0]).all() and not torch.isfinite(out[1]).any()
    assert torch.equal(out[2:], ref[2:])


def test_zero_scales_and_signed_zero(E):
    wq, ws, q, s = operands(5, 256, 256)
    s[:, 1] = 0
    ws[0, 1] = 0
    m = E.Fp8Matrix(wq, ws)
    ref, tol = R.product(q, s, wq, ws)
    R.assert_close(m.matmul(q, s, out_dtype=torch.float32), ref, tol)


@pytest.mark.parametrize("rows", [1, 40, 300])
def test_every_e4m3_value(E, rows):
    """All 254 finite bytes on both sides, subnormals among them."""
    b = torch.arange(256, device="cuda", dtype=torch.int32)
    b = b[(b & 0x7F) != 0x7F].to(torch.uint8)
    wq = b[(torch.arange(254, device="cuda")[:, None] * 3 + torch.arange(96, device="cuda")[None] * 7) % 254]
    wq = wq.contiguous().view(torch.float8_e4m3fn)
    q = torch.zeros(rows, 256, device="cuda", dtype=torch.uint8)
    q[:, :254] = b[(torch.arange(254, device="cuda")[None] + 5 * torch.arange(rows, device="cuda")[:, None]) % 254]
    q = q.view(torch.float8_e4m3fn)[:, :254]
    s = torch.rand(rows, 2, device="cuda", generator=gen(1)) + 0.5
    ws = torch.rand(2, 1, device="cuda", generator=gen(2)) - 0.5
    ref, tol = R.product(q, s, wq, ws)
    R.assert_close(E.Fp8Matrix(wq, ws).matmul(q, s, out_dtype=torch.float32), ref, tol)


def test_one_nonzero_entry(E):
    """A single product lands at its place, for places all over the tiles."""
    i, o = 300, 270
    for r, k, n in [(0, 0, 0), (5, 127, 127), (8, 128, 128), (37, 299, 269), (16, 200, 255), (31, 17, 256)]:
        wq = torch.zeros(i, o, device="cuda").to(torch.float8_e4m3fn)
        wq.view(torch.uint8)[k, n] = 0x38  # 1.0
        q = torch.zeros(38, 304, device="cuda", dtype=torch.uint8)
        q[r, k] = 0xC0  # -2.0
        ws = torch.full((3, 3), 0.5, device="cuda")
        s = torch.full((38, 3), 3.0, device="cuda")
        out = E.Fp8Matrix(wq, ws).matmul(q.view(torch.float8_e4m3fn)[:, :i], s, out_dtype=torch.float32)
        want = torch.zeros(38, o, device="cuda")
        want[r, n] = -3.0
        assert torch.equal(out, want), (r, k, n)


def test_streams_and_graphs(E):
    """One matrix on two streams at once and in two graphs replayed side by side."""
    wq, ws, q, s = operands(24, 4096, 1024)
    m = E.Fp8Matrix(wq, ws)
    sets = [(q, s)] + [operands(24, 4096, 1024, 10 * k)[2:] for k in (1, 2, 3)]
    ref = [m.matmul(a, b) for a, b in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [None] * 4
    torch.cuda.synchronize()
    for _ in range(3):
        for k, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[k] = m.matmul(*sets[k])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    graphs = []
    for a, b in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = m.matmul(a, b)
        graphs.append((g, o))
    for k, (g, _) in enumerate(graphs):
        with torch.cuda.stream(streams[k]):
            for _ in range(5):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for (_, o), r in zip(graphs, ref))


def test_no_rows(E):
    wq, ws, _, _ = operands(1, 128, 64)
    out = E.Fp8Matrix(wq, ws).matmul(torch.empty(0, 128, device="cuda").to(torch.float8_e4m3fn),
                                     torch.empty(0, 1, device="cuda"))
    assert out.shape == (0, 64)


def test_nonfinite_weights_are_refused(E):
    wq, ws, _, _ = operands(1, 128, 64)
    bad = wq.clone()
    bad.view(torch.uint8)[3, 5] = 0xFF
    with pytest.raises(E.EffortError) as e:
        E.Fp8Matrix(bad, ws)
    assert e.value.status == 4
    with pytest.raises(E.EffortError) as e:
        E.Fp8Matrix(wq, ws * float("inf"))
    assert e.value.status == 4


def test_binding_refuses(E):
    wq, ws, q, s = operands(4, 128, 64)
    m = E.Fp8Matrix(wq, ws)
    assert m.info()["in_dim"] == 128 and m.info()["out_dim"] == 64
    with pytest.raises(ValueError):
        m.matmul(q[:, :127], s)
    with pytest.raises(ValueError):
        m.matmul(q, s[:3])
    with pytest.raises(TypeError):
        m.matmul(q.view(torch.uint8), s)
    with pytest.raises(TypeError):
        m.matmul(q, s, out_dtype=torch.float64)
    with pytest.raises(E.EffortError):  # rows that start off the 16-byte boundaries
        m.matmul(torch.zeros(4, 136, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)[:, :128], s)
    with pytest.raises(E.EffortError):
        m.matmul(torch.zeros(4, 160, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)[:, 8:136], s)
    with pytest.raises(ValueError):
        E.Fp8Matrix(wq, ws[:, :0])


def test_norm_into_product(E):
    """The norm's quantised output is the product's input, odd widths too."""
    for rows, i, o in [(1, 4096, 1024), (33, 1000, 500), (200, 777, 300)]:
        wq, ws, _, _ = operands(1, i, o)
        m = E.Fp8Matrix(wq, ws)
        x = torch.randn(rows, i, device="cuda", generator=gen(3)).bfloat16()
        r = E.block_norm(x, x, post="rms", pre="rms", quantize=True)
        ref, tol = R.product(r.q, r.scales, wq, ws)
        R.assert_close(m.matmul(r.q, r.scales), ref, tol)
