"""The feed-forward operators in 64 bits, with the error that 32-bit sums and
one rounding may add, for the GPU tests."""
import torch

BLOCK = 128
U32 = 2.0 ** -24  # half a step of fp32, relative
HALF_STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def blocks(n):
    return -(-n // BLOCK)


def quantise_weights(w):
    """(e4m3 q, fp32 scales) of w [..., in, out], one scale per 128 x 128 block."""
    i, o = w.shape[-2:]
    pad = torch.nn.functional.pad(w.float(), (0, blocks(o) * BLOCK - o, 0, blocks(i) * BLOCK - i))
    b = pad.reshape(*w.shape[:-2], blocks(i), BLOCK, blocks(o), BLOCK)
    s = b.abs().amax(dim=(-3, -1)) / 448.0
    d = torch.where(s == 0, torch.ones_like(s), s)
    q = (b / d[..., :, None, :, None]).reshape(pad.shape)[..., :i, :o]
    return q.contiguous().to(torch.float8_e4m3fn), s


def dequantise_weights(q, s):
    i, o = q.shape[-2:]
    w = q.double()
    return w * s.double().repeat_interleave(BLOCK, -2)[..., :i, :].repeat_interleave(BLOCK, -1)[..., :o]


def dequantise_rows(q, s):
    return q.double() * s.double().repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


def assert_close(got, ref, tol, what=""):
    """|got - ref| <= tol element by element, plus the rounding of got's type."""
    ref = ref.to(got.device)
    bound = tol.to(got.device) * (1 + HALF_STEP[got.dtype]) + ref.abs() * HALF_STEP[got.dtype] + TINY[got.dtype]
    d = (got.double() - ref).abs()
    assert bool(torch.isfinite(got).all()), what
    worst = float((d / bound).max()) if d.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3g} of the bound"


# -- the block norm ----------------------------------------------------------
# A sum of n fp32 terms in any grouping is off by at most (n - 1) U32 times the
# sum of magnitudes; the kernel's groupings have at most n / 32 + 32 additions
# in a row, which DEPTH counts.  A norm multiplies by r = (mean v^2 + eps)^-1/2,
# off by half the relative error of the mean plus two roundings (and 2 ulp of
# the approximate root); three more roundings apply weight, offset and bias.

def depth(n):
    return n / 32 + 32


def norm(v, dv, kind, w, b, off, eps):
    """(value, error) of a norm of v that is itself off by dv."""
    n = v.shape[1]
    if kind is None:
        return v, dv
    if kind == "layer":
        mean = v.mean(1, keepdim=True)
        dmean = dv.mean(1, keepdim=True) + depth(n) * U32 * v.abs().mean(1, keepdim=True)
        c = v - mean
        dc = dv + dmean + U32 * c.abs()
    else:
        c, dc = v, dv
    ms = (c * c).mean(1, keepdim=True)
    dms = (2 * c.abs() * dc + dc * dc).mean(1, keepdim=True) + (depth(n) + 3) * U32 * ms
    r = (ms + eps) ** -0.5
    # (ms + eps) may fall to nothing when a row is constant: the error of r is then bounded by its largest value
    low = torch.clamp(ms - dms, min=0.0) + eps
    dr = torch.where(low > 0, low, ms + eps) ** -0.5 - r + 6 * U32 * r
    scale = torch.ones(n, dtype=v.dtype, device=v.device) if w is None else off + w.double()
    out = c * r * scale
    mag = scale.abs() + (0 if w is None else abs(off) + w.double().abs()) * U32 * 2
    dout = (dc * (r + dr) + c.abs() * dr) * mag + 4 * U32 * out.abs()
    if b is not None:
        out = out + b.double()
        dout = dout + U32 * (out.abs() + dout)
    return out, dout


def block_norm(x, y, post, pre, gate, a, bs, pw, pb, w, b, off, eps):
    """(x', error), (h, error) in 64 bits."""
    x64 = x.double()
    if y is not None:
        u, du = norm(y.double(), torch.zeros_like(x64), post, pw, pb, off, eps)
        g = torch.ones_like(u) if gate is None else gate.double().expand_as(u)
        v = a * x64 + bs * g * u
        mag = abs(a) * x64.abs() + abs(bs) * (g * u).abs()
        dv = abs(bs) * g.abs() * du + 4 * U32 * mag
    else:
        v = a * x64
        dv = 2 * U32 * v.abs()
    h, dh = norm(v, dv, pre, w, b, off, eps)
    return (v, dv), (h, dh)


def check_quantised(q, scales, h, dh, what=""):
    """q and scales of h [rows, n] that is known to within dh.  The scale is max|h| / 448
    (the maximum off by at most the largest dh of the block, one rounding); q is
    within half a step of h / scale: 2^-4 relative, 2^-10 absolute below 2^-6."""
    m, n = h.shape
    pad = (0, blocks(n) * BLOCK - n)
    amax = torch.nn.functional.pad(h.abs(), pad).reshape(m, -1, BLOCK).amax(2)
    dmax = torch.nn.functional.pad(dh, pad).reshape(m, -1, BLOCK).amax(2)
    ref = amax / 448.0
    assert_close(scales, ref, dmax / 448.0 + U32 * ref, what + " scales")
    s = scales.double().repeat_interleave(BLOCK, 1)[:, :n]
    live = s > 0
    t = torch.where(live, h / torch.where(live, s, torch.ones_like(s)), torch.zeros_like(h))
    dt = torch.where(live, dh / torch.where(live, s, torch.ones_like(s)), torch.zeros_like(h)) + 2 * U32 * t.abs()
    step = torch.clamp(t.abs() * 2.0 ** -4, min=2.0 ** -10)
    worst = float(((q.double() - t).abs() / (step + dt * 1.1)).max())
    assert worst <= 1.0, f"{what} q: {worst:.3g} of the bound"
    assert bool((q.double()[~live] == 0).all())


# -- the product -------------------------------------------------------------
# Products of e4m3 values are exact.  A sum is off by at most one fp32 step
# (2 U32: the tensor core may truncate) of the sum of magnitudes for each
# addition in a row: K / 16 of matrix steps at most, K / 128 of scaled blocks,
# and 64 for the joins of splits and the scales' own products.

def product(q, s, wq, ws):
    x, w = dequantise_rows(q, s), dequantise_weights(wq, ws)
    k = x.shape[1]
    return x @ w, (x.abs() @ w.abs()) * (2 * U32) * (k / 16 + k / 128 + 64)


# -- mixture of experts ------------------------------------------------------

#: bits with which the hidden activations enter the second product, by out's type
HIDDEN = {torch.float32: 2.0 ** -21, torch.float16: 2.0 ** -16, torch.bfloat16: 2.0 ** -11}


def moe(x, w1, w3, w2, ids, gates, out_dtype):
    """(out, error) in 64 bits; w1, w3, w2 in double [E, ...]; ids outside 0..E-1 add nothing."""
    e, i, f = w1.shape
    x64 = x.double()
    # x itself enters in at least 22 bits, values below 2^-36 of a block's largest as nothing.
    # The hidden activations are scaled by a power of two that brings B = |x|^2 |w1| |w3| (the
    # largest column norms of a block; below: of the matrix) to 2^12 or more of binary16's
    # 2^15, so half a step of its subnormals, 2^-25, is at most 2^-37 of B.
    dx = x64.abs() * 2.0 ** -21 + x64.abs().amax(1, keepdim=True) * 2.0 ** -36
    out = torch.zeros(x.shape[0], i, dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(out)

    def steps(k):
        return (2 * U32) * (k / 8 + 64)

    for j in range(e):
        t, slot = (ids == j).nonzero(as_tuple=True)
        if not len(t):
            continue
        xt = x64[t]
        a, b = xt @ w1[j], xt @ w3[j]
        da = xt.abs() @ w1[j].abs() * steps(i) + dx[t] @ w1[j].abs()
        db = xt.abs() @ w3[j].abs() * steps(i) + dx[t] @ w3[j].abs()
        sg = a * torch.sigmoid(a)
        h = sg * b
        dsg = 1.1 * da + 8 * U32 * sg.abs()  # |silu'| < 1.1; exp, sum, quotient
        dh = dsg * (b.abs() + db) + sg.abs() * db + 4 * U32 * h.abs()
        bound = xt.square().sum(1, keepdim=True) * w1[j].norm(dim=0).max() * w3[j].norm(dim=0).max()
        dh = dh + HIDDEN[out_dtype] * (h.abs() + dh) + bound * 2.0 ** -37
        g = gates[t, slot].double()[:, None]
        y = h @ w2[j]
        dy = dh @ w2[j].abs() + (h.abs() + dh) @ w2[j].abs() * steps(f)
        out.index_put_((t,), g * y, accumulate=True)
        tol.index_put_((t,), g.abs() * (dy + 32 * U32 * y.abs()), accumulate=True)
    return out, tol


def route(x, router, k):
    """(ids, softmax over the chosen, chosen of the softmax over all) in 64 bits, ties to the lower expert."""
    l = x.double() @ router.double().T
    best, ids = torch.sort(l, dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    return ids.to(torch.int32), torch.softmax(best, 1), torch.gather(torch.softmax(l, 1), 1, ids)
