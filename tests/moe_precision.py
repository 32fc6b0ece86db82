"""The mixture of experts in 64 bits, with an error bound term by term of what the
header of the library promises: how x and the hidden activations enter the
products, what the matrix instructions may lose, and where fp32 sums join.

U = 2^-24, half a step of fp32.

x.  16-bit x enters exactly beside weights of bfloat16, and binary16 x beside
binary16 and e4m3 weights.  Else a K block (64 or 128 inputs) of a token is scaled
by a power of two that brings its largest value M (2^-97 if that is larger) to
2^14 or more: one binary16 part holds bfloat16's 8 bits down to an absolute half
step of 2^-25, which is 2^-39 M; two parts, the second scaled by 2^11 once more,
hold 22 bits (error 2^-23) down to 2^-36 / 2^14 = 2^-50 M.  Three bfloat16
parts hold 24 bits and more (error 2^-26).

Hidden activations.  With binary16 and e4m3 weights likewise, with the bound
B = |x|^2 |w1| |w3| (norms of x and of the largest columns of the K block; 2^-96 if
that is larger) in M's place; a bfloat16 out takes one part, 11 bits (error 2^-11, and 2^-39 B), unless
norms of columns differ by more than 32 times within a K block.  With bfloat16
weights two parts (16-bit out; error 2^-17), or three.

Products.  They are exact.  A matrix instruction adds 16 of them to a sum: it
may drop what lies below 2^-25 of the largest of the 17 addends (16 times) and
round toward zero (2 U), relative to the sum of magnitudes together at most 10 U.
A K block is a chain of KE / 16 instructions a part; its sum meets up to three
roundings (the parts' sums, the scales) and then goes through fp32 additions: a
warp's K blocks (a sixth of them at most), the warps, the shares and the pairs.
"""
import torch

U = 2.0 ** -24


def block_max(v, ke):
    n = v.shape[1]
    pad = torch.nn.functional.pad(v, (0, -n % ke)).reshape(v.shape[0], -1, ke)
    return pad.amax(2).repeat_interleave(ke, 1)[:, :n]


def spread(w, ke):
    """Whether norms of the columns of w [in, hidden] differ by more than 32 times within a K block."""
    n = w.norm(dim=0)[None]
    low = -block_max(-torch.where(n > 0, n, torch.full_like(n, 1e300)), ke)
    return bool((block_max(n, ke) > 32 * low).any())


def moe(x, w1, w3, w2, ids, gates, out_dtype, kind):
    """(out, error) in 64 bits; w1, w3, w2 in double [E, ...], kind: "f16", "bf16" or "e4m3"."""
    e, i, f = w1.shape
    x64, ke, wide = x.double(), 128 if kind == "e4m3" else 64, kind == "bf16"
    top = block_max(x64.abs(), ke).clamp(min=2.0 ** -97)
    f32, same = x.dtype == torch.float32, x.dtype == torch.float16
    if wide:
        dx = x64.abs() * (2.0 ** -26 if f32 else 0.0)
    else:
        dx = x64.abs() * 2.0 ** -23 + top * 2.0 ** -50 if f32 else top * (0.0 if same else 2.0 ** -39)
    parts = {torch.float32: 3, torch.float16: 2, torch.bfloat16: 2}[out_dtype]

    def steps(k):  # relative to the sum of magnitudes; the parts of bfloat16 weights share a chain
        chain = ke / 16 * (3 if wide else 1)
        return 10 * U * chain + U * (k / ke / 6 + 40)

    out = torch.zeros(x.shape[0], i, dtype=torch.float64, device=x.device)
    tol = torch.zeros_like(out)
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
        dsg = 1.1 * da + 8 * U * sg.abs()  # |silu'| < 1.1; exp, sum, quotient
        dh = dsg * (b.abs() + db) + sg.abs() * db + 4 * U * h.abs()
        if wide:
            dh = dh + (h.abs() + dh) * (2.0 ** -26 if parts == 3 else 2.0 ** -17)
        else:
            bound = xt.square().sum(1, keepdim=True) * block_max(w1[j].norm(dim=0)[None], ke) * block_max(w3[j].norm(dim=0)[None], ke)
            few = out_dtype == torch.bfloat16 and not any(spread(w[k], ke) for w in (w1, w3) for k in range(e))
            dh = dh + (h.abs() + dh) * 2.0 ** (-11 if few else -23) + bound.clamp(min=2.0 ** -96) * 2.0 ** (-39 if few else -50)
        g = gates[t, slot].double()[:, None]
        y = h @ w2[j]
        dy = dh @ w2[j].abs() + (h.abs() + dh) @ w2[j].abs() * steps(f)
        out.index_put_((t,), g * y, accumulate=True)
        tol.index_put_((t,), g.abs() * (dy + 32 * U * y.abs()), accumulate=True)
    return out, tol
