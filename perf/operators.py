"""What is measured of the feed-forward operators: the e4m3 product with a scale
for each block of 128, the norm / gate / residual step around a block, and the
mixture-of-experts layer for a few tokens.

Each operator is written here in its plain form (torch operations in 32 bits),
as a definition in 64 bits (`exact`), and as the call that a user of the
library makes (`own`)."""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def listed():
    return [
        # -- product: rows x in_dim times in_dim x out_dim
        # one token through the smallest projection: latency
        {"name": "product 1x512x512", "op": "product", "rows": 1, "in_dim": 512, "out_dim": 512, "out": "f32"},
        # one decoded token through an FFN up projection
        {"name": "product 1x4096x14336", "op": "product", "rows": 1, "in_dim": 4096, "out_dim": 14336, "out": "f16"},
        # a few requests decoded together through an FFN down projection
        {"name": "product 13x14336x4096", "op": "product", "rows": 13, "in_dim": 14336, "out_dim": 4096, "out": "bf16"},
        # a short prompt, sizes that end inside every tile and block
        {"name": "product 200x4091x1003", "op": "product", "rows": 200, "in_dim": 4091, "out_dim": 1003, "out": "bf16"},
        # a long prompt through an FFN up projection
        {"name": "product 4096x4096x14336", "op": "product", "rows": 4096, "in_dim": 4096, "out_dim": 14336,
         "out": "bf16"},
        # -- norm: rows x dim
        # between two blocks of one decoded token
        {"name": "norm 1x4096", "op": "norm", "rows": 1, "dim": 4096, "kind": "rms", "dtype": "f32", "gate": "none",
         "quant": False},
        # odd width, layer norm with biases, one gate row for all tokens
        {"name": "norm 61x5003", "op": "norm", "rows": 61, "dim": 5003, "kind": "layer", "dtype": "f16",
         "gate": "one", "quant": False},
        # a prompt on its way into an e4m3 product, gated per token
        {"name": "norm 8192x4096 e4m3", "op": "norm", "rows": 8192, "dim": 4096, "kind": "rms", "dtype": "bf16",
         "gate": "row", "quant": True},
        # -- moe: tokens through the top experts of in_dim x hidden
        # one token, experts an eighth of the usual width: latency
        {"name": "moe 1 of 8x512x1792 f16", "op": "moe", "tokens": 1, "experts": 8, "top": 2, "in_dim": 512,
         "hidden": 1792, "weights": "f16", "dtype": "f16"},
        # one decoded token, full width, e4m3 weights
        {"name": "moe 1 of 8x4096x14336 e4m3", "op": "moe", "tokens": 1, "experts": 8, "top": 2, "in_dim": 4096,
         "hidden": 14336, "weights": "e4m3", "dtype": "f32"},
        # sixteen requests decoded together, binary16 weights
        {"name": "moe 16 of 8x4096x14336 f16", "op": "moe", "tokens": 16, "experts": 8, "top": 2, "in_dim": 4096,
         "hidden": 14336, "weights": "f16", "dtype": "f16"},
        # many small experts of odd widths, more tokens than one matrix tile holds
        {"name": "moe 37 of 64x1000x523 bf16", "op": "moe", "tokens": 37, "experts": 64, "top": 6, "in_dim": 1000,
         "hidden": 523, "weights": "bf16", "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "norm", "moe"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    while True:
        if op == "product":
            c = {"op": op, "rows": _log_int(rng, 1, 8192), "in_dim": _log_int(rng, 64, 14336),
                 "out_dim": _log_int(rng, 64, 14336), "out": dtype}
            if c["rows"] * c["in_dim"] * c["out_dim"] <= 4096 * 4096 * 14336:
                return c
        elif op == "norm":
            c = {"op": op, "rows": _log_int(rng, 1, 8192), "dim": _log_int(rng, 64, 16384),
                 "kind": rng.choice(["rms", "layer"]), "dtype": dtype, "gate": rng.choice(["none", "one", "row"]),
                 "quant": rng.random() < 0.5}
            if c["rows"] * c["dim"] <= 8192 * 4096:
                return c
        else:
            c = {"op": op, "tokens": _log_int(rng, 1, 64), "experts": _log_int(rng, 4, 64), "top": rng.randint(1, 4),
                 "in_dim": _log_int(rng, 256, 4096), "hidden": _log_int(rng, 128, 14336),
                 "weights": rng.choice(["e4m3", "f16", "bf16"]), "dtype": dtype}
            if c["experts"] * c["in_dim"] * c["hidden"] <= 8 * 4096 * 14336 // 2:
                return c


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _blocks(n):
    return -(-n // BLOCK)


def _quantise_weights(w):
    """e4m3 values and one scale per 128 x 128 block of w [..., in, out]."""
    i, o = w.shape[-2:]
    pad = torch.nn.functional.pad(w, (0, _blocks(o) * BLOCK - o, 0, _blocks(i) * BLOCK - i))
    b = pad.reshape(*w.shape[:-2], _blocks(i), BLOCK, _blocks(o), BLOCK)
    s = b.abs().amax(dim=(-3, -1)) / E4M3_MAX
    q = (b / s[..., :, None, :, None]).reshape(pad.shape)[..., :i, :o]
    return q.contiguous().to(torch.float8_e4m3fn), s


def _quantise_rows(x):
    """e4m3 values (rows a multiple of 16 bytes apart) and one scale per row and 128 columns."""
    m, i = x.shape
    pad = torch.nn.functional.pad(x, (0, _blocks(i) * BLOCK - i)).reshape(m, _blocks(i), BLOCK)
    s = pad.abs().amax(dim=-1) / E4M3_MAX
    q = torch.zeros(m, -(-i // 16) * 16, device=x.device, dtype=torch.float8_e4m3fn)
    q[:, :i] = (pad / s[..., None]).reshape(m, -1)[:, :i].to(torch.float8_e4m3fn)
    return q[:, :i], s


def _activations(g, m, n):
    """Unit normal with a heavy tail in a few channels, as activations have it."""
    heavy = 1.0 + 9.0 * (torch.rand(n, generator=g, device="cuda") < 0.01)
    return _randn(g, m, n) * heavy


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "product":
        st["wq"], st["ws"] = _quantise_weights(_randn(g, case["in_dim"], case["out_dim"]) * 0.02)
        st["xq"], st["xs"] = _quantise_rows(_activations(g, case["rows"], case["in_dim"]))
        if own:
            import dynamic_approximate_gemv_b200 as E
            st["matrix"] = E.Fp8Matrix(st["wq"], st["ws"])
    elif case["op"] == "norm":
        m, n, t = case["rows"], case["dim"], DTYPES[case["dtype"]]
        st["x"] = (4.0 * _activations(g, m, n)).to(t)
        st["y"] = (0.5 * _activations(g, m, n) + 0.1).to(t)
        st["gate"] = {"none": None, "one": torch.tanh(_randn(g, 1, n)).to(t),
                      "row": torch.tanh(_randn(g, m, n)).to(t)}[case["gate"]]
        st["post_weight"] = (1.0 + 0.1 * _randn(g, n)).to(t)
        st["pre_weight"] = (1.0 + 0.1 * _randn(g, n)).to(t)
        layer = case["kind"] == "layer"
        st["post_bias"] = (0.1 * _randn(g, n)).to(t) if layer else None
        st["pre_bias"] = (0.1 * _randn(g, n)).to(t) if layer else None
        st["residual_scale"], st["branch_scale"], st["eps"] = 0.75, 1.25, 1e-5
    else:
        e, i, h, t = case["experts"], case["in_dim"], case["hidden"], DTYPES[case["dtype"]]
        st["x"] = _activations(g, case["tokens"], i).to(t)
        st["router"] = (_randn(g, e, i) / 64.0).to(t)
        for name, a, b in (("w1", i, h), ("w3", i, h), ("w2", h, i)):
            if case["weights"] == "e4m3":
                per = [_quantise_weights(_randn(g, a, b) * 0.02) for _ in range(e)]
                st[name] = torch.stack([q.view(torch.uint8) for q, _ in per]).view(torch.float8_e4m3fn)
                st["s" + name[1]] = torch.stack([s for _, s in per])
                del per
            else:
                st[name] = torch.stack([(_randn(g, a, b) * 0.02).to(DTYPES[case["weights"]]) for _ in range(e)])
        if own:
            import dynamic_approximate_gemv_b200 as E
            scales = (st["s1"], st["s3"], st["s2"]) if case["weights"] == "e4m3" else None
            st["layer"] = E.MoeLayer(st["w1"], st["w3"], st["w2"], scales=scales, router=st["router"])
    return st


# ---------------------------------------------------------------- one pass

def _spread_blocks(s, i, o):
    """Scales per 128 x 128 block to one per element of i x o."""
    return s.repeat_interleave(BLOCK, -2)[..., :i, :].repeat_interleave(BLOCK, -1)[..., :o]


def _plain_product(st):
    c = st["case"]
    x = st["xq"].float() * st["xs"].repeat_interleave(BLOCK, 1)[:, : c["in_dim"]]
    w = st["wq"].float() * _spread_blocks(st["ws"], c["in_dim"], c["out_dim"])
    return (x @ w).to(DTYPES[c["out"]])


def _plain_norm_step(v, kind, weight, bias, eps):
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + eps) * weight.float()
    return v if bias is None else v + bias.float()


def _plain_norm(st):
    c = st["case"]
    u = _plain_norm_step(st["y"].float(), c["kind"], st["post_weight"], st["post_bias"], st["eps"])
    if st["gate"] is not None:
        u = u * st["gate"].float()
    x = st["residual_scale"] * st["x"].float() + st["branch_scale"] * u
    h = _plain_norm_step(x, c["kind"], st["pre_weight"], st["pre_bias"], st["eps"])
    t = DTYPES[c["dtype"]]
    if not c["quant"]:
        return {"x": x.to(t), "h": h.to(t)}
    q, s = _quantise_rows(h)
    return {"x": x.to(t), "q": q, "scales": s}


def _plain_moe(st):
    c = st["case"]
    n, e, k, i, h = c["tokens"], c["experts"], c["top"], c["in_dim"], c["hidden"]
    x = st["x"].float()
    # which experts: borders between logits are decided in 64 bits
    logits = st["x"].double() @ st["router"].double().T
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    gates = torch.exp(best - best[:, :1])
    gates = (gates / gates.sum(dim=1, keepdim=True)).float()

    def weights(name, a, b, rows):
        w = st[name][rows].float() if rows is not None else st[name].float()
        if c["weights"] == "e4m3":
            s = st["s" + name[1]]
            w *= _spread_blocks(s[rows] if rows is not None else s, a, b)
        return w

    if n * k <= e:  # few pairs: their experts' weights alone
        pair = ids.reshape(-1)
        xp = x.repeat_interleave(k, 0)[:, None, :]
        a, b = torch.bmm(xp, weights("w1", i, h, pair)), torch.bmm(xp, weights("w3", i, h, pair))
        y = torch.bmm(a / (1 + torch.exp(-a)) * b, weights("w2", h, i, pair))[:, 0, :]
        out = (gates[:, :, None] * y.reshape(n, k, i)).sum(dim=1)
    else:  # every expert on every token, weighted by its gate or by nothing
        xe = x.expand(e, n, i)
        a, b = torch.bmm(xe, weights("w1", i, h, None)), torch.bmm(xe, weights("w3", i, h, None))
        y = torch.bmm(a / (1 + torch.exp(-a)) * b, weights("w2", h, i, None))
        share = torch.zeros(n, e, device=x.device).scatter(1, ids, gates)
        out = (share.T[:, :, None] * y).sum(dim=0)
    return {"out": out.to(DTYPES[c["dtype"]]), "ids": ids.to(torch.int32), "gates": gates}


def run(st):
    c = st["case"]
    if not own:
        return {"product": _plain_product, "norm": _plain_norm, "moe": _plain_moe}[c["op"]](st)
    import dynamic_approximate_gemv_b200 as E
    if c["op"] == "product":
        return st["matrix"].matmul(st["xq"], st["xs"], out_dtype=DTYPES[c["out"]])
    if c["op"] == "norm":
        r = E.block_norm(st["x"], st["y"], post=c["kind"], post_weight=st["post_weight"], post_bias=st["post_bias"],
                         gate=st["gate"], residual_scale=st["residual_scale"], branch_scale=st["branch_scale"],
                         pre=c["kind"], pre_weight=st["pre_weight"], pre_bias=st["pre_bias"], eps=st["eps"],
                         quantize=c["quant"])
        return {"x": r.x, "q": r.q, "scales": r.scales} if c["quant"] else {"x": r.x, "h": r.h}
    out, ids, gates = st["layer"](st["x"], top_k=c["top"])
    return {"out": out, "ids": ids, "gates": gates}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
    if case["op"] == "product":
        m, i, o = case["rows"], case["in_dim"], case["out_dim"]
        return {"bytes": m * i + 4 * m * _blocks(i) + i * o + 4 * _blocks(i) * _blocks(o) + m * o * size[case["out"]],
                "flops": 2 * m * i * o}
    if case["op"] == "norm":
        m, n, z = case["rows"], case["dim"], size[case["dtype"]]
        read = 2 * m * n + {"none": 0, "one": n, "row": m * n}[case["gate"]] + (4 if case["kind"] == "layer" else 2) * n
        wrote = m * n * z + (m * n + 4 * m * _blocks(n) if case["quant"] else m * n * z)
        return {"bytes": read * z + wrote, "flops": 14 * m * n}
    n, e, k, i, h = case["tokens"], case["experts"], case["top"], case["in_dim"], case["hidden"]
    met = e * (1 - (1 - k / e) ** n)  # experts that n tokens meet, on average
    w = size[case["weights"]]
    scales = 3 * 4 * _blocks(i) * _blocks(h) if w == 1 else 0
    z = size[case["dtype"]]
    return {"bytes": met * (3 * i * h * w + scales) + e * i * z + 2 * n * i * z + 8 * n * k,
            "flops": 6 * n * k * i * h + 2 * n * e * i}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_matrix(q, s):
    """sum over blocks, written out: each 128 x 128 block of q times its scale."""
    w = q.double()
    for r in range(s.shape[0]):
        for c in range(s.shape[1]):
            w[r * BLOCK:(r + 1) * BLOCK, c * BLOCK:(c + 1) * BLOCK] *= s[r, c].double()
    return w


def _exact_norm_step(v, kind, weight, bias, eps):
    n = v.shape[1]
    if kind == "layer":
        v = v - v.sum(1)[:, None] / n
    r = 1.0 / torch.sqrt(v.pow(2).sum(1) / n + eps)
    v = v * r[:, None] * weight.double()[None]
    return v + bias.double()[None] if bias is not None else v


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "product":
        x = st["xq"].double()
        for b in range(st["xs"].shape[1]):
            x[:, b * BLOCK:(b + 1) * BLOCK] *= st["xs"][:, b:b + 1].double()
        return x @ _exact_matrix(st["wq"], st["ws"])
    if case["op"] == "norm":
        u = _exact_norm_step(st["y"].double(), case["kind"], st["post_weight"], st["post_bias"], st["eps"])
        if st["gate"] is not None:
            u = u * st["gate"].double()
        x = st["residual_scale"] * st["x"].double() + st["branch_scale"] * u
        h = _exact_norm_step(x, case["kind"], st["pre_weight"], st["pre_bias"], st["eps"])
        if not case["quant"]:
            return {"x": x, "h": h}
        q, s = torch.empty_like(h), torch.empty(h.shape[0], _blocks(h.shape[1]), device=h.device, dtype=h.dtype)
        for b in range(s.shape[1]):
            part = h[:, b * BLOCK:(b + 1) * BLOCK]
            s[:, b] = part.abs().amax(1) / E4M3_MAX
            q[:, b * BLOCK:(b + 1) * BLOCK] = part / s[:, b:b + 1]
        return {"x": x, "q": q, "scales": s}
    n, e, k = case["tokens"], case["experts"], case["top"]
    x = st["x"].double()
    logits = x @ st["router"].double().T
    picked = [sorted(range(e), key=lambda j, row=row: (-row[j], j))[:k] for row in logits.tolist()]
    ids = torch.tensor(picked, device=x.device)
    gates = torch.softmax(torch.gather(logits, 1, ids), dim=1)
    out = torch.zeros(n, case["in_dim"], device=x.device, dtype=torch.float64)
    for j in sorted(set(sum(picked, []))):
        t, slot = (ids == j).nonzero(as_tuple=True)
        if case["weights"] == "e4m3":
            w1, w3, w2 = (_exact_matrix(st["w" + d][j], st["s" + d][j]) for d in "132")
        else:
            w1, w3, w2 = (st["w" + d][j].double() for d in "132")
        a = x[t] @ w1
        out[t] += gates[t, slot][:, None] * ((a * torch.sigmoid(a) * (x[t] @ w3)) @ w2)
    return {"out": out, "ids": ids.to(torch.int32), "gates": gates}
