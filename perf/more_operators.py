"""Cases of the operators that serve a mixture of experts with any top-k: the
routing of tokens to experts (softmax or sigmoid scores, a bias for balance,
groups, renormalised weights) with its gradient, the experts' products in
8-bit integers with a scale for each token and channel, and the weighted
combine of each token's expert rows.

Where ``own`` is false ``run`` computes them with elementary torch operations
in 32 bits (the routing's choice in 64, so that close scores are told apart);
where it is true it calls the package.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_SCALE = 2.5  # of the routing weights


def listed():
    return [
        # a decoding batch over many experts in groups: latency of the choice
        dict(name="route 32x256 groups", op="route", tokens=32, experts=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renorm=True, masked=False),
        # the benchmark's step routed by a balance bias, sequences padded at their ends
        dict(name="route 131072x64 bias", op="route", tokens=131072, experts=64, k=6, score="sigmoid", bias=True, groups=1,
             top_groups=1, renorm=True, masked=True),
        # an odd, short batch over few experts, probabilities as they are
        dict(name="route grad 999x5", op="route_grad", tokens=999, experts=5, k=2, score="softmax", renorm=False, masked=True,
             add=False),
        # the benchmark's step: the routing's part added to that of the balance loss
        dict(name="route grad 131072x64", op="route_grad", tokens=131072, experts=64, k=6, score="sigmoid", renorm=True,
             masked=True, add=True),
        # one token being served: the first product of its eight experts
        dict(name="product 1x8 1024-4096", op="product", tokens=1, k=8, experts=64, d=1024, n=4096, second=False, gelu=True,
             dtype="bf16", masked=False),
        # a decoding batch: the second product of its experts, rows back in token order
        dict(name="product 48x8 4096-1024", op="product", tokens=48, k=8, experts=64, d=4096, n=1024, second=True, gelu=False,
             dtype="bf16", masked=False),
        # one matrix for every row: a pipeline stage of the benchmark
        dict(name="product 2048 1024-1024", op="product", tokens=2048, k=1, experts=1, d=1024, n=1024, second=False, gelu=True,
             dtype="bf16", masked=False),
        # odd sizes in fp32, padding left out
        dict(name="product 999x3 1000-515 f32", op="product", tokens=999, k=3, experts=5, d=1000, n=515, second=False,
             gelu=False, dtype="f32", masked=True),
        # the benchmark's step: both products of its experts
        dict(name="product 131072x2 1024-4096", op="product", tokens=131072, k=2, experts=64, d=1024, n=4096, second=False,
             gelu=True, dtype="bf16", masked=False),
        dict(name="product 131072x2 4096-1024", op="product", tokens=131072, k=2, experts=64, d=4096, n=1024, second=True,
             gelu=False, dtype="bf16", masked=True),
        # a decoding batch, a shared expert's rows added
        dict(name="combine 48x8x1024", op="combine", tokens=48, k=8, d=1024, dtype="bf16", masked=False, add=True),
        # the benchmark's step with more experts a token
        dict(name="combine 131072x6x1024", op="combine", tokens=131072, k=6, d=1024, dtype="bf16", masked=True, add=True),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "product", "product", "combine"])
    if op in ("route", "route_grad"):
        experts = _between(rng, 2, 256)
        tokens = _between(rng, 1, 131072 * 64 // max(64, experts))
        k = min(experts, rng.choice([1, 2, 4, 6, 8]))
        case = dict(op=op, tokens=tokens, experts=experts, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    renorm=k > 1 and rng.random() < 0.7, masked=rng.random() < 0.5)
        if op == "route_grad":
            return dict(case, add=rng.random() < 0.5)
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0])
        least = -(-k // (experts // groups))  # groups that hold k experts
        return dict(case, bias=rng.random() < 0.6, groups=groups, top_groups=rng.randint(least, groups))
    if op == "combine":
        k, d = rng.randint(1, 8), rng.choice([8 * _between(rng, 2, 512), _between(rng, 16, 4096)])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        tokens = _between(rng, 1, min(131072, (1 << (29 if dtype == "bf16" else 28)) // (k * d)))
        return dict(op=op, tokens=tokens, k=k, d=d, dtype=dtype, masked=rng.random() < 0.5, add=rng.random() < 0.5)
    experts = rng.choice([1, _between(rng, 2, 64)])
    k = 1 if experts == 1 else min(experts, rng.choice([1, 2, 4, 8]))
    d, n = (rng.choice([64 * rng.randint(1, 64), _between(rng, 16, 4096)]) for _ in range(2))
    tokens = _between(rng, 1, min(131072, (1 << 29) // (k * max(d, n)), (1 << 39) // (k * d * n)))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    return dict(op=op, tokens=tokens, k=k, experts=experts, d=d, n=n, second=experts > 1 and rng.random() < 0.5,
                gelu=rng.random() < 0.5, dtype=dtype, masked=experts > 1 and rng.random() < 0.5)


def _codes(x):
    """Rows as whole numbers in [-127, 127] times a scale, all in 32 bits: the
    row's largest magnitude over 127, and the nearest whole number (ties to
    even) to the quotient as it is rounded to 32 bits."""
    x = x.float()
    scale = x.abs().amax(dim=-1, keepdim=True) / 127.0
    some = scale > 0
    q = torch.round(x / torch.where(some, scale, torch.ones_like(scale)))
    return torch.where(some, q, torch.zeros_like(q)).clamp(-127.0, 127.0), scale


def _padded(d):
    """Bytes of a row of codes: whole steps of the matrix instructions, zeros behind its d."""
    return (d + 63) // 64 * 64


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dev, T, k = case["op"], "cuda", case["tokens"], case["k"]

    def randn(*shape, dtype=torch.float32, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale + mean).to(dtype)

    s = {"case": case}
    valid = torch.ones(T, dtype=torch.bool, device=dev)
    if case["masked"]:
        valid = torch.rand(T, generator=gen, device=dev) < 0.9
    if op in ("route", "route_grad"):
        E = case["experts"]
        s["logits"] = randn(T, E, scale=1.2) + torch.linspace(0.7, -0.7, E, device=dev)
        s["valid"] = valid if case["masked"] else None
        if op == "route":
            s["bias"] = randn(E, scale=0.05) if case["bias"] else None
        else:
            s["experts"] = s["logits"].topk(k, dim=1).indices.to(torch.int32)
            s["experts"][~valid] = E  # no expert, as the routing leaves padding
            s["dweights"] = randn(T, k, scale=1e-2)
            s["add"] = randn(T, E, scale=1e-3) if case["add"] else None
    elif op == "product":
        E, d, n, dt = case["experts"], case["d"], case["n"], _DT[case["dtype"]]
        rows = T * k
        q, scale = _codes(randn(E, n, d, scale=d ** -0.5))
        s["w"] = torch.zeros(E, n, _padded(d), dtype=torch.int8, device=dev)
        s["w"][:, :, :d] = q.to(torch.int8)
        s["w_scale"] = scale.squeeze(-1).contiguous()
        s["offsets"] = s["src_index"] = None
        s["most"] = rows
        if E > 1:
            logits = randn(T, E, scale=1.2) + torch.linspace(0.7, -0.7, E, device=dev)
            experts = logits.topk(k, dim=1).indices
            experts[~valid] = E
            dest = experts.reshape(-1)
            counts = torch.bincount(dest, minlength=E + 1)[:E]
            s["offsets"] = torch.zeros(E + 1, dtype=torch.int64, device=dev)
            s["offsets"][1:] = counts.cumsum(0)
            s["src_index"] = torch.argsort(dest, stable=True).to(torch.int32)
            s["most"] = int(counts.max())
        s["x"] = randn(rows if case["second"] else T, d, dtype=dt)
        s["out"] = torch.zeros(rows, n, dtype=dt, device=dev)
    else:
        d, dt = case["d"], _DT[case["dtype"]]
        s["y"] = randn(T * k, d, dtype=dt)
        s["weights"] = torch.softmax(randn(T, k), dim=1) * _SCALE
        s["weights"][~valid] = 0.0  # no expert
        s["add"] = randn(T, d, dtype=dt) if case["add"] else None
    s["handle"] = _handle(case, s) if own else None
    return s


def _handle(case, s):
    """What a program keeps between its calls: the operator with its output buffers and workspace."""
    import sparse_shard_exchange_amd as pw
    if case["op"] == "route":
        return pw.Router(case["tokens"], case["experts"], case["k"], score=case["score"], groups=case["groups"],
                         top_groups=case["top_groups"], renorm=case["renorm"], scale=_SCALE)
    if case["op"] == "route_grad":
        return pw.Router(case["tokens"], case["experts"], case["k"], score=case["score"], renorm=case["renorm"], scale=_SCALE)
    dtype = pw.PW_BF16 if case["dtype"] == "bf16" else pw.PW_F32
    if case["op"] == "combine":
        return pw.TopkCombine(case["tokens"], case["d"], case["k"], dtype=dtype)
    gather = case["k"] if case["experts"] > 1 and not case["second"] else 0
    return pw.Int8Product(s["w"], s["w_scale"], case["d"], s["out"].shape[0], gather=gather, scatter=case["second"],
                          gelu=case["gelu"], dtype=dtype)


def run(state):
    if own:
        return _call(state)
    op = state["case"]["op"]
    if op == "route":
        return _route(state)
    if op == "route_grad":
        return _route_grad(state)
    if op == "product":
        return _product(state)
    return _combine(state)


def _call(s):
    op, f = s["case"]["op"], s["handle"]
    if op == "route":
        experts, weights = f.forward(s["logits"], bias=s["bias"], valid=s["valid"])
        return {"experts": experts, "weights": weights}
    if op == "route_grad":
        return {"dlogits": f.grad(s["logits"], s["experts"], s["dweights"], valid=s["valid"], add=s["add"])}
    if op == "product":
        return {"out": f.forward(s["x"], offsets=s["offsets"], src_index=s["src_index"], out=s["out"])}
    return {"out": f.forward(s["y"], s["weights"], add=s["add"])}


# ---- plain forms ---------------------------------------------------------------


def _scores(logits, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-logits))
    z = torch.exp(logits - logits.amax(dim=1, keepdim=True))
    return z / z.sum(dim=1, keepdim=True)


def _best(v, k):
    """Indices of the k highest values of each row, best first, ties to the lowest index."""
    return torch.argsort(v, dim=1, descending=True, stable=True)[:, :k]


def _choose(case, s, p):
    """The experts: by the scores p [T][E] in 64 bits, with the bias, inside the best groups."""
    T, E, G = case["tokens"], case["experts"], case["groups"]
    c = p if s["bias"] is None else p + s["bias"].double()
    if case["top_groups"] < G:
        two = torch.sort(c.view(T, G, E // G), dim=2, descending=True).values[:, :, :2].sum(dim=2)
        kept = torch.zeros(T, G, dtype=torch.bool, device=c.device)
        kept.scatter_(1, _best(two, case["top_groups"]), True)
        c = torch.where(kept.unsqueeze(2).expand(T, G, E // G).reshape(T, E), c, torch.full_like(c, -math.inf))
    return _best(c, case["k"])


def _route(s):
    case = s["case"]
    p = _scores(s["logits"].double(), case["score"])
    idx = _choose(case, s, p)
    w = torch.gather(p, 1, idx).float()
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    w, idx = w * _SCALE, idx.to(torch.int32)
    if s["valid"] is not None:
        w = torch.where(s["valid"].unsqueeze(1), w, torch.zeros_like(w))
        idx = torch.where(s["valid"].unsqueeze(1), idx, torch.full_like(idx, case["experts"]))
    return {"experts": idx, "weights": w}


def _route_grad(s):
    case = s["case"]
    E = case["experts"]
    live = s["experts"] < E
    idx = s["experts"].long().clamp(max=E - 1)
    p = _scores(s["logits"].float(), case["score"])
    chosen = torch.gather(p, 1, idx)
    g = torch.where(live, s["dweights"], torch.zeros_like(s["dweights"])) * _SCALE
    if case["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        g = (g - (g * chosen).sum(dim=1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_add_(1, idx, torch.where(live, g, torch.zeros_like(g)))
    d = dp * p * (1.0 - p) if case["score"] == "sigmoid" else p * (dp - (dp * p).sum(dim=1, keepdim=True))
    if s["add"] is not None:
        d = d + s["add"]
    if s["valid"] is not None:
        d = torch.where(s["valid"].unsqueeze(1), d, torch.zeros_like(d))
    return {"dlogits": d}


def _gelu(z):
    return z * 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5))


def _product(s):
    case = s["case"]
    E, n, d, rows = case["experts"], case["n"], case["d"], s["out"].shape[0]
    q, scale = _codes(s["x"])
    w = s["w"][:, :, :d].float().transpose(1, 2).contiguous()
    if E == 1:
        z = (q @ w[0]) * scale * s["w_scale"]
        return {"out": (_gelu(z) if case["gelu"] else z).to(s["out"].dtype)}
    # every segment padded to the longest, one batched product
    offsets, src = s["offsets"], s["src_index"].long()
    at = (offsets[:-1].unsqueeze(1) + torch.arange(s["most"], device=q.device)).clamp(max=rows - 1)
    if not case["second"]:
        at = src[at] // case["k"]
    z = torch.bmm(q[at], w) * scale[at] * s["w_scale"].unsqueeze(1)
    if case["gelu"]:
        z = _gelu(z)
    row = torch.arange(rows, device=q.device)
    e = torch.searchsorted(offsets, row, right=True) - 1
    kept = e < E
    place = e.clamp(max=E - 1) * s["most"] + torch.where(kept, row - offsets[e], torch.zeros_like(row))
    out = torch.where(kept.unsqueeze(1), z.view(-1, n)[place], torch.zeros((), device=q.device)).to(s["out"].dtype)
    if case["second"]:
        out = torch.empty_like(out).index_copy_(0, src, out)  # rows of padding are the zeros that the buffer had
    return {"out": out}


def _combine(s):
    T, k, d = s["case"]["tokens"], s["case"]["k"], s["case"]["d"]
    out = (s["y"].view(T, k, d).float() * s["weights"].unsqueeze(2)).sum(dim=1)
    if s["add"] is not None:
        out = out + s["add"].float()
    return {"out": out.to(s["y"].dtype)}


# ---- what one pass cannot do without -------------------------------------------


def work(case):
    op, T, k = case["op"], case["tokens"], case["k"]
    if op == "route":
        E = case["experts"]
        return {"bytes": 4 * T * E + 8 * T * k + (T if case["masked"] else 0) + (4 * E if case["bias"] else 0),
                "flops": 8 * T * E}
    if op == "route_grad":
        E = case["experts"]
        # a renormalised or sigmoid weight depends on the chosen logits alone
        read = k if case["renorm"] or case["score"] == "sigmoid" else E
        return {"bytes": 4 * T * (E + read + (E if case["add"] else 0)) + 8 * T * k + (T if case["masked"] else 0),
                "flops": 10 * T * k + 2 * T * E}
    size = 2 if case["dtype"] == "bf16" else 4
    if op == "combine":
        return {"bytes": size * T * case["d"] * (k + 1 + (1 if case["add"] else 0)) + 4 * T * k, "flops": 2 * T * k * case["d"]}
    E, d, n, rows = case["experts"], case["d"], case["n"], T * k
    used = min(E, rows)  # experts that have a row, at most
    x_rows = rows if case["second"] else T
    return {"bytes": size * (x_rows * d + rows * n) + used * n * (d + 4) + (4 * rows + 8 * (E + 1) if E > 1 else 0),
            "flops": 2 * rows * d * n}


# ---- the definitions in 64 bits ------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "route_grad": _exact_route_grad, "product": _exact_product,
            "combine": _exact_combine}[case["op"]](case, s)


def _exact_route(case, s):
    """The weights of the k best of a search one after the other."""
    T, E, k, G = case["tokens"], case["experts"], case["k"], case["groups"]
    l = s["logits"].double()
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)
    c = p.clone() if s["bias"] is None else p + s["bias"].double()
    rows = torch.arange(T, device="cuda")
    if case["top_groups"] < G:
        part = c.view(T, G, E // G)
        mark = part.topk(min(2, E // G), dim=2).values.sum(2)
        rest = mark.clone()
        keep = torch.zeros_like(mark, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            g = rest.argmax(dim=1)
            keep[rows, g] = True
            rest[rows, g] = -math.inf
        part[~keep] = -math.inf
    weights = torch.empty(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        e = c.argmax(dim=1)
        weights[:, j] = p[rows, e]
        c[rows, e] = -math.inf
    if case["renorm"]:
        weights /= weights.sum(1, keepdim=True)
    weights *= _SCALE
    if s["valid"] is not None:
        weights[~s["valid"]] = 0.0
    return {"experts": None, "weights": weights}


def _exact_route_grad(case, s):
    """The gradient by differentiating the weights in 64 bits."""
    E, T = case["experts"], case["tokens"]
    valid = torch.ones(T, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"]
    out = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    if bool(valid.any()):
        l = s["logits"][valid].double().requires_grad_(True)
        with torch.enable_grad():
            p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)
            w = torch.gather(p, 1, s["experts"][valid].long())
            if case["renorm"]:
                w = w / w.sum(dim=1, keepdim=True)
            (out[valid],) = torch.autograd.grad((w * _SCALE * s["dweights"][valid].double()).sum(), l)
        if s["add"] is not None:
            out[valid] += s["add"][valid].double()
    return {"dlogits": out}


def _exact_product(case, s):
    E, n, d = case["experts"], case["n"], case["d"]
    rows = s["out"].shape[0]
    out = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    bounds = [0, rows] if E == 1 else s["offsets"].tolist()
    for e in range(E):
        w = s["w"][e, :, :d].double() * s["w_scale"][e].double().unsqueeze(1)
        w = w.T.contiguous()
        for lo in range(bounds[e], bounds[e + 1], 32768):
            hi = min(lo + 32768, bounds[e + 1])
            i = torch.arange(lo, hi, device="cuda")
            g = i if E == 1 else s["src_index"][lo:hi].long()
            x = s["x"][i if E == 1 or case["second"] else g // case["k"]].float()
            scale = x.abs().amax(dim=1, keepdim=True) / 127.0
            # the quotient's rounding to 32 bits is part of the definition
            q = torch.round((x.double() / scale.double()).float()).double()
            z = torch.matmul(q, w) * scale.double()
            if case["gelu"]:
                z = torch.special.ndtr(z) * z
            out[g if case["second"] else i] = z
    return {"out": out}


def _exact_combine(case, s):
    T, k, d = case["tokens"], case["k"], case["d"]
    out = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    for lo in range(0, T, 16384):
        y = s["y"].view(T, k, d)[lo:lo + 16384].double()
        for j in range(k):
            out[lo:lo + 16384] += s["weights"][lo:lo + 16384, j:j + 1].double() * y[:, j]
        if s["add"] is not None:
            out[lo:lo + 16384] += s["add"][lo:lo + 16384].double()
    return {"out": out}
