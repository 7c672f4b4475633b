"""Cases of the operators around the mixture-of-experts step: the router's
balance loss with per-expert counts and its gradient, the gradients of the
gated combine and of dispatch and router, and the norms around a block with
its gate and residual scale.

Where ``own`` is false ``run`` computes them with elementary torch operations
in 32 bits; where it is true it calls the package.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_BALANCE, _Z = 1e-2, 1e-3
_X_SCALE, _Y_SCALE = 1.0, 0.75


def listed():
    return [
        # one decoding batch: latency of the loss and the counts alone
        dict(name="balance 48x8", op="balance", tokens=48, experts=8, k=2, masked=False),
        # the benchmark's MoE step, sequences padded at their ends
        dict(name="balance 131072x64", op="balance", tokens=131072, experts=64, k=2, masked=True),
        # an odd, short batch over few experts
        dict(name="router grad 999x5", op="router_grad", tokens=999, experts=5, k=2, masked=True),
        # the benchmark's MoE step: loss and gate gradients down to the logits
        dict(name="router grad 131072x64", op="router_grad", tokens=131072, experts=64, k=2, masked=False),
        # few tokens, an expert capacity that drops some
        dict(name="combine grad 300x512", op="combine_grad", tokens=300, d=512, experts=64, capacity=8),
        # the benchmark's MoE step, no capacity
        dict(name="combine grad 131072x1024", op="combine_grad", tokens=131072, d=1024, experts=64, capacity=0),
        # an odd token count, five experts, a capacity
        dict(name="dispatch grad 1000x256", op="dispatch_grad", tokens=1000, d=256, experts=5, capacity=350),
        # the benchmark's MoE step
        dict(name="dispatch grad 131072x1024", op="dispatch_grad", tokens=131072, d=1024, experts=64, capacity=0),
        # one token being served: after one block and before the next
        dict(name="norm 1x1024", op="norm", rows=1, d=1024, dtype="bf16", post=True, norm_y=True, gates=1, pre=True),
        # a training batch of eight sequences, each with its gate, between two blocks
        dict(name="norm 131072x1024", op="norm", rows=131072, d=1024, dtype="bf16", post=True, norm_y=True, gates=8, pre=True),
        # an odd width in fp32: residual addition, then the next block's norm
        dict(name="norm grad 2047x1001 f32", op="norm_grad", rows=2047, d=1001, dtype="f32", post=True, norm_y=False, gates=0, pre=True),
        # the backward pass of that training batch
        dict(name="norm grad 131072x1024", op="norm_grad", rows=131072, d=1024, dtype="bf16", post=True, norm_y=True, gates=8, pre=True),
    ]


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["balance", "router_grad", "combine_grad", "dispatch_grad", "norm", "norm_grad"])
    if op in ("balance", "router_grad"):
        experts = _between(rng, 2, 256)
        return dict(op=op, tokens=_between(rng, 1, 131072 * 64 // max(64, experts)), experts=experts,
                    k=min(experts, rng.choice([1, 2, 2, 3, 8])), masked=rng.random() < 0.5)
    if op in ("combine_grad", "dispatch_grad"):
        d, experts, tokens = 256 * rng.randint(1, 5), rng.randint(2, 64), _between(rng, 1, 100000)
        capacity = rng.choice([0, max(1, int(2 * tokens / experts * rng.uniform(0.5, 1.5)))])
        return dict(op=op, tokens=tokens, d=d, experts=experts, capacity=min(capacity, 2 * tokens))
    d = _between(rng, 16, 8192) if rng.random() < 0.5 else 64 * _between(rng, 1, 128)
    gates = rng.choice([0, 1, _between(rng, 2, 32)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    rows = _between(rng, 1, min(131072, (1 << (27 if dtype == "bf16" else 26)) // d))
    rows = max(1, gates) * max(1, rows // max(1, gates))
    post = rng.random() < 0.8
    return dict(op=op, rows=rows, d=d, dtype=dtype, post=post, norm_y=post and rng.random() < 0.6,
                gates=gates if post else 0, pre=not post or rng.random() < 0.8)


def _route(gen, tokens, experts, k):
    """Router logits with popular and rare experts, the chosen experts (best
    first) and their gates."""
    dev = "cuda"
    bias = torch.linspace(0.7, -0.7, experts, device=dev)
    logits = torch.randn(tokens, experts, generator=gen, device=dev) * 1.2 + bias
    kept, idx = logits.topk(k, dim=1)
    return logits, idx.to(torch.int32), torch.softmax(kept, dim=1)


def _dispatch(experts, gates_of, capacity):
    """Segment offsets and the tuple index held by each dispatched row: a
    stable sort by expert, each expert keeping its first `capacity` tuples. The
    index has the rows of the static bound; those behind the last kept tuple hold nothing."""
    dest = experts.reshape(-1).long()
    order = torch.argsort(dest, stable=True)
    counts = torch.bincount(dest, minlength=gates_of)
    start = counts.cumsum(0) - counts
    if capacity:
        place = torch.arange(dest.numel(), device=dest.device) - start[dest[order]]
        order = order[place < capacity]
        counts = counts.clamp(max=capacity)
    offsets = torch.zeros(gates_of + 1, dtype=torch.int64, device=dest.device)
    offsets[1:] = counts.cumsum(0)
    rows = min(dest.numel(), gates_of * capacity) if capacity else dest.numel()
    src_index = torch.full((rows,), -7, dtype=torch.int32, device=dest.device)
    src_index[:order.numel()] = order.to(torch.int32)
    return offsets, src_index


def _slots(src_index, offsets, tokens):
    """The row of each tuple, -1 where it was dropped."""
    rows = torch.arange(src_index.numel(), device=src_index.device)
    src = torch.where(rows < offsets[-1], src_index.long(), 2 * tokens)
    slot_of = torch.full((2 * tokens + 1,), -1, dtype=torch.int32, device=src_index.device)
    slot_of[src] = rows.to(torch.int32)
    return slot_of[:2 * tokens].view(tokens, 2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dev = case["op"], "cuda"

    def randn(*shape, dtype=torch.float32, scale=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device=dev) * scale + mean).to(dtype)

    s = {"case": case}
    if op in ("balance", "router_grad"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        s["logits"], s["experts"], s["gates"] = _route(gen, T, E, k)
        s["valid"] = (torch.rand(T, generator=gen, device=dev) < 0.9) if case["masked"] else None
        if op == "router_grad":
            s["dgates"] = randn(T, k, scale=1e-2)
            s["grad_loss"] = torch.rand(2, generator=gen, device=dev) + 0.5
            seen = s["experts"] if s["valid"] is None else s["experts"][s["valid"]]
            s["counts"] = torch.cat([torch.bincount(seen.reshape(-1).long(), minlength=E),
                                     torch.tensor([seen.shape[0]], device=dev)]).to(torch.int32)
    elif op in ("combine_grad", "dispatch_grad"):
        T, E, d = case["tokens"], case["experts"], case["d"]
        _, experts, s["gates"] = _route(gen, T, E, 2)
        s["offsets"], s["src_index"] = _dispatch(experts, E, case["capacity"])
        rows = s["src_index"].numel()
        if op == "combine_grad":
            s["dout"] = randn(T, d, dtype=torch.bfloat16, scale=1e-2)
            s["y"] = randn(rows, d, dtype=torch.bfloat16)
            s["dy"] = torch.zeros(rows, d, dtype=torch.bfloat16, device=dev)
        else:
            s["slot_of"] = _slots(s["src_index"], s["offsets"], T)
            s["x"] = randn(T, d, dtype=torch.bfloat16)
            s["dxd"] = randn(rows, d, dtype=torch.bfloat16, scale=1e-2)
            s["dlogits"] = randn(T, E, scale=1e-2)
            s["w_router"] = randn(d, E, dtype=torch.bfloat16, scale=d ** -0.5)
    else:
        T, d, dt = case["rows"], case["d"], _DT[case["dtype"]]
        s["w_y"] = randn(d, dtype=dt, scale=0.1, mean=1.0) if case["norm_y"] else None
        s["w_r"] = randn(d, dtype=dt, scale=0.1, mean=1.0) if case["pre"] else None
        s["gate"] = randn(case["gates"], d, dtype=dt, scale=0.3, mean=0.5) if case["gates"] else None
        s["y"] = randn(T, d, dtype=dt, scale=2.0) if case["post"] else None
        if op == "norm":
            s["x"] = randn(T, d, dtype=dt, scale=3.0)
        else:
            s["r"] = randn(T, d, dtype=dt, scale=3.0) if case["pre"] else None
            s["dr"] = randn(T, d, dtype=dt, scale=1e-2)
            s["dh"] = randn(T, d, dtype=dt, scale=1e-2) if case["pre"] else None
    s["handle"] = _handle(case, s) if own else None
    return s


def _handle(case, s):
    """What a program keeps between its calls: the operator with its output buffers and workspace."""
    import sparse_shard_exchange_amd as pw
    if case["op"] in ("balance", "router_grad"):
        return pw.RouterBalance(case["tokens"], case["experts"], top_k=case["k"], balance_coef=_BALANCE, z_coef=_Z)
    if case["op"] in ("combine_grad", "dispatch_grad"):
        return pw.MoEGrad(case["tokens"], case["d"], case["experts"], rows=s["src_index"].numel())
    return pw.BlockNorm(case["rows"], case["d"], dtype=pw.PW_BF16 if case["dtype"] == "bf16" else pw.PW_F32,
                        gates=case["gates"], x_scale=_X_SCALE, y_scale=_Y_SCALE, eps=_EPS)


def run(state):
    if own:
        return _call(state)
    op = state["case"]["op"]
    if op == "balance":
        return _balance(state)
    if op == "router_grad":
        return _router_grad(state)
    if op == "combine_grad":
        return _combine_grad(state)
    if op == "dispatch_grad":
        return _dispatch_grad(state)
    if op == "norm":
        return _norm(state)
    return _norm_grad(state)


def _call(s):
    op, f = s["case"]["op"], s["handle"]
    if op == "balance":
        counts, prob_mean, loss = f.loss(s["logits"], s["experts"], valid=s["valid"])
        return {"counts": counts, "prob_mean": prob_mean, "loss": loss}
    if op == "router_grad":
        return {"dlogits": f.grad(s["logits"], s["experts"], counts=s["counts"], gates=s["gates"], dgates=s["dgates"],
                                  valid=s["valid"], grad_loss=s["grad_loss"])}
    if op == "combine_grad":
        dy, dgates, slot_of = f.combine(s["dout"], s["y"], s["gates"], s["src_index"], s["offsets"], dy=s["dy"])
        return {"dy": dy, "dgates": dgates, "slot_of": slot_of}
    if op == "dispatch_grad":
        dx, dw = f.dispatch(s["dxd"], s["dlogits"], s["w_router"], s["x"], slot_of=s["slot_of"])
        return {"dx": dx, "dw_router": dw}
    if op == "norm":
        r, h = f.forward(s["x"], y=s["y"], w_y=s["w_y"], gate=s["gate"], w_r=s["w_r"])
        return {"r": r, "h": h}
    dx, dy, dw_y, dgate, dw_r = f.grad(s["dr"], dh=s["dh"], r=s["r"], y=s["y"], w_y=s["w_y"], gate=s["gate"], w_r=s["w_r"])
    return {"dx": dx, "dy": dy, "dw_y": dw_y, "dgate": dgate, "dw_r": dw_r}


# ---- plain forms ---------------------------------------------------------------


def _balance(s):
    k, E = s["case"]["k"], s["case"]["experts"]
    logits, experts = s["logits"].float(), s["experts"]
    top = logits.amax(dim=1, keepdim=True)
    z = torch.exp(logits - top)
    total = z.sum(dim=1, keepdim=True)
    p, lse = z / total, (top + torch.log(total)).squeeze(1)
    n = torch.full((), logits.shape[0], device=logits.device)
    if s["valid"] is not None:
        n = s["valid"].sum()
        p = torch.where(s["valid"].unsqueeze(1), p, torch.zeros_like(p))
        lse = torch.where(s["valid"], lse, torch.zeros_like(lse))
        experts = torch.where(s["valid"].unsqueeze(1), experts, torch.full_like(experts, -1))
    some = n.clamp(min=1).float()
    prob_mean = p.sum(dim=0) / some
    counts = (experts.reshape(-1, 1) == torch.arange(E, device=experts.device)).sum(dim=0)
    balance = (counts.float() / (k * some) * prob_mean).sum() * (_BALANCE * E)
    loss = torch.stack([balance, (lse * lse).sum() * _Z / some])
    return {"counts": torch.cat([counts, n.reshape(1)]).to(torch.int32), "prob_mean": prob_mean, "loss": loss}


def _router_grad(s):
    k, E = s["case"]["k"], s["case"]["experts"]
    logits = s["logits"].float()
    n = s["counts"][E].clamp(min=1).float()
    top = logits.amax(dim=1, keepdim=True)
    z = torch.exp(logits - top)
    total = z.sum(dim=1, keepdim=True)
    p, lse = z / total, top + torch.log(total)
    c = s["counts"][:E].float() / n
    c = c - c.mean()  # the probabilities sum to one: a common part of the counts has no gradient
    d = p * (c - (p * c).sum(dim=1, keepdim=True)) * (s["grad_loss"][0] * (_BALANCE * E / k) / n)
    d = d + p * lse * (s["grad_loss"][1] * 2 * _Z / n)
    g, dg = s["gates"], s["dgates"]
    part = g * (dg - (g * dg).sum(dim=1, keepdim=True))
    d.scatter_add_(1, s["experts"].long(), part)
    if s["valid"] is not None:
        d = torch.where(s["valid"].unsqueeze(1), d, torch.zeros_like(d))
    return {"dlogits": d}


def _combine_grad(s):
    T = s["case"]["tokens"]
    kept = torch.arange(s["src_index"].numel(), device=s["y"].device) < s["offsets"][-1]
    src = torch.where(kept, s["src_index"].long(), 2 * T)
    at = src.clamp(max=2 * T - 1)
    rows = s["dout"].float()[at // 2]
    dy = (rows * s["gates"].reshape(-1)[at].unsqueeze(1)).to(torch.bfloat16)
    dy = torch.where(kept.unsqueeze(1), dy, s["dy"])  # rows behind the last kept tuple stay as they were
    dgates = torch.zeros(2 * T + 1, device=rows.device)
    dgates[src] = (rows * s["y"].float()).sum(dim=1)
    return {"dy": dy, "dgates": dgates[:2 * T].view(T, 2), "slot_of": _slots(s["src_index"], s["offsets"], T)}


def _dispatch_grad(s):
    slot = s["slot_of"].long()
    rows = s["dxd"].float()[slot.clamp(min=0)] * (slot >= 0).unsqueeze(2)
    dx = rows.sum(dim=1) + s["dlogits"] @ s["w_router"].float().t().contiguous()
    return {"dx": dx.to(torch.bfloat16), "dw_router": s["x"].float().t().contiguous() @ s["dlogits"]}


def _rstd(v):
    return torch.rsqrt((v * v).mean(dim=1, keepdim=True) + _EPS)


def _gate_rows(s, T):
    """The gate of every row, as a view that broadcasts inside a group."""
    g = s["gate"].float()
    return g.unsqueeze(1).expand(g.shape[0], T // g.shape[0], g.shape[1]).reshape(T, g.shape[1])


def _norm(s):
    dt = s["x"].dtype
    r = s["x"].float() * _X_SCALE
    if s["y"] is not None:
        y = s["y"].float()
        if s["w_y"] is not None:
            y = y * _rstd(y) * s["w_y"].float()
        if s["gate"] is not None:
            y = y * _gate_rows(s, y.shape[0])
        r = r + y * _Y_SCALE
    h = (r * _rstd(r) * s["w_r"].float()).to(dt) if s["w_r"] is not None else None
    return {"r": r.to(dt) if s["y"] is not None else None, "h": h}


def _norm_grad(s):
    dt = s["dr"].dtype
    out = {"dx": None, "dy": None, "dw_y": None, "dgate": None, "dw_r": None}
    dr = s["dr"].float()
    if s["w_r"] is not None:
        r, dh = s["r"].float(), s["dh"].float()
        rstd = _rstd(r)
        hat, g = r * rstd, dh * s["w_r"].float()
        out["dw_r"] = (dh * hat).sum(dim=0)
        dr = dr + rstd * (g - hat * (g * hat).mean(dim=1, keepdim=True))
    out["dx"] = (dr * _X_SCALE).to(dt)
    if s["y"] is not None:
        y = s["y"].float()
        T, d = y.shape
        hat, rstd = y, None
        if s["w_y"] is not None:
            rstd = _rstd(y)
            hat = y * rstd
        q = dr * _Y_SCALE
        if s["gate"] is not None:
            n = hat if s["w_y"] is None else hat * s["w_y"].float()
            G = s["gate"].shape[0]
            out["dgate"] = (q * n).view(G, T // G, d).sum(dim=1)
            q = q * _gate_rows(s, T)
        if s["w_y"] is not None:
            out["dw_y"] = (q * hat).sum(dim=0)
            q = q * s["w_y"].float()
            q = rstd * (q - hat * (q * hat).mean(dim=1, keepdim=True))
        out["dy"] = q.to(dt)
    return out


# ---- what one pass cannot do without -------------------------------------------


def work(case):
    op = case["op"]
    if op in ("balance", "router_grad"):
        T, E, k = case["tokens"], case["experts"], case["k"]
        moved = T * E * 4 + T * k * 4 + (T if case["masked"] else 0) + 8 * E + 12
        if op == "balance":
            return {"bytes": moved, "flops": 6 * T * E}
        return {"bytes": moved + T * E * 4 + 8 * T * k, "flops": 10 * T * E + 6 * T * k}
    if op in ("combine_grad", "dispatch_grad"):
        T, E, d = case["tokens"], case["experts"], case["d"]
        rows = min(2 * T, E * case["capacity"]) if case["capacity"] else 2 * T  # kept at most
        if op == "combine_grad":
            return {"bytes": 2 * d * (T + 2 * rows) + 4 * rows + 24 * T, "flops": 3 * rows * d}
        return {"bytes": 2 * d * (2 * T + rows) + 8 * T + 4 * T * E + 6 * d * E, "flops": 4 * T * d * E + 2 * T * d}
    n = case["rows"] * case["d"]
    size = 2 if case["dtype"] == "bf16" else 4
    tensors = (2 if case["post"] else 0) + (1 if case["pre"] else 0)
    if op == "norm":
        return {"bytes": size * (n * (1 + tensors) + case["d"] * (2 + case["gates"])), "flops": 10 * n}
    tensors += 2 + (1 if case["pre"] else 0)
    return {"bytes": size * (n * tensors + case["d"] * (2 + case["gates"])) + 4 * case["d"] * (2 + case["gates"]), "flops": 20 * n}


# ---- the definitions in 64 bits ------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    return {"balance": _exact_balance, "router_grad": _exact_router, "combine_grad": _exact_combine,
            "dispatch_grad": _exact_dispatch, "norm": _exact_norm, "norm_grad": _exact_norm_grad}[case["op"]](case, s)


def _exact_balance(case, s):
    E, k, T = case["experts"], case["k"], case["tokens"]
    valid = torch.ones(T, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"]
    l = s["logits"].double()
    p = torch.softmax(l, dim=1)
    n = int(valid.sum())
    counts = torch.bincount(s["experts"][valid].reshape(-1).long(), minlength=E)
    if n == 0:
        zero = torch.zeros(E, dtype=torch.float64, device="cuda")
        return {"counts": None, "prob_mean": zero, "loss": zero[:2]}
    mean = p[valid].mean(dim=0)
    loss_b = _BALANCE * E * torch.dot(counts.double() / (k * n), mean)
    loss_z = _Z * torch.logsumexp(l[valid], dim=1).square().mean()
    return {"counts": None, "prob_mean": mean, "loss": torch.stack([loss_b, loss_z])}


def _exact_router(case, s):
    """The gradient by differentiating the losses and the gates in 64 bits."""
    E, k, T = case["experts"], case["k"], case["tokens"]
    valid = torch.ones(T, dtype=torch.bool, device="cuda") if s["valid"] is None else s["valid"]
    counts, n = s["counts"][:E].double(), max(1, int(s["counts"][E]))
    l = s["logits"].double().requires_grad_(True)
    u = s["grad_loss"].double()
    with torch.enable_grad():
        lv = l[valid]
        lse = torch.logsumexp(lv, dim=1, keepdim=True)
        p = torch.exp(lv - lse)
        total = u[0] * _BALANCE * E / (k * n) * (p.sum(dim=0) / n * counts).sum() + u[1] * _Z / n * lse.square().sum()
        (d,) = torch.autograd.grad(total, l)
    # the gates are inputs: their softmax is differentiated at their own values
    g, dg = s["gates"].double(), s["dgates"].double()
    for a in range(k):
        for b in range(k):
            j = g[:, a] * ((1.0 if a == b else 0.0) - g[:, b]) * dg[:, b]
            d[torch.arange(T, device="cuda"), s["experts"][:, a].long()] += torch.where(valid, j, torch.zeros_like(j))
    return {"dlogits": d}


def _exact_combine(case, s):
    T, d = case["tokens"], case["d"]
    n = int(s["offsets"][-1])
    dy = torch.zeros(s["src_index"].numel(), d, dtype=torch.float64, device="cuda")
    dgates = torch.zeros(T, 2, dtype=torch.float64, device="cuda")
    for lo in range(0, n, 65536):
        hi = min(lo + 65536, n)
        g = s["src_index"][lo:hi].long()
        t, j = g >> 1, g & 1
        rows = s["dout"][t].double()
        dy[lo:hi] = s["gates"][t, j].double()[:, None] * rows
        dgates[t, j] = (rows * s["y"][lo:hi].double()).sum(1)
    return {"dy": dy, "dgates": dgates, "slot_of": None}


def _exact_dispatch(case, s):
    T, d = case["tokens"], case["d"]
    w = s["w_router"].double()
    dx = torch.empty(T, d, dtype=torch.float64, device="cuda")
    dw = torch.zeros(d, case["experts"], dtype=torch.float64, device="cuda")
    for lo in range(0, T, 32768):
        dl = s["dlogits"][lo:lo + 32768].double()
        part = torch.matmul(dl, w.T.contiguous())
        for j in range(2):
            slot = s["slot_of"][lo:lo + 32768, j].long()
            have = slot >= 0
            part[have] += s["dxd"][slot[have]].double()
        dx[lo:lo + 32768] = part
        dw += torch.matmul(s["x"][lo:lo + 32768].double().T.contiguous(), dl)
    return {"dx": dx, "dw_router": dw}


def _parts(case):
    """Row ranges of one gate each, of at most 32768 rows."""
    groups = max(1, case["gates"])
    size = case["rows"] // groups
    return [(g, lo, min(lo + 32768, (g + 1) * size)) for g in range(groups) for lo in range(g * size, (g + 1) * size, 32768)]


def _exact_norm(case, s):
    T, d = case["rows"], case["d"]
    r = torch.empty(T, d, dtype=torch.float64, device="cuda")
    h = torch.empty_like(r) if case["pre"] else None
    for g, lo, hi in _parts(case):
        v = _X_SCALE * s["x"][lo:hi].double()
        if case["post"]:
            y = s["y"][lo:hi].double()
            if case["norm_y"]:
                y = y / torch.sqrt(y.square().mean(1, True) + _EPS) * s["w_y"].double()
            v = v + _Y_SCALE * (y * s["gate"][g].double() if case["gates"] else y)
        r[lo:hi] = v
        if case["pre"]:
            h[lo:hi] = v / torch.sqrt(v.square().mean(1, True) + _EPS) * s["w_r"].double()
    return {"r": r if case["post"] else None, "h": h}


def _exact_norm_grad(case, s):
    """The gradient by differentiating the norms in 64 bits, range by range."""
    T, d = case["rows"], case["d"]

    def new(*shape):
        return torch.zeros(*shape, dtype=torch.float64, device="cuda")

    out = {"dx": new(T, d), "dy": new(T, d) if case["post"] else None, "dw_y": new(d) if case["norm_y"] else None,
           "dgate": new(case["gates"], d) if case["gates"] else None, "dw_r": new(d) if case["pre"] else None}
    for g, lo, hi in _parts(case):
        dr = s["dr"][lo:hi].double()
        if case["pre"]:
            r, w = s["r"][lo:hi].double().requires_grad_(True), s["w_r"].double().requires_grad_(True)
            with torch.enable_grad():
                h = r / torch.sqrt(r.square().mean(1, True) + _EPS) * w
                a, b = torch.autograd.grad(h, (r, w), s["dh"][lo:hi].double())
            dr = dr + a
            out["dw_r"] += b
        out["dx"][lo:hi] = _X_SCALE * dr
        if case["post"]:
            leaves = {"dy": s["y"][lo:hi].double().requires_grad_(True)}
            if case["norm_y"]:
                leaves["dw_y"] = s["w_y"].double().requires_grad_(True)
            if case["gates"]:
                leaves["dgate"] = s["gate"][g].double().requires_grad_(True)
            with torch.enable_grad():
                v = leaves["dy"]
                if case["norm_y"]:
                    v = v / torch.sqrt(v.square().mean(1, True) + _EPS) * leaves["dw_y"]
                if case["gates"]:
                    v = v * leaves["dgate"]
                found = dict(zip(leaves, torch.autograd.grad(_Y_SCALE * v, list(leaves.values()), dr)))
            out["dy"][lo:hi] = found["dy"]
            if case["norm_y"]:
                out["dw_y"] += found["dw_y"]
            if case["gates"]:
                out["dgate"][g] += found["dgate"]
    return out
