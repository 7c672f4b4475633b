"""GPU parity of the gradients of an MoE step's combine, dispatch and router
against the oracle in 64 bits, and a run of the whole block.

Bars, u = 2^-24, bf16's half step 2^-8: dy is one fp32 product rounded once; a
gate's gradient is an fp32 sum of d <= 1280 products, 24 in a lane and 6
exchanges (64 u of its terms); dx adds a product in fp32, for which the bar
lets dlogits lose 2^-16 (they lose nothing), and two rows; dw_router's
products are exact and its sums fp32: over a token range 48 roundings (3 terms
of 16 tokens) for each 64 tokens, then 4 waves and the ranges, 65536 / d of them
at most and whole multiples of 64 tokens.
"""
import numpy as np
import pytest
import torch

import pw_inputs
from oracle import block as ob
from oracle import moe as om

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8
bf = torch.bfloat16

CASES = [(1, 256, 2, 0), (50, 256, 3, 0), (50, 512, 4, 0), (70, 256, 6, 0), (70, 256, 31, 0), (90, 256, 34, 0), (1, 256, 64, 1), (7, 512, 5, 0), (33, 256, 33, 1), (300, 1280, 8, 0), (300, 512, 64, 6),
         (1000, 256, 5, 350), (1003, 768, 12, 0), (4097, 1024, 64, 100), (5000, 256, 64, 0),
         (65600, 256, 5, 0), (66001, 512, 64, 2000)]   # more tiles than waves


def make(T, d, E, cap, seed=0, masked=False):
    rng = np.random.default_rng([T, d, E, cap, seed])
    logits = rng.standard_normal((T, E)).astype(np.float32)
    _, g, _, _, offsets, src = om.route(logits, E, 1, cap)
    kept = src.size
    rows = min(2 * T, E * cap) if cap else 2 * T
    index = np.full(rows, -5, np.int32)
    index[:kept] = src

    def t(*shape, scale=1.0):
        return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(bf)

    s = dict(dout=t(T, d), y=t(rows, d), gates=torch.from_numpy(g.astype(np.float32)), src_index=torch.from_numpy(index),
             offsets=torch.from_numpy(offsets.astype(np.int64)), dxd=t(rows, d), w_router=t(d, E, scale=d ** -0.5), x=t(T, d),
             dlogits=torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)))
    s["y"][kept:] = float("nan")                  # rows that hold nothing are not looked at
    s["dxd"][kept:] = float("nan")
    s["valid"] = torch.from_numpy(rng.random(T) < 0.7) if masked else None
    return s, kept


def f64(t):
    return None if t is None else t.double().numpy()


def check_combine(got, s, kept, before):
    dy, dg, slot_of = (t.cpu() for t in got)
    src = s["src_index"].numpy()
    T = s["dout"].shape[0]
    valid = None if s["valid"] is None else s["valid"].numpy()
    want, dgw, size = ob.combine_grad(f64(s["dout"]), f64(s["y"]), f64(s["gates"]), src, kept, valid)
    assert np.array_equal(slot_of.numpy(), ob.slots(src, kept, T))
    assert np.all(np.abs(f64(dy[:kept]) - want) <= (HALF + 2 * U) * np.abs(want) + 1e-38)
    assert torch.equal(dy[kept:], before[kept:])  # left as they were
    assert np.all(np.abs(f64(dg) - dgw) <= 64 * U * size)


def token_range(T, d):
    """Tokens of one partial sum of dw_router."""
    return -(-max(64, -(-T // (256 // (d // 256))), min(256, -(-T // 16))) // 64) * 64


def check_dispatch(got, s, kept):
    slot_of = ob.slots(s["src_index"].numpy(), kept, s["x"].shape[0])
    valid = None if s["valid"] is None else s["valid"].numpy()
    dx, size, rows, dw, dws = ob.dispatch_grad(f64(s["dxd"]), f64(s["dlogits"]), f64(s["w_router"]), f64(s["x"]), slot_of, valid)
    bound = (2.0 ** -16 + 200 * U) * size + 4 * U * rows
    assert np.all(np.abs(f64(got[0].cpu()) - dx) <= bound + HALF * (np.abs(dx) + bound) + 1e-38)
    if got[1] is not None:
        T, d = s["x"].shape
        span = token_range(T, d)
        assert np.all(np.abs(f64(got[1].cpu()) - dw) <= (48 * span // 64 + -(-T // span) + 8) * U * dws + 1e-38)


def run(pw, s, f=None, stream=None):
    c = {n: None if t is None else t.cuda() for n, t in s.items()}
    T, d = s["x"].shape
    f = f or pw.MoEGrad(T, d, s["w_router"].shape[1], rows=s["y"].shape[0])
    dy = torch.full_like(c["y"], 3.0)
    before = dy.cpu()
    a = f.combine(c["dout"], c["y"], c["gates"], c["src_index"], c["offsets"], c["valid"], dy=dy, stream=stream)
    b = f.dispatch(c["dxd"], c["dlogits"], c["w_router"], c["x"], valid=c["valid"], stream=stream)
    return a, b, before, c, f


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,d,E,cap", CASES)
def test_combine_and_dispatch_gradients(gpu, T, d, E, cap, masked):
    print(f"moe grad T={T} d={d} E={E} cap={cap} masked={masked}", flush=True)
    s, kept = make(T, d, E, cap, masked=masked)
    if masked:   # padding holds anything
        bad = ~s["valid"]
        s2 = {n: None if t is None else t.clone() for n, t in s.items()}
        for n in ("dout", "x"):
            s2[n][bad] = float("nan")
        s2["gates"][bad] = float("inf")
        s2["dlogits"][bad] = float("nan")
        s["dlogits"][bad] = 0.0
        a, b, before, c, f = run(gpu, s2)
    else:
        a, b, before, c, f = run(gpu, s)
    check_combine(a, s, kept, before)
    check_dispatch(b, s, kept)
    first = [t.clone() for t in b]
    again = f.dispatch(c["dxd"], c["dlogits"], c["w_router"], c["x"], valid=c["valid"])
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])   # equal inputs, equal bits
    dx, none = f.dispatch(c["dxd"], c["dlogits"], c["w_router"], valid=c["valid"])
    assert none is None and torch.equal(dx, first[0])


def test_everything_dropped_and_no_rows(gpu):
    """No row kept (offsets all zero), and buffers without rows."""
    for rows in (20, 0):
        s, _ = make(10, 256, 4, 0)
        s["offsets"].zero_()
        for n in ("y", "dxd"):
            s[n] = s[n][:rows].contiguous()
        s["src_index"] = s["src_index"][:rows].contiguous()
        a, b, before, _, _ = run(gpu, s)
        assert torch.equal(a[0].cpu(), before) and not a[1].any() and torch.all(a[2] == -1)
        check_dispatch(b, s, 0)


def test_foreign_indices_are_dropped(gpu):
    """Source indices outside [0, 2 T) and slots outside the rows touch nothing."""
    s, kept = make(40, 256, 4, 0)
    s["src_index"][5], s["src_index"][9] = -3, 1 << 30
    a, b, before, c, f = run(gpu, s)
    assert torch.all(a[2].cpu().view(-1)[s["src_index"][[0, 1, 2]].long()] >= 0)
    assert torch.equal(a[0][[5, 9]].cpu(), before[[5, 9]])
    slot = a[2].clone()
    slot[0, 0], slot[1, 1] = 80, -9
    dx, _ = f.dispatch(c["dxd"], c["dlogits"], c["w_router"], slot_of=slot)
    slot[0, 0], slot[1, 1] = -1, -1
    want = f.dispatch(c["dxd"], c["dlogits"], c["w_router"], slot_of=slot.clone())[0]
    assert torch.equal(dx, want)


def test_router_weights_that_are_not_16_byte_aligned(gpu):
    s, kept = make(100, 256, 8, 0)
    a, b, before, c, f = run(gpu, s)
    flat = torch.zeros(256 * 8 + 1, dtype=bf, device="cuda")
    w = flat[1:].view(256, 8)
    w.copy_(c["w_router"])
    check_dispatch(f.dispatch(c["dxd"], c["dlogits"], w, c["x"]), s, kept)


@pytest.mark.parametrize("E,cap", [(16, 700), (64, 150)])
def test_a_replayed_graph_and_another_stream(gpu, E, cap):
    T, d = 6000, 512
    data = [make(T, d, E, cap, seed) for seed in range(4)]
    a, b, before, c, f = run(gpu, data[0][0])
    dy = a[0]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a = f.combine(c["dout"], c["y"], c["gates"], c["src_index"], c["offsets"], dy=dy)
        b = f.dispatch(c["dxd"], c["dlogits"], c["w_router"], c["x"])
    for s, kept in data[1:] + data[:1]:
        for n, t in s.items():
            if t is not None:
                c[n].copy_(t.cuda())
        dy.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        check_combine(a, s, kept, before)
        check_dispatch(b, s, kept)
    side.wait_stream(torch.cuda.current_stream())
    a = f.combine(c["dout"], c["y"], c["gates"], c["src_index"], c["offsets"], stream=side)
    b = f.dispatch(c["dxd"], c["dlogits"], c["w_router"], c["x"], stream=side)
    side.synchronize()
    check_dispatch(b, s, kept)


@pytest.mark.parametrize("T,d,E", [(60001, 1280, 37), (70000, 1024, 24)])
def test_rows_beyond_the_caches(gpu, T, d, E):
    """512 MiB of rows and more, read past the caches; 64-bit sums on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    src = torch.randperm(2 * T, generator=g, device="cuda").int()
    n = 2 * T
    offsets = torch.full((E + 1,), n, dtype=torch.int64, device="cuda")
    dout, y, gates = rnd(T, d).to(bf), rnd(n, d).to(bf), torch.rand(T, 2, generator=g, device="cuda")
    f = gpu.MoEGrad(T, d, E)
    dy, dg, slot_of = f.combine(dout, y, gates, src, offsets)
    assert torch.equal(src[slot_of.view(-1).long()], torch.arange(n, device="cuda", dtype=torch.int32))
    dl, w, x = rnd(T, E), (rnd(d, E) * d ** -0.5).to(bf), rnd(T, d).to(bf)
    dx, dw = f.dispatch(y, dl, w, x)
    want_dw, terms = torch.zeros(d, E, dtype=torch.float64, device="cuda"), torch.zeros(d, E, dtype=torch.float64, device="cuda")
    for lo in range(0, T, 16384):
        hi = min(lo + 16384, T)
        o, s = dout[lo:hi].double(), slot_of[lo:hi].long()
        dl64, x64 = dl[lo:hi].double(), x[lo:hi].double()
        part, size = dl64 @ w.double().t().contiguous(), dl64.abs() @ w.double().abs().t().contiguous()
        rows = torch.zeros_like(part)
        for j in range(2):
            yj = y[s[:, j]].double()
            want = gates[lo:hi, j:j + 1].double() * o
            assert bool(((dy[s[:, j]].double() - want).abs() <= (HALF + 2 * U) * want.abs() + 1e-38).all())
            assert bool(((dg[lo:hi, j].double() - (o * yj).sum(1)).abs() <= 64 * U * (o * yj).abs().sum(1)).all())
            part += yj
            rows += yj.abs()
        bound = (2.0 ** -16 + 200 * U) * size + 4 * U * rows
        assert bool(((dx[lo:hi].double() - part).abs() <= bound + HALF * (part.abs() + bound) + 1e-38).all())
        want_dw += x64.t().contiguous() @ dl64
        terms += x64.abs().t().contiguous() @ dl64.abs()
    span = token_range(T, d)
    assert bool(((dw.double() - want_dw).abs() <= (48 * span // 64 + -(-T // span) + 8) * U * terms).all())


def test_offsets_past_32_bits(gpu):
    """More than 2^32 elements of dispatched rows: the last tokens as in a call of their own."""
    T, d, E, k = 1700000, 1280, 8, 40
    assert 2 * T * d > 1 << 32
    dev = "cuda"
    src = torch.arange(2 * T, dtype=torch.int32, device=dev)
    offsets = torch.full((E + 1,), 2 * T, dtype=torch.int64, device=dev)
    g = torch.Generator(device=dev).manual_seed(3)
    tail = lambda n, *s, dt=bf: torch.randn(n, *s, generator=g, device=dev).to(dt)  # noqa: E731

    def long(n, last, dt=bf):
        t = torch.zeros(n, last.shape[1], dtype=dt, device=dev)
        t[-last.shape[0]:] = last
        return t

    dout, y, gates, dl, x, w = tail(k, d), tail(2 * k, d), tail(k, 2, dt=torch.float32), tail(k, E, dt=torch.float32), tail(k, d), tail(d, E)
    big, small = gpu.MoEGrad(T, d, E), gpu.MoEGrad(k, d, E)
    Y = long(2 * T, y)
    a = big.combine(long(T, dout), Y, long(T, gates, torch.float32), src, offsets)
    b = small.combine(dout, y, gates, src[:2 * k].contiguous(), torch.full_like(offsets, 2 * k))
    assert torch.equal(a[0][-2 * k:], b[0]) and torch.equal(a[1][-k:], b[1])
    assert torch.equal(a[2].view(-1), src) and not a[0][:2 * (T - k)].any()
    p = big.dispatch(Y, long(T, dl, torch.float32), w, long(T, x))
    q = small.dispatch(y, dl, w, x)
    assert torch.equal(p[0][-k:], q[0]) and not p[0][:T - k].any()
    size = x.double().abs().t().contiguous() @ dl.double().abs()
    assert bool(((p[1].double() - x.double().t().contiguous() @ dl.double()).abs() <= 200 * U * size).all())


def test_more_tokens_than_a_grid_has_threads(gpu):
    """2^27 tokens of a few kept tuples: the workgroups walk on."""
    T, d, E, k = (1 << 27) + 40, 256, 4, 24
    assert (T + 7) // 8 * 256 >= 1 << 32
    rng = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=rng, device="cuda")  # noqa: E731
    src = torch.cat([torch.arange(0, k // 2), torch.arange(2 * T - k // 2, 2 * T)]).int().cuda()  # the first and last tokens
    offsets = torch.full((E + 1,), k, dtype=torch.int64, device="cuda")
    y, ends = rnd(k, d).to(bf), rnd(k // 2, d).to(bf)
    dout = torch.zeros(T, d, dtype=bf, device="cuda")
    dout[:k // 4], dout[-(k // 4):] = ends[:k // 4], ends[k // 4:]
    gates = torch.full((T, 2), 0.5, device="cuda")
    dy, dg, slot_of = gpu.MoEGrad(T, d, E, rows=k).combine(dout, y, gates, src, offsets)
    per_row = ends.repeat_interleave(2, dim=0)
    assert torch.equal(dy, (per_row.float() * 0.5).to(bf))
    want = (per_row.double() * y.double()).sum(1)
    got = torch.cat([dg[:k // 4].view(-1), dg[-(k // 4):].view(-1)]).double()
    assert bool(((got - want).abs() <= 64 * U * (per_row.double() * y.double()).abs().sum(1)).all())
    assert not dg[k // 4:-(k // 4)].any() and bool((slot_of[k // 4:-(k // 4)] == -1).all())


def test_refusals(gpu):
    s, _ = make(16, 256, 4, 0)
    f = gpu.MoEGrad(16, 256, 4)
    c = {n: None if t is None else t.cuda() for n, t in s.items()}
    args = ("dout", "y", "gates", "src_index", "offsets")
    for n in args:
        short = c[n][:, 1:] if n == "y" else c[n][1:]    # (fewer rows of y are another capacity's)
        for bad in (c[n].cpu(), short, c[n].to(torch.float16)):
            with pytest.raises(gpu.PwError):
                f.combine(*[bad if m == n else c[m] for m in args])
    with pytest.raises(gpu.PwError):
        f.dispatch(c["dxd"], c["dlogits"], c["w_router"], c["x"])     # no slot_of yet
    with pytest.raises(gpu.PwError):
        gpu.MoEGrad(16, 320, 4)
    with pytest.raises(gpu.PwError):
        gpu.MoEGrad(16, 256, 4, rows=8).combine(*[c[m] for m in args])


# ---- the whole block -----------------------------------------------------------------


def expert_products(m, xd, w1, w2, dy, offs):
    """Gradient of the experts' products, dy to dxd, as a caller runs it."""
    dxd = torch.zeros_like(xd)
    for e in range(m.E):
        lo, hi = int(offs[e]), int(offs[e + 1])
        if hi > lo:
            a = xd[lo:hi].float() @ w1[e].float()
            a.requires_grad_(True)
            with torch.enable_grad():
                h = torch.nn.functional.gelu(a)
            (da,) = torch.autograd.grad(h, a, dy[lo:hi].float() @ w2[e].float().t().contiguous())
            dxd[lo:hi] = (da @ w1[e].float().t().contiguous()).to(bf)
    return dxd


@pytest.mark.parametrize("T,E,cap,masked", [(300, 8, 0, False), (300, 8, 40, True), (1, 4, 0, False)])
def test_block_forward_and_backward(gpu, T, E, cap, masked):
    """Norm, MoE step, norm with gate and residual, balance loss, and back, on
    one stream with nothing waited for, against automatic differentiation of
    the whole block in 64 bits with the routing that the GPU took.

    Bar: relative 2-norms. About ten bf16 roundings (half a step, 2^-8, each at
    most) lie on a gradient's way (h, hidden, y, out and r forward; dout, dy, dxd, dh,
    dx back): 10 x 2^-8. dw_router sees two more, the norm's weights one."""
    d, H, ax, ay, eps = 256, 256, 1.0, 0.5, 1e-5
    inp = pw_inputs.moe(T, d, E, H)
    wr, w1, w2 = inp.w_router.cuda(), inp.w1.cuda(), inp.w2.cuda()
    rng = np.random.default_rng(T)
    t = lambda *s, k=1.0, m=0.0: torch.from_numpy((rng.standard_normal(s) * k + m).astype(np.float32)).to(bf).cuda()  # noqa: E731
    x, w_in, w_out, gate, dr = t(T, d), t(d, k=0.1, m=1.0), t(d, k=0.1, m=1.0), t(1, d, k=0.3, m=0.6), t(T, d)
    valid = (torch.arange(T) % 5 != 2).cuda() if masked else None
    if masked:
        dr[~valid] = 0
    up = torch.tensor([1.5, 0.5], device="cuda")
    m = gpu.MoE(wr, w1, w2, T, num_src_shards=1, capacity=cap)
    block = gpu.MoEBlock(m, w_in, w_out, gate, ax, ay, eps, balance_coef=0.1, z_coef=0.01)
    r, loss, counts, fut = block.forward(x, valid)
    dy = block.grad_begin(dr)
    offs = m.offsets.cpu()
    g = block.grad_end(expert_products(m, m.xd, w1, w2, dy, offs), up)
    gpu.future_wait(fut, 60_000_000_000)

    # the same block in 64 bits, routed as the GPU routed
    D = lambda v: v.double().cpu().requires_grad_(True)  # noqa: E731
    X, WI, WO, G, WR = D(x), D(w_in), D(w_out), D(gate), D(wr)
    norm = lambda v, w: v / torch.sqrt(v.square().mean(1, True) + eps) * w  # noqa: E731
    experts, src = m.experts.cpu().long(), m.src_index.cpu().numpy()
    kept = int(offs[-1])
    with torch.enable_grad():
        h = norm(X, WI)
        lg = h @ WR
        gt = torch.softmax(torch.gather(lg, 1, experts), dim=1)
        slot = torch.from_numpy(ob.slots(src, kept, T))
        out = torch.zeros(T, d, dtype=torch.float64)
        for s in range(2):
            y = torch.stack([torch.nn.functional.gelu(h[i] @ w1[e].double().cpu()) @ w2[e].double().cpu()
                             for i, e in enumerate(experts[:, s].tolist())])
            out = out + torch.where(slot[:, s:s + 1] >= 0, gt[:, s:s + 1] * y, torch.zeros_like(y))
        R = ax * X + ay * G * norm(out, WO)
        v = torch.ones(T, dtype=torch.bool) if valid is None else valid.cpu()
        n = int(v.sum())
        p = torch.softmax(lg[v], dim=1)
        c = counts.cpu().double()[:E]
        L = torch.stack([0.1 * E * (c / (2 * n) * p.mean(0)).sum(), 0.01 * torch.logsumexp(lg[v], 1).square().mean()])
        live = v.unsqueeze(1)
        total = (torch.where(live, R, torch.zeros_like(R)) * dr.double().cpu()).sum() + (L * up.double().cpu()).sum()
        want = torch.autograd.grad(total, [X, WI, WO, G, WR])
    assert torch.equal(counts.cpu()[:E].long(), torch.bincount(experts[v].reshape(-1), minlength=E))
    assert torch.allclose(loss.double().cpu(), L.detach(), rtol=2e-2, atol=0)
    off = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert off(r[v.cuda()], R.detach()[v]) <= 6 * HALF
    for name, b, k in zip(("x", "w_in", "w_out", "gate", "w_router"), want, (10, 11, 11, 11, 12)):
        assert off(g[name], b.view_as(g[name].cpu())) <= k * HALF, (name, off(g[name], b))


def test_block_calls_out_of_order(gpu):
    T, d, E, H = 64, 256, 4, 256
    inp = pw_inputs.moe(T, d, E, H)
    w = inp.w_router.cuda(), inp.w1.cuda(), inp.w2.cuda()
    x, one = torch.ones(T, d, dtype=bf, device="cuda"), torch.ones(d, dtype=bf, device="cuda")
    block = gpu.MoEBlock(gpu.MoE(*w, T, num_src_shards=1), one)
    split = gpu.MoEBlock(gpu.MoE(*w, T, num_src_shards=1, static_buffers=False), one)
    for call in (lambda: block.grad_begin(x), lambda: block.grad_end(x), lambda: split.forward(x)):
        with pytest.raises(gpu.PwError) as e:
            call()
        assert e.value.code == gpu.PW_ERR_STATE
    *_, f = block.forward(x)
    with pytest.raises(gpu.PwError):
        block.grad_end(x)             # no grad_begin yet
    gpu.future_wait(f, 60_000_000_000)


def test_router_gradient_of_many_equal_tokens(gpu):
    """2^26 equal tokens, where fp32 additions err to the same side. The products
    are exact, and so is the sum of a matrix instruction's 16 equal ones; it is
    added to the accumulator in one rounding: 3 for each 64 tokens of a range of at
    most 2^14, then 3 across waves, 64 ranges, and 4 slices."""
    T, d, E = 1 << 26, 256, 2
    g = torch.Generator().manual_seed(1)
    x, dl, w = torch.randn(1, d, generator=g).to(bf), torch.randn(1, E, generator=g), torch.randn(d, E, generator=g).to(bf)
    long = lambda t: t.cuda().expand(T, t.shape[1]).contiguous()  # noqa: E731
    slot_of = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
    none = torch.empty(0, d, dtype=bf, device="cuda")
    _, dw = gpu.MoEGrad(T, d, E, rows=0).dispatch(none, long(dl), w.cuda(), long(x), slot_of=slot_of)
    want = x.double().t().contiguous() @ dl.double()
    off = (dw.double().cpu() / T - want).abs()
    assert bool((off <= (3 * 256 + 3 + 64 + 4 + 2) * U * want.abs()).all())


@pytest.mark.parametrize("T,d,E", [(50, 256, 3), (300, 512, 8), (200, 256, 33), (66000, 256, 64)])
def test_router_terms_that_cancel(gpu, T, d, E):
    """Pairs of experts with the same weights and opposite logit gradients but for
    the last bits: dx is what the lowest bits of dlogits leave. Bar: all 24 bits of
    them, fp32 sums of 3 E terms, and dx's own rounding."""
    rng = np.random.default_rng([T, d, E])
    dl = np.zeros((T, E), np.float32)
    w = torch.from_numpy(rng.standard_normal((d, E)).astype(np.float32)).to(bf)
    for e in range(0, E - 1, 2):
        a = (1 + rng.random(T)).astype(np.float32)
        dl[:, e], dl[:, e + 1] = a, -(a + 2.0 ** -20 * rng.integers(1, 9, T)).astype(np.float32)
        w[:, e + 1] = w[:, e]
    if E % 2:
        dl[:, -1] = 0
    slot_of = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
    dx, _ = gpu.MoEGrad(T, d, E, rows=0).dispatch(torch.empty(0, d, dtype=bf, device="cuda"), torch.from_numpy(dl).cuda(),
                                                  w.cuda(), slot_of=slot_of)
    want = dl.astype(np.float64) @ f64(w).T
    size = np.abs(dl).astype(np.float64) @ np.abs(f64(w)).T
    bound = 3 * E * U * size
    assert np.all(np.abs(f64(dx.cpu()) - want) <= bound + HALF * (np.abs(want) + bound))


@pytest.mark.parametrize("T,E", [(70, 3), (70, 8), (3000, 64)])
def test_the_largest_finite_logit_gradients(gpu, T, E):
    """The largest fp32 value, which rounds to no finite bf16, gives what the formula
    gives: finite results next to small weights and tokens."""
    d = 256
    rng = np.random.default_rng([T, E])
    dl = rng.standard_normal((T, E)).astype(np.float32)
    top = np.finfo(np.float32).max
    dl[5, 1], dl[7, 0], dl[9, 2] = top, -top, top * np.float32(0.9999)
    t = lambda *s, k: torch.from_numpy((rng.standard_normal(s) * k).astype(np.float32)).to(bf)  # noqa: E731
    w, x = t(d, E, k=2.0 ** -12), t(T, d, k=2.0 ** -12)
    none, slot_of = torch.empty(0, d, dtype=bf, device="cuda"), torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
    dx, dw = gpu.MoEGrad(T, d, E, rows=0).dispatch(none, torch.from_numpy(dl).cuda(), w.cuda(), x.cuda(), slot_of=slot_of)
    dl64, w64, x64 = dl.astype(np.float64), f64(w), f64(x)
    want, size = dl64 @ w64.T, np.abs(dl64) @ np.abs(w64).T
    bound = 3 * E * U * size
    assert np.all(np.abs(f64(dx.cpu()) - want) <= bound + HALF * (np.abs(want) + bound) + 1e-38)
    span = token_range(T, d)
    want, size = x64.T @ dl64, np.abs(x64).T @ np.abs(dl64)
    assert np.all(np.abs(f64(dw.cpu()) - want) <= (48 * span // 64 + -(-T // span) + 8) * U * size + 1e-38)


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,d,E", [(68000, 1280, 37), (68000, 1024, 64), (140000, 512, 20)])
def test_all_of_the_router_weights_in_lds(gpu, T, d, E, masked):
    """From 65521 tokens on a workgroup keeps all of W, 160 KiB of it at d = 1280 and
    more than 32 experts, here with 512 MiB of rows and more, a capacity that drops
    tuples, and padding that holds anything; 64-bit sums on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(T + masked)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    n = 2 * T - 5000                                    # kept tuples; 3000 rows behind them hold nothing
    rows = n + 3000
    src = torch.full((rows,), -5, dtype=torch.int32, device="cuda")
    src[:n] = torch.randperm(2 * T, generator=g, device="cuda")[:n].int()
    offsets = torch.full((E + 1,), n, dtype=torch.int64, device="cuda")
    dout, y, gates = rnd(T, d).to(bf), rnd(rows, d).to(bf), torch.rand(T, 2, generator=g, device="cuda")
    dxd, dl, w, x = rnd(rows, d).to(bf), rnd(T, E), (rnd(d, E) * d ** -0.5).to(bf), rnd(T, d).to(bf)
    valid, live = None, torch.ones(T, dtype=torch.bool, device="cuda")
    y[n:] = dxd[n:] = float("nan")
    if masked:
        valid = live = torch.rand(T, generator=g, device="cuda") < 0.8
        for t in (dout, x, dl):
            t[~valid] = float("nan")
        gates[~valid] = float("inf")
    assert (T + 2 * rows) * d * 2 >= 512 << 20 and (2 * T + rows) * d * 2 >= 512 << 20 or d == 512
    f = gpu.MoEGrad(T, d, E, rows=rows)
    dy = torch.full_like(y, 3.0)
    dy, dg, slot_of = f.combine(dout, y, gates, src, offsets, valid, dy=dy)
    assert bool((dy[n:] == 3).all())
    want_slot = torch.full((2 * T,), -1, dtype=torch.int32, device="cuda")
    want_slot[src[:n].long()] = torch.arange(n, device="cuda", dtype=torch.int32)
    assert torch.equal(slot_of.view(-1), want_slot)
    dx, dw = f.dispatch(dxd, dl, w, x, valid=valid)
    assert not dx[~live].any() and not dg[~live].any()
    want_dw, terms = (torch.zeros(d, E, dtype=torch.float64, device="cuda") for _ in range(2))
    zero = lambda t, v: torch.where(v[:, None], t, torch.zeros_like(t)).double()  # noqa: E731
    w64 = w.double().t().contiguous()
    for lo in range(0, T, 16384):
        hi = min(lo + 16384, T)
        v, s = live[lo:hi], slot_of[lo:hi].long()
        o, dl64, x64 = zero(dout[lo:hi], v), zero(dl[lo:hi], v), zero(x[lo:hi], v)
        part, size = dl64 @ w64, dl64.abs() @ w64.abs()
        add = torch.zeros_like(part)
        for j in range(2):
            have = s[:, j] >= 0
            at = s[:, j].clamp(min=0)
            yj, gj = zero(y[at], have & v), torch.where(v, gates[lo:hi, j], 0.0).double()[:, None]
            assert bool(((dg[lo:hi, j].double() - (o * yj).sum(1)).abs() <= 64 * U * (o * yj).abs().sum(1)).all())
            want = gj * o
            assert bool((((dy[at].double() - want).abs() <= (HALF + 2 * U) * want.abs() + 1e-38) | ~have[:, None]).all())
            r = zero(dxd[at], have & v)
            part += r
            add += r.abs()
        bound = 200 * U * size + 4 * U * add
        assert bool(((dx[lo:hi].double() - part).abs() <= bound + HALF * (part.abs() + bound) + 1e-38).all())
        want_dw += x64.t().contiguous() @ dl64
        terms += x64.abs().t().contiguous() @ dl64.abs()
    span = token_range(T, d)
    assert bool(((dw.double() - want_dw).abs() <= (48 * span // 64 + -(-T // span) + 8) * U * terms).all())


def test_missing_arguments_are_refused(gpu):
    s, _ = make(16, 256, 4, 0)
    f = gpu.MoEGrad(16, 256, 4)
    c = {n: None if t is None else t.cuda() for n, t in s.items()}
    args = ("dout", "y", "gates", "src_index", "offsets")
    for n in args:
        with pytest.raises(gpu.PwError):
            f.combine(*[None if m == n else c[m] for m in args])
    f.combine(*[c[m] for m in args])
    args = ("dxd", "dlogits", "w_router")
    for n in args:
        with pytest.raises(gpu.PwError):
            f.dispatch(*[None if m == n else c[m] for m in args])
