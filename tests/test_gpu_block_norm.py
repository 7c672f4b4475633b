"""GPU parity of the norms around a block (forward and gradients) against the
oracle in 64 bits.

Bars, with u = 2^-24 and e half a step of the rows' type (2^-8 or 2^-24): a
row's sums run over at most 32 elements of a thread, 6 lane exchanges and 4
waves, the products before and after them over fewer than 20 roundings, so
each term of a row's result is off by less than N = 64 u of its size, twice
that behind two norms; the weights' gradients add at most 256 more roundings (rows of a
team, teams, segments, partial rows).
"""
import numpy as np
import pytest
import torch

from oracle import block as ob

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5
HALF = 2.0 ** -8

# rows, d, dtype, gates, parts (y: block output, w: its norm, h: next norm)
CASES = [
    (1, 1, "f32", 0, "ywh"), (1, 1024, "bf16", 1, "ywh"), (3, 7, "bf16", 3, "ywh"), (5, 100, "f32", 0, "yh"),
    (40, 256, "bf16", 40, "ywh"), (33, 1000, "bf16", 0, "h"), (21, 1001, "bf16", 3, "ywh"), (17, 1001, "f32", 0, "yh"),
    (100, 1024, "f32", 4, "yw"), (64, 1280, "bf16", 2, "yh"), (9, 2048, "bf16", 1, "ywh"), (9, 2056, "bf16", 3, "ywh"),
    (6, 2049, "bf16", 0, "ywh"), (10, 4096, "bf16", 2, "ywh"), (7, 4100, "f32", 7, "ywh"), (5, 8192, "f32", 1, "ywh"),
    (4, 8192, "bf16", 0, "h"), (3, 8191, "bf16", 1, "ywh"), (20000, 64, "bf16", 2, "ywh"), (18001, 24, "f32", 0, "ywh"),
    (1300, 64, "bf16", 1300, "yh"), (2600, 40, "bf16", 1300, "ywh"), (4500, 520, "bf16", 5, "yw"), (300, 512, "bf16", 0, "y")]


def make(rows, d, dtype, gates, parts, seed=0):
    rng = np.random.default_rng([rows, d, gates, seed])
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32

    def t(*shape, scale=1.0, mean=0.0):
        return torch.from_numpy((rng.standard_normal(shape) * scale + mean).astype(np.float32)).to(dt)

    s = dict(x=t(rows, d, scale=3), y=t(rows, d, scale=2) if "y" in parts else None,
             w_y=t(d, scale=0.2, mean=1) if "w" in parts else None, gate=t(gates, d, scale=0.5) if gates else None,
             w_r=t(d, scale=0.2, mean=1) if "h" in parts else None, dr=t(rows, d), dh=t(rows, d) if "h" in parts else None)
    return s


def f64(t):
    return None if t is None else t.double().numpy()


def cuda(t):
    return None if t is None else t.cuda()


def half_step(dt):
    return torch.finfo(dt).eps / 2


def check_forward(got, s, ax, ay):
    x, y, w_y, gate, w_r = (f64(s[n]) for n in ("x", "y", "w_y", "gate", "w_r"))
    r, h, size = ob.block_norm(x, y, w_y, gate, w_r, ax, ay, EPS)
    e, N = half_step(s["x"].dtype), 64 * U
    gr, gh = (None if t is None else t.double().cpu().numpy() for t in got)
    if y is not None:
        assert np.all(np.abs(gr - r) <= N * size + e * np.abs(r) * (1 + N) + 1e-38)
    if w_r is not None:
        c = ob.rstd(r, EPS)
        off = np.sqrt((size ** 2).mean(axis=1, keepdims=True)) * c   # r's errors in its own norm
        assert np.all(np.abs(gh - h) <= N * (size * c * np.abs(w_r) + np.abs(h) * (1 + off)) + e * np.abs(h) * (1 + N) + 1e-38)


def check_grad(got, s, r, ax, ay, valid=None):
    a = {n: f64(s[n]) for n in ("dr", "dh", "y", "w_y", "gate", "w_r")}
    v = None if valid is None else valid.numpy()
    want, err = ob.block_norm_grad(r=f64(r), x_scale=ax, y_scale=ay, eps=EPS, valid=v, u=128 * U, **a)
    _, more = ob.block_norm_grad(r=f64(r), x_scale=ax, y_scale=ay, eps=EPS, valid=v, u=320 * U, **a)
    e = half_step(s["dr"].dtype)
    for name, t in zip(("dx", "dy", "dw_y", "dgate", "dw_r"), got):
        assert (t is None) == (name not in want), name
        if t is None:
            continue
        g = t.double().cpu().numpy()
        if name in ("dx", "dy"):
            bound = err[name] + e * (np.abs(want[name]) + err[name]) + 1e-38
        else:
            bound = more[name] + U * np.abs(want[name]) + 1e-38
        assert np.all(np.abs(g - want[name]) <= bound), (name, float((np.abs(g - want[name]) / bound).max()))


@pytest.mark.parametrize("rows,d,dtype,gates,parts", CASES)
def test_norm_and_gradients(gpu, rows, d, dtype, gates, parts):
    print(f"norm rows={rows} d={d} {dtype} gates={gates} {parts}", flush=True)
    ax, ay = 0.9, 0.7
    s = make(rows, d, dtype, gates, parts)
    f = gpu.BlockNorm(rows, d, gpu.PW_BF16 if dtype == "bf16" else gpu.PW_F32, gates, ax, ay, EPS)
    c = {n: cuda(t) for n, t in s.items()}
    got = f.forward(c["x"], y=c["y"], w_y=c["w_y"], gate=c["gate"], w_r=c["w_r"])
    check_forward(got, s, ax, ay)
    r = got[0] if got[0] is not None else (ax * s["x"].float()).to(s["x"].dtype).cuda()
    back = lambda: f.grad(c["dr"], c["dh"], r, y=c["y"], w_y=c["w_y"], gate=c["gate"], w_r=c["w_r"])  # noqa: E731
    check_grad(back(), s, r.cpu(), ax, ay)
    first = [None if t is None else t.clone() for t in back()]
    assert all(a is None or torch.equal(a, b) for a, b in zip(first, back()))   # equal inputs, equal bits
    if s["dh"] is not None:   # no gradient from the stream's other uses
        s["dr"] = torch.zeros_like(s["dr"])
        check_grad(f.grad(None, c["dh"], r, y=c["y"], w_y=c["w_y"], gate=c["gate"], w_r=c["w_r"]), s, r.cpu(), ax, ay)


def test_in_place(gpu):
    """r over x and dx over dr give the bits of separate buffers."""
    for d in (1024, 1001, 4096):
        s = make(500, d, "bf16", 5, "ywh")
        c = {n: cuda(t) for n, t in s.items()}
        f = gpu.BlockNorm(500, d, gpu.PW_BF16, 5, 0.9, 0.7, EPS)
        kw = dict(y=c["y"], w_y=c["w_y"], gate=c["gate"], w_r=c["w_r"])
        r, h = (t.clone() for t in f.forward(c["x"], **kw))
        dx = f.grad(c["dr"], c["dh"], r, **kw)[0].clone()
        x = c["x"].clone()
        r2, h2 = f.forward(x, r=x, **kw)
        assert r2 is x and torch.equal(r, r2) and torch.equal(h, h2)
        dr = c["dr"].clone()
        assert torch.equal(dx, f.grad(dr, c["dh"], r, dx=dr, **kw)[0])


EDGES = [(50, 127, "bf16", 0, "ywh"), (33, 129, "bf16", 3, "ywh"), (70, 9, "bf16", 0, "ywh"), (70, 8, "bf16", 7, "ywh"),
         (40, 7, "bf16", 0, "yw"), (3, 5, "f32", 0, "ywh"), (40, 3, "f32", 2, "ywh"), (1000, 15, "bf16", 8, "yh"),
         (5000, 65, "f32", 1, "ywh"), (40, 128, "f32", 4, "ywh"), (70, 256, "f32", 0, "h"), (31, 257, "bf16", 0, "ywh"),
         (31, 511, "f32", 31, "ywh"), (12, 513, "f32", 0, "yw"), (8, 1025, "bf16", 2, "y"), (6, 2047, "f32", 1, "ywh"),
         (6, 4095, "bf16", 3, "ywh"), (4, 4097, "bf16", 1, "yw"), (4, 4097, "f32", 2, "ywh"), (3, 8190, "f32", 0, "h")]


@pytest.mark.parametrize("rows,d,dtype,gates,parts", EDGES)
def test_widths_around_the_variants(gpu, rows, d, dtype, gates, parts):
    """Widths next to those where the number of threads changes, and rows whose
    last chunk is not whole."""
    test_norm_and_gradients(gpu, rows, d, dtype, gates, parts)


@pytest.mark.parametrize("parts", ["y", "yw", "yh"])
@pytest.mark.parametrize("d", [61, 509, 1001, 2001, 4095, 8191])
def test_in_place_with_a_part_of_a_chunk_left(gpu, d, parts):
    rows = 700
    s = make(rows, d, "bf16", 7, parts)
    c = {n: cuda(t) for n, t in s.items()}
    f = gpu.BlockNorm(rows, d, gpu.PW_BF16, 7, 0.9, 0.7, EPS)
    kw = dict(y=c["y"], w_y=c["w_y"], gate=c["gate"], w_r=c["w_r"])
    r = f.forward(c["x"], **kw)[0].clone()
    dx = f.grad(c["dr"], c["dh"], r, **kw)[0].clone()
    x, dr = c["x"].clone(), c["dr"].clone()
    assert torch.equal(r, f.forward(x, r=x, **kw)[0])
    assert torch.equal(dx, f.grad(dr, c["dh"], r, dx=dr, **kw)[0])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [128, 1003, 1024])
def test_gradient_of_rows_at_any_element(gpu, d, dtype):
    """Every row buffer begins one element after a 16-byte boundary, with a guard
    element before and after that stays as it was."""
    rows, ax, ay = 37, 0.9, 0.7
    s = make(rows, d, dtype, 0, "ywh")
    dt = s["x"].dtype

    def odd(t):
        flat = torch.full((t.numel() + 2,), 7.0, dtype=dt, device="cuda")
        v = flat[1:-1].view(t.shape)
        v.copy_(t)
        return v, flat
    c = {n: odd(t)[0] for n, t in s.items() if t is not None}
    f = gpu.BlockNorm(rows, d, gpu.PW_BF16 if dtype == "bf16" else gpu.PW_F32, 0, ax, ay, EPS)
    r, r_flat = odd(torch.zeros(rows, d))
    got = f.forward(c["x"], y=c["y"], w_y=c["w_y"], w_r=c["w_r"], r=r)
    check_forward(got, s, ax, ay)
    dx, dx_flat = odd(torch.zeros(rows, d))
    check_grad(f.grad(c["dr"], c["dh"], r, y=c["y"], w_y=c["w_y"], w_r=c["w_r"], dx=dx), s, r.cpu(), ax, ay)
    for flat in (r_flat, dx_flat):
        assert flat[0] == 7 and flat[-1] == 7


def test_rows_that_are_not_16_byte_aligned(gpu):
    rows, d = 30, 512
    s = make(rows, d, "bf16", 0, "ywh")
    flat = torch.zeros(rows * d + 1, dtype=torch.bfloat16, device="cuda")
    x = flat[1:].view(rows, d)
    x.copy_(cuda(s["x"]))
    f = gpu.BlockNorm(rows, d, gpu.PW_BF16, 0, 1.0, 1.0, EPS)
    check_forward(f.forward(x, y=cuda(s["y"]), w_y=cuda(s["w_y"]), w_r=cuda(s["w_r"])), s, 1.0, 1.0)


def test_padding_holds_anything(gpu):
    """Rows with valid 0 get zeros and leave the weights' gradients alone, whatever they hold."""
    for d in (1024, 1001, 4096):
        rows, gates = 120, 3
        s = make(rows, d, "bf16", gates, "ywh")
        valid = torch.ones(rows, dtype=torch.bool)
        valid[[0, 7, 41, 80, 119]] = False
        valid[40:80] = False                      # a gate without rows
        c = {n: cuda(t) for n, t in s.items()}
        r = s["x"].clone()
        for name in ("dr", "dh", "y"):
            c[name][~valid.cuda()] = float("nan")
        r[~valid] = float("inf")
        f = gpu.BlockNorm(rows, d, gpu.PW_BF16, gates, 0.9, 0.7, EPS)
        got = f.grad(c["dr"], c["dh"], r.cuda(), y=c["y"], w_y=c["w_y"], gate=c["gate"], w_r=c["w_r"], valid=valid.cuda())
        check_grad(got, s, r, 0.9, 0.7, valid)
        assert not got[0][~valid.cuda()].any() and not got[1][~valid.cuda()].any() and not got[3][1].any()


def test_offsets_past_32_bits(gpu):
    """More than 2^32 elements a tensor: the last rows as in a call of their own."""
    rows, d, k = 1060000, 4104, 24
    assert rows * d > 1 << 32
    s = make(k, d, "bf16", 0, "ywh")
    c = {n: cuda(t) for n, t in s.items()}
    kw = dict(w_y=c["w_y"], w_r=c["w_r"])

    def long(t):
        z = torch.zeros(rows, d, dtype=t.dtype, device="cuda")
        z[-k:] = t
        return z

    big, small = gpu.BlockNorm(rows, d, eps=EPS), gpu.BlockNorm(k, d, eps=EPS)
    x, y = long(c["x"]), long(c["y"])
    r, h = big.forward(x, y=y, r=x, **kw)
    r2, h2 = small.forward(c["x"], y=c["y"], **kw)
    assert torch.equal(r[-k:], r2) and torch.equal(h[-k:], h2) and not h[:rows - k].any()
    h.zero_()
    h[-k:] = c["dh"]
    dr = long(c["dr"])
    got = big.grad(dr, h, r, y=y, dx=dr, **kw)
    one = small.grad(c["dr"], c["dh"], r2, y=c["y"], **kw)
    assert torch.equal(got[0][-k:], one[0]) and torch.equal(got[1][-k:], one[1]) and not got[1][:rows - k].any()
    s["gate"] = None
    check_grad((one[0], one[1], got[2], None, got[4]), s, r2.cpu(), 1.0, 1.0)


def test_more_rows_than_a_grid_has_threads(gpu):
    """70 million short rows: the workgroups walk on."""
    rows, d = 70_000_000, 2
    assert rows // 4 * 256 >= 1 << 32
    s = make(1000, d, "bf16", 0, "ywh")
    c = {n: cuda(t) for n, t in s.items()}
    x, y = c["x"].repeat(rows // 1000, 1), c["y"].repeat(rows // 1000, 1)
    r, h = gpu.BlockNorm(rows, d, eps=EPS).forward(x, y=y, w_y=c["w_y"], w_r=c["w_r"])
    r2, h2 = gpu.BlockNorm(1000, d, eps=EPS).forward(c["x"], y=c["y"], w_y=c["w_y"], w_r=c["w_r"])
    check_forward((r2, h2), s, 1.0, 1.0)
    assert bool((r.view(-1, 1000, d) == r2).all()) and bool((h.view(-1, 1000, d) == h2).all())


def test_zero_rows_and_zero_vectors(gpu):
    f = gpu.BlockNorm(0, 64, gpu.PW_F32, 2)
    e, w, g = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda"), torch.ones(2, 64, device="cuda")
    r, h = f.forward(e, y=e, w_y=w, gate=g, w_r=w)
    assert r.shape == (0, 64) and h.shape == (0, 64)
    for t in f.grad(e, e, e, y=e, w_y=w, gate=g, w_r=w)[2:]:
        assert not t.any()
    f = gpu.BlockNorm(3, 64, gpu.PW_F32)
    z = torch.zeros(3, 64, device="cuda")
    r, h = f.forward(z, y=z, w_y=w, w_r=w)
    assert not r.any() and not h.any()
    assert all(torch.isfinite(t).all() for t in f.grad(torch.ones_like(z), z + 1, z, y=z, w_y=w, w_r=w) if t is not None)


def test_a_replayed_graph_and_another_stream(gpu):
    rows, d, gates, ax, ay = 3000, 640, 3, 1.0, 0.5
    f = gpu.BlockNorm(rows, d, gpu.PW_BF16, gates, ax, ay, EPS)
    data = [make(rows, d, "bf16", gates, "ywh", seed) for seed in range(4)]
    c = {n: cuda(t) for n, t in data[0].items()}

    def step(stream=None):
        r, h = f.forward(c["x"], y=c["y"], w_y=c["w_y"], gate=c["gate"], w_r=c["w_r"], stream=stream)
        return r, h, f.grad(c["dr"], c["dh"], r, y=c["y"], w_y=c["w_y"], gate=c["gate"], w_r=c["w_r"], stream=stream)

    step()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r, h, back = step()
    for s in data[1:] + data[:1]:
        for n, t in s.items():
            c[n].copy_(cuda(t))
        graph.replay()
        torch.cuda.synchronize()
        check_forward((r, h), s, ax, ay)
        check_grad(back, s, r.cpu(), ax, ay)
    side.wait_stream(torch.cuda.current_stream())
    r, h, back = step(side)
    side.synchronize()
    check_grad(back, s, r.cpu(), ax, ay)


def test_refusals(gpu):
    f = gpu.BlockNorm(8, 64, gpu.PW_BF16, 2)
    x, w = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(2, 64, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(w_r=w), dict(y=x, w_r=w), dict(y=x, gate=g[:1], w_r=w), dict(y=x.float(), gate=g),
               dict(y=x[:, :32], gate=g), dict(y=x, gate=g, w_r=w[:63]), dict(y=x.t().contiguous().t(), gate=g)):
        with pytest.raises(gpu.PwError):
            f.forward(x, **kw)
    with pytest.raises(gpu.PwError):
        f.grad(x, y=x, gate=g, w_r=w)                 # no dh, no r
    with pytest.raises(gpu.PwError):
        gpu.BlockNorm(8, 64, gates=3)


@pytest.mark.parametrize("rows,d,parts", [(1 << 29, 8, "ywh"), (1 << 22, 1025, "yw")])
def test_gradients_of_many_equal_rows(gpu, rows, d, parts):
    """Thousands of equal rows for each workgroup, where fp32 additions err to the
    same side: the weights' sums stay within 512 additions in a chain. Bar: a term
    by 128 u, those additions, 112 more across teams and partial rows."""
    s = make(1, d, "bf16", 0, parts)
    s["x"] = None
    if "h" in parts:
        s["dr"], s["r"] = None, make(1, d, "bf16", 0, parts, 1)["x"]
    long = {n: t if t is None or t.dim() == 1 else cuda(t).expand(rows, d).contiguous() for n, t in s.items()}
    f = gpu.BlockNorm(rows, d, eps=EPS)
    got = f.grad(long["dr"], long["dh"], long.get("r"), y=long["y"], w_y=cuda(s["w_y"]), w_r=cuda(s["w_r"]))
    a = {n: f64(s[n]) for n in ("dr", "dh", "y", "w_y", "w_r")}
    one = dict(r=f64(s.get("r")), x_scale=1.0, y_scale=1.0, eps=EPS, gate=None)
    want, err = ob.block_norm_grad(u=128 * U, **a, **one)
    _, more = ob.block_norm_grad(u=(128 + 512 + 112) * U, **a, **one)
    for name, t in zip(("dx", "dy"), got):
        assert bool((t == t[0]).all())
        bound = err[name] + HALF * (np.abs(want[name]) + err[name]) + 1e-38
        assert np.all(np.abs(f64(t[:1].cpu()) - want[name]) <= bound)
    for name, t in (("dw_y", got[2]), ("dw_r", got[4])):
        assert (t is None) == (name not in want)
        if t is not None:
            off = np.abs(f64(t.cpu()) / rows - want[name])
            print(name, float((off / (more[name] + U * np.abs(want[name]))).max()), flush=True)
            assert np.all(off <= more[name] + U * np.abs(want[name]))


def test_more_gates_in_segments_than_a_grid_is_high(gpu):
    """66000 gates of 16384 rows, each in two segments: the join is two grids deep. Whole
    numbers, so that the sums are exact."""
    gates, group = 66000, 16384
    rows = gates * group
    y = torch.ones(rows, 1, dtype=torch.bfloat16, device="cuda")
    dr = torch.ones_like(y)
    k = torch.arange(gates, device="cuda") % 5
    dr.view(gates, group)[:, -3:] = k[:, None].to(torch.bfloat16)
    gate = (1 + torch.arange(gates, device="cuda") % 3).to(torch.bfloat16)[:, None]
    f = gpu.BlockNorm(rows, 1, gates=gates, eps=EPS)
    dx, dy, _, dgate, _ = f.grad(dr, y=y, gate=gate)
    assert torch.equal(dgate[:, 0], (group - 3 + 3 * k).float())
    assert torch.equal(dx, dr) and torch.equal(dy.view(gates, group), dr.view(gates, group) * gate)


@pytest.mark.parametrize("dtype,d", [("f32", 5), ("f32", 1001), ("bf16", 64), ("bf16", 1024)])
def test_the_smallest_eps(gpu, dtype, d):
    """eps below the normal numbers, next to rows of zeros: 1 / sqrt(eps) is finite,
    its square is not. Bar: as elsewhere."""
    rows, eps = 40, float(np.float32(1e-40))
    s = make(rows, d, dtype, 0, "ywh")
    zero = torch.arange(rows) % 3 == 0
    c = {n: cuda(t) for n, t in s.items()}
    x, y = c["x"].clone(), c["y"].clone()
    x[zero.cuda()], y[zero.cuda()] = 0, 0
    f = gpu.BlockNorm(rows, d, gpu.PW_BF16 if dtype == "bf16" else gpu.PW_F32, 0, 1.0, 1.0, eps)
    e = half_step(s["x"].dtype)
    v = dict(valid=None, x_scale=1.0, y_scale=1.0, eps=eps, gate=None, u=128 * U)
    dx, dy, dw_y = (t.clone() for t in f.grad(c["dr"], y=y, w_y=c["w_y"])[:3])
    want, err = ob.block_norm_grad(f64(s["dr"]), None, None, f64(y.cpu()), f64(s["w_y"]), w_r=None, **v)
    hx, _, _, _, dw_r = f.grad(None, c["dh"], x, w_r=c["w_r"])
    want2, err2 = ob.block_norm_grad(None, f64(s["dh"]), f64(x.cpu()), None, None, w_r=f64(s["w_r"]), **v)
    assert float(np.abs(want["dy"][zero.numpy()]).max()) > 1e19
    for got, w, b in ((dx, want["dx"], err["dx"]), (dy, want["dy"], err["dy"]), (hx, want2["dx"], err2["dx"])):
        assert np.all(np.abs(f64(got.cpu()) - w) <= b + e * (np.abs(w) + b) + 1e-38)
    for got, w, b in ((dw_y, want["dw_y"], err["dw_y"]), (dw_r, want2["dw_r"], err2["dw_r"])):
        assert np.all(np.abs(f64(got.cpu()) - w) <= 3 * b + U * np.abs(w) + 1e-38)
    r, h = f.forward(x, y=y, w_y=c["w_y"], w_r=c["w_r"])
    assert not r[zero.cuda()].any() and not h[zero.cuda()].any() and bool(torch.isfinite(h).all())


@pytest.mark.parametrize("parts", ["y", "yw", "yh", "ywh"])
@pytest.mark.parametrize("d", [513, 519, 1025, 1031, 1537, 2049, 4097])
def test_in_place_where_two_waves_share_elements(gpu, d, parts):
    """bf16 rows whose last chunk, moved back, begins in the last chunk of the wave
    before: ceil(d / 8) = 64 n + 1. Both waves write those elements, and neither may
    do so before the other has read them."""
    assert -(-d // 8) % 64 == 1
    rows = 6000
    s = make(rows, d, "bf16", 6, parts)
    c = {n: cuda(t) for n, t in s.items()}
    f = gpu.BlockNorm(rows, d, gpu.PW_BF16, 6, 0.9, 0.7, EPS)
    kw = dict(y=c["y"], w_y=c["w_y"], gate=c["gate"], w_r=c["w_r"])
    r, h = (None if t is None else t.clone() for t in f.forward(c["x"], **kw))
    back = [None if t is None else t.clone() for t in f.grad(c["dr"], c["dh"], r, **kw)]
    few = slice(0, 1000 * 6, 1000)   # a row of each gate against the oracle
    some = {n: t if t is None or n in ("w_y", "w_r", "gate") else t[few] for n, t in s.items()}
    check_forward((r[few], None if h is None else h[few]), some, 0.9, 0.7)
    same = lambda a, b: (a is None and b is None) or torch.equal(a, b)  # noqa: E731
    for _ in range(3):
        x, dr = c["x"].clone(), c["dr"].clone()
        r2, h2 = f.forward(x, r=x, **kw)
        assert r2 is x and same(r, r2) and same(h, h2)
        assert all(same(a, b) for a, b in zip(back, f.grad(dr, c["dh"], r, dx=dr, **kw)))
