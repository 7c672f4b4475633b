"""GPU parity of the 8-bit rows, the experts' products and the combine against
the oracle in 64 bits.

Codes and scales are equal bit for bit. Bars, with u = 2^-24: a product's sum is
exact, its conversion and the two scales round three times, 3 u of z; GELU
carries a relative error of z on as at most z^2 + 2 times itself (its slope over
its value), and its own is 5.1e-5 in bf16 (8 u of the error function in fp32, whose
rounded argument counts z^2 times); the result is rounded once, by half a step
of its type. The combine's sum of k + 1 terms is off by (k + 2) u of their
absolute values.
"""
import numpy as np
import pytest
import torch

from oracle import experts as ox

pytestmark = pytest.mark.gpu
U = ox.U
HALF = {"bf16": 2.0 ** -8, "f32": U}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def pwt(gpu, dtype):
    return gpu.PW_BF16 if dtype == "bf16" else gpu.PW_F32


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def rows_of(rng, rows, d, dtype, scale=1.0):
    """Random rows as the type holds them (fp32 array)."""
    x = torch.from_numpy((rng.standard_normal((rows, d)) * scale).astype(np.float32))
    return x.to(DT[dtype]).float().numpy()


# ---- rows as codes ------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (5, 64), (70, 65), (300, 128), (33, 200), (64, 1000), (257, 1024),
                                    (9, 2048), (20, 2049), (1001, 120), (401, 250), (130, 500), (70, 1500), (5, 4096), (7, 8191), (3, 8192), (2, 12345), (2, 65536)])
def test_codes_are_equal(gpu, rows, d, dtype):
    print(f"quant {rows} x {d} {dtype}", flush=True)
    rng = np.random.default_rng([rows, d])
    x = rows_of(rng, rows, d, dtype, 3.0)
    x[:, d // 2] = x[:, 0] / 2  # the middle of two codes, where the scale rounds evenly
    x = torch.from_numpy(x).to(DT[dtype]).float().numpy()
    q, s = gpu.RowQuant(rows, d, pwt(gpu, dtype)).forward(dev(x, DT[dtype]))
    wq, ws = ox.quant(x)
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q.cpu().numpy(), wq)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [40, 1024, 9000])
def test_codes_of_ties_zeros_and_extremes(gpu, d, dtype):
    rng = np.random.default_rng(d)
    x = rows_of(rng, 16, d, dtype)
    x[0] = 0
    x[1] = 0
    x[1, d - 1] = 1e-45 if dtype == "f32" else 2.0 ** -133
    x[2] *= 1e-37
    x[3, 5] = np.inf
    x[4, d - 1] = -np.inf
    x[5, 0] = np.nan
    x[6] = -np.float32(3.0e38)
    x[7] *= 1e37
    m = rng.integers(-254, 255, d)
    x[8], x[8, 0] = m * 0.5, 127               # every half
    x[9], x[9, 0] = m * 0.25, 254 * 0.25       # amax / 2 and the like
    x[10], x[10, 0] = m * 2.0 ** -130, 254 * 2.0 ** -130
    x[11] = 2.0 ** -126 * np.sign(x[11])
    x = torch.from_numpy(x).to(DT[dtype]).float().numpy()
    q, s = gpu.RowQuant(16, d, pwt(gpu, dtype)).forward(dev(x, DT[dtype]))
    wq, ws = ox.quant(x)
    assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), wq)


def test_codes_up_to_a_limit_and_unaligned_rows(gpu):
    rng = np.random.default_rng(1)
    x = rows_of(rng, 50, 131, "bf16")
    flat = torch.zeros(50 * 131 + 1, dtype=torch.bfloat16, device="cuda")
    X = flat[1:].view(50, 131)
    X.copy_(dev(x))
    wq, ws = ox.quant(x)
    for limit in (-3, 0, 1, 20, 50, 1 << 40):
        q = torch.full((50, 192), 99, dtype=torch.int8, device="cuda")
        s = torch.full((50,), -1.0, device="cuda")
        gpu.RowQuant(50, 131).forward(X, limit=torch.tensor([limit], device="cuda"), q=q, scale=s)
        n = min(max(limit, 0), 50)
        assert np.array_equal(q.cpu().numpy()[:n], wq[:n]) and np.array_equal(s.cpu().numpy()[:n], ws[:n])
        assert bool((q[n:] == 99).all()) and bool((s[n:] == -1).all())


# ---- products -----------------------------------------------------------------

def weights(gpu, rng, E, n, d):
    w = (rng.standard_normal((E * n, d)) * d ** -0.5).astype(np.float32)
    wq, ws = ox.quant(w)
    return wq.reshape(E, n, -1), ws.reshape(E, n)


def route(rng, T, k, E, kind):
    """offsets, src_index of T k tuples: some experts popular, some without any; the last tuples are padding's."""
    p = np.linspace(3, 0, E) ** 2 if kind == "skewed" else np.ones(E)
    dest = rng.choice(E, T * k, p=p / p.sum())
    if kind == "padded":
        dest = np.where(rng.random(T * k) < 0.3, E, dest)
    if kind == "one":
        dest[:] = E - 1
    off = np.concatenate([[0], np.cumsum(np.bincount(dest, minlength=E + 1)[:E])])
    return off, np.argsort(dest, kind="stable").astype(np.int32)


def check_product(got, want, pre, dtype, act):
    e = 3 * U
    if act:
        e = e * (pre ** 2 + 2) + (5.2e-5 if dtype == "bf16" else (8 + 3 * pre ** 2) * U)
    ok = np.abs(got.cpu().double().numpy() - want) <= np.abs(want) * (HALF[dtype] + 1.01 * e) + 1e-37
    assert ok.all(), np.argwhere(~ok)[:5]


# tokens, k, experts, d, n, kind, gather, scatter, act, dtype
CASES = [(1, 1, 1, 1, 1, "even", True, False, False, "f32"), (1, 8, 16, 64, 64, "even", True, False, True, "bf16"),
         (3, 2, 4, 100, 70, "one", True, True, False, "bf16"), (16, 2, 8, 128, 256, "even", False, True, False, "bf16"),
         (17, 1, 1, 64, 16, "even", False, False, True, "f32"), (48, 8, 64, 256, 128, "skewed", True, False, True, "bf16"),
         (65, 4, 5, 333, 131, "padded", False, True, True, "bf16"), (100, 3, 5, 200, 77, "skewed", True, True, True, "f32"),
         (128, 1, 1, 512, 384, "even", False, False, False, "bf16"), (200, 2, 256, 64, 96, "even", True, False, False, "bf16"),
         (300, 2, 7, 1000, 515, "padded", True, False, True, "f32"), (500, 2, 3, 192, 264, "skewed", False, True, True, "bf16"),
         (700, 4, 2, 128, 128, "one", True, False, False, "bf16"), (1025, 1, 1, 640, 512, "even", False, False, True, "bf16"),
         (1500, 2, 4, 320, 513, "skewed", True, False, False, "bf16"), (1111, 2, 6, 130, 520, "padded", False, True, False, "f32"),
         (2048, 2, 3, 256, 768, "padded", True, True, True, "bf16"), (4000, 1, 1, 448, 250, "even", False, False, False, "bf16"),
         (3000, 2, 8, 512, 512, "skewed", True, False, True, "bf16"),
         (40, 8, 64, 2100, 600, "skewed", True, False, True, "bf16"), (60, 4, 40, 4096, 777, "padded", False, True, False, "f32"),
         (30, 1, 1, 4000, 700, "even", False, False, False, "bf16"), (90, 2, 3, 2048, 128, "padded", True, False, True, "bf16"),
         (8, 1, 1, 4096, 300, "even", False, False, True, "f32"), (2, 4, 8, 1500, 100, "even", True, False, False, "bf16"),
         (4, 2, 6, 2500, 96, "one", False, True, True, "bf16"), (2, 4, 8, 700, 9, "even", True, True, False, "bf16"),
         (2100, 1, 1, 2112, 1000, "even", False, False, True, "bf16"), (1000, 4, 20, 2304, 700, "skewed", False, True, False, "f32"),
         (1, 7, 64, 1100, 37, "padded", True, False, True, "f32"), (8, 1, 3, 3000, 21, "skewed", False, True, False, "bf16"), (600, 1, 1, 1000, 2000, "even", False, False, True, "bf16")]


@pytest.mark.parametrize("T,k,E,d,n,kind,gather,scatter,act,dtype", CASES)
def test_product(gpu, T, k, E, d, n, kind, gather, scatter, act, dtype):
    print(f"product T={T} k={k} E={E} d={d} n={n} {kind} gather={gather} scatter={scatter} {dtype}", flush=True)
    rng = np.random.default_rng([T, k, E, d, n])
    rows = T * k
    w, ws = weights(gpu, rng, E, n, d)
    off, src = route(rng, T, k, E, kind) if E > 1 else (None, None)
    indexed = E > 1 and (gather or scatter)
    gather = k if indexed and gather else 0
    scatter = indexed and scatter
    x = rows_of(rng, T if gather else rows, d, dtype)
    W, WS = dev(w), dev(ws)
    f = gpu.Int8Product(W, WS, d, rows, gather=gather, scatter=scatter, gelu=act, dtype=pwt(gpu, dtype))
    out = torch.full((rows, n), 7.0, dtype=DT[dtype], device="cuda")
    q, s = ox.quant(x)
    want, pre = ox.product(q, s, w, ws, off, src if indexed else None, rows, gather, scatter, act, np.full((rows, n), 7.0))
    kw = dict(offsets=None if off is None else dev(off), src_index=dev(src) if indexed else None)
    check_product(f.forward(dev(x, DT[dtype]), out=out, **kw), want, pre, dtype, act)
    first = out.clone()
    # codes given: the same bits; a kept buffer
    out.fill_(7.0)
    got = f.forward(dev(q), x_scale=dev(s), out=out, **kw)
    assert got is out and torch.equal(got, first)
    assert f.forward(dev(x, DT[dtype]), **kw).shape == (rows, n)


@pytest.mark.parametrize("T,k,E,d,n,kind,gather,scatter,act,dtype",
                         [(5500, 2, 5, 192, 6500, "skewed", True, False, True, "bf16"), (6000, 2, 3, 64, 6144, "padded", False, True, False, "f32"),
                          (20000, 1, 1, 512, 4096, "even", False, False, True, "bf16"), (4000, 8, 130, 320, 2500, "skewed", True, True, False, "bf16"),
                          (70000, 1, 2, 100, 1030, "one", False, True, False, "bf16"), (17000, 2, 64, 1024, 2048, "padded", True, False, True, "f32"),
                          (9000, 2, 5, 700, 1030, "skewed", True, False, True, "bf16"), (16000, 1, 1, 1152, 2049, "even", False, False, False, "bf16"),
                          (33000, 2, 5, 640, 4096, "padded", True, True, False, "bf16"), (33000, 2, 3, 576, 2080, "skewed", False, True, True, "f32"),
                          (8000, 2, 2, 640, 2060, "padded", True, False, False, "f32"), (9000, 1, 1, 600, 3000, "even", False, False, True, "bf16")])
def test_many_tiles(gpu, T, k, E, d, n, kind, gather, scatter, act, dtype):
    """As test_product at sizes where workgroups walk over tiles; the plain form in 64 bits by torch, on the GPU."""
    print(f"product T={T} k={k} E={E} d={d} n={n} {kind} gather={gather} scatter={scatter} {dtype}", flush=True)
    rng = np.random.default_rng([T, k, E, d, n])
    rows = T * k
    w, ws = weights(gpu, rng, E, n, d)
    off, src = route(rng, T, k, E, kind) if E > 1 else (np.array([0, rows]), np.arange(rows, dtype=np.int32))
    x = rows_of(rng, T if gather else rows, d, dtype)
    q, s = (dev(t) for t in ox.quant(x))
    W, WS, S = dev(w), dev(ws), dev(src).long()
    f = gpu.Int8Product(W, WS, d, rows, gather=k if gather else 0, scatter=scatter, gelu=act, dtype=pwt(gpu, dtype))
    out = torch.full((rows, n), 7.0, dtype=DT[dtype], device="cuda")
    f.forward(q, x_scale=s, out=out, offsets=None if E == 1 else dev(off), src_index=dev(src) if gather or scatter else None)
    again = torch.full_like(out, 7.0)
    f.forward(dev(x, DT[dtype]), out=again, offsets=None if E == 1 else dev(off), src_index=dev(src) if gather or scatter else None)
    assert torch.equal(out, again)
    seen = torch.zeros(rows, dtype=torch.bool, device="cuda")
    for e in range(E):
        i = torch.arange(int(off[e]), int(off[e + 1]), device="cuda")
        for i in i.split(8192):
            a = S[i] // k if gather else i
            o = S[i] if scatter else i
            z = (q[a].double() @ W[e].double().t().contiguous()) * s[a].double().unsqueeze(1) * WS[e].double()
            want = z * 0.5 * torch.special.erfc(-z * 0.5 ** 0.5) if act else z
            err = 3 * U * (z * z + 2 if act else 1) + ((5.2e-5 if dtype == "bf16" else (8 + 3 * z * z) * U) if act else 0)
            bad = (out[o].double() - want).abs() > want.abs() * (HALF[dtype] + 1.01 * err) + 1e-37
            assert not bool(bad.any()), (e, bad.nonzero()[:5])
            seen[o] = True
    assert bool((out[~seen] == 7.0).all()) and int(seen.sum()) == int(off[E])


@pytest.mark.parametrize("n,T", [(64, 60), (130, 60), (256, 60), (21, 4), (4096, 4500)])
@pytest.mark.parametrize("E", [3, 70])
def test_offsets_and_indexes_that_are_none(gpu, n, E, T):
    """Descending, negative and far offsets, ids outside the tuples: nothing out of range is read or written, no row twice."""
    rng = np.random.default_rng(n)
    k, d = 2, 96
    rows = T * k
    w, ws = weights(gpu, rng, E, n, d)
    x = rows_of(rng, T, d, "bf16")
    q, s = ox.quant(x)
    src = rng.permutation(rows).astype(np.int32)
    src[::7] = -1
    src[3::11] = 1 << 30
    src[4::13] = rows
    for off in ([0, 50, 40, 200], [-5, 10, 100, 1 << 40], [60, 60, 60, 60], [3, 100, 1 << 33, 7], [0, 5, rows + 9, -1]):
        off = np.array(off + [off[-1]] * (E - 3), np.int64)
        for gather, scatter in ((k, False), (k, True), (0, True)):
            xs = x if gather else np.concatenate([x, x])
            f = gpu.Int8Product(dev(w), dev(ws), d, rows, gather=gather, scatter=scatter)
            out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
            f.forward(dev(xs, torch.bfloat16), offsets=dev(off), src_index=dev(src), out=out)
            qq, ss = ox.quant(xs)
            want, pre = ox.product(qq, ss, w, ws, off, src, rows, gather, scatter, False, np.full((rows, n), 7.0))
            check_product(out, want, pre, "bf16", False)


def test_scales_that_are_not_numbers_and_zero_rows(gpu):
    rng = np.random.default_rng(2)
    x = rows_of(rng, 40, 80, "bf16")
    x[3], x[5, 7], x[6, 0] = 0, np.inf, np.nan
    w, ws = weights(gpu, rng, 1, 50, 80)
    ws[0, 9] = np.inf
    out = gpu.Int8Product(dev(w), dev(ws), 80, 40).forward(dev(x, torch.bfloat16)).float().cpu().numpy()
    assert np.isnan(out[[5, 6]]).all() and np.isnan(out[3, 9]) and not out[3, :9].any()
    clean = np.delete(np.delete(out, [3, 5, 6], 0), 9, 1)
    assert np.isfinite(clean).all()


def test_the_largest_sums(gpu):
    """Every code at its limit over the widest row: the sum needs all 31 bits' worth of room that there is."""
    d, n = 65536, 20
    w = np.full((1, n, d), 127, np.int8)
    w[0, 1] = -127
    x = np.ones((3, d), np.float32)
    x[1] = -1
    out = gpu.Int8Product(dev(w), dev(np.ones((1, n), np.float32)), d, 3, dtype=gpu.PW_F32).forward(dev(x)).cpu().numpy()
    top = np.float32(127 * 127 * 65536) * (np.float32(1) / np.float32(127))
    assert np.all(np.abs(np.abs(out) - top) <= 2 * U * top) and out[0, 0] > 0 > out[0, 1] and out[1, 0] < 0 < out[1, 1]


def test_offsets_past_32_bits(gpu):
    """Outputs, codes and weights beyond 2^32 bytes; the last rows alone are computed."""
    rng = np.random.default_rng(4)
    T, d, n, E = 2400000, 1024, 1024, 3
    w, ws = weights(gpu, rng, E, n, d)
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    last = rows_of(rng, 50, d, "bf16")
    x[-50:] = dev(last, torch.bfloat16)
    off = torch.tensor([T - 50, T - 50, T - 20, T], device="cuda")
    f = gpu.Int8Product(dev(w), dev(ws), d, T)
    out = torch.zeros(T, n, dtype=torch.bfloat16, device="cuda")
    f.forward(x, offsets=off, out=out)
    q, s = ox.quant(last)
    want, pre = ox.product(q, s, w, ws, np.array([0, 0, 30, 50]), None, 50)
    check_product(out[-50:], want, pre, "bf16", False)
    assert float(out[:-50].abs().max()) == 0


def test_product_refusals(gpu):
    w, ws = torch.zeros(4, 32, 128, dtype=torch.int8, device="cuda"), torch.zeros(4, 32, device="cuda")
    with pytest.raises(gpu.PwError):
        gpu.Int8Product(w, ws, 200, 8)           # rows of codes of another length
    with pytest.raises(gpu.PwError):
        gpu.Int8Product(w.float(), ws, 100, 8)
    with pytest.raises(gpu.PwError):
        gpu.Int8Product(w, ws[:3], 100, 8)
    with pytest.raises(gpu.PwError):
        gpu.Int8Product(w[0], ws, 100, 8)
    f = gpu.Int8Product(w, ws, 100, 8)
    x = torch.zeros(8, 100, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(), dict(offsets=torch.zeros(4, dtype=torch.int64, device="cuda")),
               dict(offsets=torch.zeros(5, dtype=torch.int32, device="cuda")),
               dict(offsets=torch.zeros(5, dtype=torch.int64, device="cuda"),
                    src_index=torch.zeros(8, dtype=torch.int32, device="cuda"))):
        with pytest.raises(gpu.PwError):
            f.forward(x, **kw)
    with pytest.raises(gpu.PwError):
        f.forward(x.float(), offsets=torch.zeros(5, dtype=torch.int64, device="cuda"))
    none = gpu.Int8Product(w, ws, 100, 0).forward(x[:0], offsets=torch.zeros(5, dtype=torch.int64, device="cuda"))
    assert none.shape == (0, 32)


# ---- combine ------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,k", [(1, 1, 1), (1, 1024, 8), (3, 7, 2), (48, 1024, 8), (100, 130, 3), (257, 64, 6), (33, 4096, 5),
                                   (500, 1001, 4), (2, 65536, 2), (1000, 24, 7), (4099, 256, 2)])
def test_combine(gpu, T, d, k, dtype):
    print(f"combine {T} x {k} x {d} {dtype}", flush=True)
    rng = np.random.default_rng([T, d, k])
    y, add = rows_of(rng, T * k, d, dtype), rows_of(rng, T, d, dtype)
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[rng.random((T, k)) < 0.2] = 0
    if T > 1:
        w[1] = 0
    y[(w == 0).reshape(-1)] = np.nan            # what nothing wrote
    f = gpu.TopkCombine(T, d, k, pwt(gpu, dtype))
    for a in (None, add):
        got = f.forward(dev(y, DT[dtype]), dev(w), add=None if a is None else dev(a, DT[dtype]))
        want, size = ox.combine(y, w, a)
        assert np.all(np.abs(got.cpu().double().numpy() - want) <= (k + 2) * U * size + HALF[dtype] * np.abs(want) * 1.01 + 1e-37)
    out = dev(add, DT[dtype])
    assert f.forward(dev(y, DT[dtype]), dev(w), add=out, out=out) is out and torch.equal(out, got)


def test_combine_of_unaligned_rows_and_far_ones(gpu):
    rng = np.random.default_rng(6)
    T, d, k = 30, 72, 3
    y = rows_of(rng, T * k, d, "bf16")
    w = rng.standard_normal((T, k)).astype(np.float32)
    flat = torch.zeros(T * k * d + 1, dtype=torch.bfloat16, device="cuda")
    flat[1:] = dev(y, torch.bfloat16).view(-1)
    got = gpu.TopkCombine(T, d, k).forward(flat[1:].view(T * k, d), dev(w))
    want, size = ox.combine(y, w, None)
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= (k + 2) * U * size + HALF["bf16"] * np.abs(want) * 1.01)
    T, d, k = 1100000, 1024, 4                  # more than 2^32 elements
    far = torch.zeros(T * k, d, dtype=torch.bfloat16, device="cuda")
    far[-k:] = 1.0
    out = gpu.TopkCombine(T, d, k).forward(far, torch.full((T, k), 0.25, device="cuda"))
    assert float(out[-1].float().min()) == 1.0 and float(out[:-1].float().abs().max()) == 0


# ---- together -------------------------------------------------------------------

@pytest.mark.parametrize("T,E,k,d,hidden,masked", [(1, 8, 8, 256, 512, False), (40, 16, 4, 192, 320, True), (600, 64, 6, 256, 384, True)])
def test_route_order_products_and_combine(gpu, T, E, k, d, hidden, masked):
    """A token's way: routing, the exchange that orders its tuples (padding behind the last expert), both products, the combine."""
    rng = np.random.default_rng([T, E, k])
    l = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    valid = rng.random(T) < 0.8 if masked else None
    x, shared = rows_of(rng, T, d, "bf16"), rows_of(rng, T, d, "bf16")
    w1, s1 = weights(gpu, rng, E, hidden, d)
    w2, s2 = weights(gpu, rng, E, d, hidden)
    rows = T * k
    router = gpu.Router(T, E, k, "sigmoid", groups=4, top_groups=4, scale=2.0)
    order = gpu.Exchange(E + 1, rows, 1, num_src_shards=1)
    first = gpu.Int8Product(dev(w1), dev(s1), d, rows, gather=k, gelu=True)
    second = gpu.Int8Product(dev(w2), dev(s2), hidden, rows, scatter=True)
    join = gpu.TopkCombine(T, d, k)
    y = torch.full((rows, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    experts, wt = router.forward(dev(l), bias=dev(bias), valid=None if valid is None else dev(valid))
    gpu.future_wait(order.step(wt.view(rows, 1), experts.view(rows)))
    off = order.offsets[:E + 1]
    h = first.forward(dev(x, torch.bfloat16), offsets=off, src_index=order.src_index)
    second.forward(h, offsets=off, src_index=order.src_index, out=y)
    out = join.forward(y, wt, add=dev(shared, torch.bfloat16)).float().cpu().numpy()
    ids, w = ox.route(l, bias, valid, k, True, 4, 4, 2, True, 2.0)
    assert np.array_equal(experts.cpu().numpy(), ids)
    # the oracle's way, tuple by tuple, from the GPU's hidden rows as they are rounded
    q, s = ox.quant(x)
    src = np.argsort(ids.reshape(-1), kind="stable").astype(np.int32)
    offs = np.concatenate([[0], np.cumsum(np.bincount(ids.reshape(-1), minlength=E + 1)[:E])])
    assert np.array_equal(off.cpu().numpy(), offs) and np.array_equal(order.src_index.cpu().numpy(), src)
    want_h, pre = ox.product(q, s, w1, s1, offs, src, rows, k, False, True)
    n = offs[-1]
    check_product(h[:n], want_h[:n], pre[:n], "bf16", True)
    hq, hs = ox.quant(h.float().cpu().numpy()[:n])
    yy, pre = ox.product(np.concatenate([hq, np.zeros((rows - n, hq.shape[1]), np.int8)]), np.concatenate([hs, np.zeros(rows - n, np.float32)]),
                         w2, s2, offs, src, rows, 0, True)
    live = ids.reshape(-1) < E
    check_product(y[dev(live)], yy[live], pre[live], "bf16", False)
    assert bool(torch.isnan(y[dev(~live)]).all())
    want, size = ox.combine(np.where(live[:, None], y.float().cpu().numpy(), 0), wt.cpu().numpy(), shared)
    assert np.all(np.abs(out - want) <= (k + 2) * U * size + HALF["bf16"] * np.abs(want) * 1.01)


@pytest.mark.parametrize("T,E,k,d,hidden", [(2, 16, 4, 128, 192), (24, 16, 4, 128, 192), (500, 4, 2, 128, 192), (9000, 3, 2, 128, 4096)])
def test_captured_with_the_exchange_and_replayed(gpu, T, E, k, d, hidden):
    """The whole way in a graph, with the exchange's form that can be captured; and two objects in one graph."""
    rng = np.random.default_rng(9)
    rows = T * k
    w1, s1 = (dev(t) for t in weights(gpu, rng, E, hidden, d))
    w2, s2 = (dev(t) for t in weights(gpu, rng, E, d, hidden))
    router = gpu.Router(T, E, k, "sigmoid")
    ex = gpu.desc(gpu.PW_GRAPH_EXCHANGE, E + 1, rows, 1, num_src_shards=1)
    sorted_w = torch.empty(rows, 1, device="cuda")
    off = torch.empty(E + 2, dtype=torch.int64, device="cuda")
    src = torch.empty(rows, dtype=torch.int32, device="cuda")
    first = gpu.Int8Product(w1, s1, d, rows, gather=k, gelu=True)
    second = gpu.Int8Product(w2, s2, hidden, rows, scatter=True)
    join = gpu.TopkCombine(T, d, k)
    l, x = torch.zeros(T, E, device="cuda"), torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")

    def way():
        experts, wt = router.forward(l)
        gpu.exchange_scratch(ex, gpu.exchange_io(wt, experts, sorted_w, 1, E + 1, 1, src_index=src, offsets=off))
        h = first.forward(x, offsets=off[:E + 1], src_index=src)
        return join.forward(second.forward(h, offsets=off[:E + 1], src_index=src), wt)

    with pytest.raises(gpu.PwError):  # buffers are not made under capture
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            gpu.TopkCombine(T, d, k).forward(torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, k, device="cuda"))
    way()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = way()
    for seed in range(4):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        l.copy_(torch.randn(T, E, generator=gen, device="cuda"))
        x.copy_(torch.randn(T, d, generator=gen, device="cuda"))
        g.replay()
        got = out.clone()
        assert torch.equal(got, way())
        torch.cuda.synchronize()


# ---- rounding and range of the results ------------------------------------------

def dense(gpu, rows, d, n, dtype, act, x_scale, w_scale, seed=0):
    """A product of one matrix from given scales: (got, z in 64 bits, from the codes)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randint(-127, 128, (rows, ox.q8_row(d)), dtype=torch.int8, device="cuda", generator=gen)
    w = torch.randint(-127, 128, (1, n, ox.q8_row(d)), dtype=torch.int8, device="cuda", generator=gen)
    q[:, d:], w[:, :, d:] = 0, 0
    s = torch.full((rows,), x_scale, device="cuda") if np.isscalar(x_scale) else x_scale
    ws = torch.full((1, n), w_scale, device="cuda") if np.isscalar(w_scale) else w_scale
    got = gpu.Int8Product(w, ws, d, rows, gelu=act, dtype=pwt(gpu, dtype)).forward(q, x_scale=s)
    z = (q.double() @ w[0].double().t().contiguous()) * s.double().unsqueeze(1) * ws.double()
    return got, z


@pytest.mark.parametrize("rows,d,n", [(8, 700, 4000), (40, 2100, 1000), (300, 1000, 515), (2500, 512, 520), (20000, 640, 4096)])
def test_gelu_is_rounded_to_the_nearest_but_for_its_own_last_bits(gpu, rows, d, n):
    """bf16 results are those of a number that is at most e off z Phi(z): z is rounded three times and carries z^2 + 2
    times that, and GELU adds (2 z^2 + 26) u and 2.9e-7 of itself (below 5 u)."""
    got, z = dense(gpu, rows, d, n, "bf16", True, 1.8 / 73.3, 1 / (73.3 * d ** 0.5))
    for g, y in zip(got.split(2048), z.split(2048)):
        e = (3 * (y * y + 2) + 2 * y * y + 31) * U * 1.01
        want = y * 0.5 * torch.special.erfc(-y * 0.5 ** 0.5)
        ends = torch.stack([want * (1 - e), want * (1 + e)]).float().bfloat16()
        ok = (g >= ends.min(0).values) & (g <= ends.max(0).values) | (y.abs() > 12)
        assert bool(ok.all()), (int((~ok).sum()), ok.numel())


VARIANTS = [(7, 700, 400), (40, 2100, 1000), (300, 1000, 515), (2500, 512, 520), (20000, 640, 1024)]  # every kernel


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d,n", VARIANTS)
def test_infinite_and_huge_results(gpu, rows, d, n, dtype):
    """z Phi(z) of +infinity is +infinity, of -infinity 0; 0 x infinity and NaN are NaN; the same without GELU but for -infinity."""
    s = torch.full((rows,), 1e-3, device="cuda")
    ws = torch.full((1, n), 1e-3, device="cuda")
    s[1], s[2], s[rows - 1] = float("inf"), float("nan"), 1e30
    ws[0, 3], ws[0, 5], ws[0, 7], ws[0, n - 1] = float("inf"), float("nan"), 1e34, -float("inf")
    for act in (False, True):
        got, z = dense(gpu, rows, d, n, dtype, act, s, ws)
        z = torch.where(z.abs() > torch.finfo(torch.float32).max, torch.sign(z) * float("inf"), z)
        want = torch.where(z < -40, torch.zeros_like(z), z * 0.5 * torch.special.erfc(-z * 0.5 ** 0.5)) if act else z
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.isinf(got), torch.isinf(want)) and bool((got[torch.isinf(got)].sign() == z[torch.isinf(got)].sign()).all())
        ok = torch.isfinite(want)
        err = (5 * torch.where(ok & (z.abs() < 13), z, torch.zeros_like(z)) ** 2 + 32) * U + HALF[dtype] * 1.01
        assert bool(((got.double() - want).abs() <= want.abs() * err + 1e-30)[ok].all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,d,n", VARIANTS)
def test_rows_of_the_largest_numbers(gpu, rows, d, n, dtype):
    """Sums that pass fp32 before the column's scale brings them back, and scales below the normal numbers: a result
    is off by three roundings and its own (z^2 + 2 times them with GELU, and (2 z^2 + 31) u), whatever the scales."""
    top = torch.finfo(torch.float32).max / 127
    s = torch.full((rows,), 1.0, device="cuda")
    s[::5], s[1::5], s[2::5], s[3::5] = top, 2.0 ** 97, 1.5 * 2.0 ** 96, 2.0 ** -149
    for scale in (1.0, 1e-3, 1e-36, 1e-38, 1e30):
        for act in (False, True):
            got, z = dense(gpu, rows, d, n, dtype, act, s, scale, seed=rows)
            want = z * 0.5 * torch.special.erfc(-z * 0.5 ** 0.5) if act else z
            # (where the result passes the type it is infinite; next to its end either will do)
            most = float(torch.finfo(DT[dtype]).max)
            fits = want.abs() < most * (1 - 2.0 ** -7)
            assert bool(torch.isinf(got[want.abs() > most * (1 + 2.0 ** -7)]).all())
            a = z.abs().clamp(max=13.0)
            err = (3 * (a * a + 2) + 2 * a * a + 31 if act else torch.full_like(z, 3)) * U * 1.01 + HALF[dtype] * 1.01
            if act:
                fits &= z > -13
            assert bool(((got.double() - want).abs() <= want.abs() * err + 2.0 ** -126)[fits].all())


@pytest.mark.parametrize("rows,d,n", [(8, 512, 64), (3000, 4096, 64)])
def test_codes_need_no_workspace(gpu, rows, d, n):
    """A call that is given codes makes no room for any: nothing is allocated, also under capture, where nothing may be."""
    w, ws = torch.ones(1, n, d, dtype=torch.int8, device="cuda"), torch.ones(1, n, device="cuda")
    q, s = torch.ones(rows, d, dtype=torch.int8, device="cuda"), torch.ones(rows, device="cuda")
    x, out = torch.ones(rows, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    f = gpu.Int8Product(w, ws, d, rows)
    before = torch.cuda.memory_allocated()
    f.forward(q, x_scale=s, out=out)
    assert torch.cuda.memory_allocated() == before and bool((out == d).all())
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpu.Int8Product(w, ws, d, rows).forward(q, x_scale=s, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        assert bool((out == d).all())
    with pytest.raises(gpu.PwError):          # this one needs it
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            f.forward(x, out=out)
    f.forward(x, out=out)
    assert torch.cuda.memory_allocated() > before and bool((out == d).all())


@pytest.mark.parametrize("d", [64, 960, 1024, 1025, 1088, 2048, 2049, 2112, 3000, 4032, 4096])
@pytest.mark.parametrize("rows", [1, 5, 8])
def test_few_rows_at_the_ends_of_what_a_wave_holds(gpu, rows, d):
    rng = np.random.default_rng([rows, d])
    n, E = 70, 3
    w, ws = weights(gpu, rng, E, n, d)
    x = rows_of(rng, rows, d, "bf16")
    q, s = ox.quant(x)
    off = np.array([0, rows // 2, rows // 2, rows])
    out = gpu.Int8Product(dev(w), dev(ws), d, rows).forward(dev(x, torch.bfloat16), offsets=dev(off))
    want, pre = ox.product(q, s, w, ws, off, None, rows)
    check_product(out, want, pre, "bf16", False)


# ---- calls that the documentation allows ------------------------------------------

@pytest.mark.parametrize("E,each,d,n,kind", [(256, 600, 64, 520, "even"), (200, 640, 192, 512, "holes"), (64, 2100, 320, 300, "holes")])
def test_many_experts_where_workgroups_walk(gpu, E, each, d, n, kind):
    """Up to 256 experts, many of them without a row, in the kernel whose workgroups walk over tiles; misaligned outputs too."""
    rng = np.random.default_rng([E, n])
    rows = E * each
    p = np.ones(E) if kind == "even" else (rng.random(E) < 0.4) + 1e-9
    dest = rng.choice(E, rows, p=p / p.sum())
    off = np.concatenate([[0], np.cumsum(np.bincount(dest, minlength=E))])
    src = np.argsort(dest, kind="stable").astype(np.int32)
    w, ws = weights(gpu, rng, E, n, d)
    q = rng.integers(-127, 128, (rows, ox.q8_row(d))).astype(np.int8)
    q[:, d:] = 0
    s = (rng.random(rows) * 0.02).astype(np.float32)
    f = gpu.Int8Product(dev(w), dev(ws), d, rows, scatter=True)
    flat = torch.full((rows * n + 1,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = flat[1:].view(rows, n)
    f.forward(dev(q), x_scale=dev(s), offsets=dev(off), src_index=dev(src), out=out)
    pick = np.sort(rng.choice(rows, 3000, replace=False))           # dispatched rows that are looked at
    e = np.searchsorted(off, pick, side="right") - 1
    W, P, X = dev(w), torch.from_numpy(pick), dev(q)
    for i in range(0, len(pick), 500):
        rr, ee = P[i:i + 500].cuda(), torch.from_numpy(e[i:i + 500]).cuda()
        z = (X[rr].double().unsqueeze(1) * W[ee].double()).sum(2) if n * d < 40000 else torch.stack(
            [W[int(b)].double() @ X[int(a)].double() for a, b in zip(rr, ee)])
        want = z * dev(s)[rr].double().unsqueeze(1) * dev(ws)[ee].double()
        got = out[dev(src)[rr].long()].double()
        assert bool(((got - want).abs() <= want.abs() * (HALF["bf16"] + 3.03 * U) + 1e-37).all())
    assert float(flat[0]) == 7.0


@pytest.mark.parametrize("rows,d,n,E", [(8, 700, 64, 5), (40, 2100, 1000, 5), (300, 1000, 515, 5), (6000, 512, 520, 5), (20000, 640, 1024, 5), (20000, 640, 1024, 1)])
def test_no_row_at_all(gpu, rows, d, n, E):
    """Segments that are all empty: nothing is read, nothing written."""
    rng = np.random.default_rng(rows)
    w, ws = weights(gpu, rng, E, n, d)
    x = torch.full((rows, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    for at in (0, -3, 1 << 40):
        off = torch.full((E + 1,), at, dtype=torch.int64, device="cuda")
        out = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
        gpu.Int8Product(dev(w), dev(ws), d, rows).forward(x, offsets=off, out=out)
        assert bool((out == 7.0).all())


def test_two_streams_at_once(gpu):
    """Objects of their own on two streams, products of every kernel among them, give what they give one after the other."""
    rng = np.random.default_rng(11)
    calls = []
    for i, (rows, d, n) in enumerate(VARIANTS * 2):
        w, ws = weights(gpu, rng, 1, n, d)
        x = dev(rows_of(rng, rows, d, "bf16"), torch.bfloat16)
        f = gpu.Int8Product(dev(w), dev(ws), d, rows, gelu=bool(i % 2))
        calls.append((f, x, f.forward(x).clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(3):
        for i, (f, x, want) in enumerate(calls):
            outs.append((f.forward(x, stream=streams[i % 2]), want))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)


@pytest.mark.parametrize("rows,d,n", [(7, 701, 65), (40, 2101, 130), (300, 999, 131)])
def test_rows_that_begin_anywhere(gpu, rows, d, n):
    """x, out and the scales aligned to their elements alone."""
    rng = np.random.default_rng(rows)
    w, ws = weights(gpu, rng, 1, n, d)
    for dtype in ("bf16", "f32"):
        x = rows_of(rng, rows, d, dtype)
        q, s = ox.quant(x)

        def off(a, t):
            flat = torch.zeros(a.size + 1, dtype=t, device="cuda")
            v = flat[1:].view(a.shape)
            v.copy_(dev(a))
            return v

        for act in (False, True):
            f = gpu.Int8Product(dev(w), off(ws, torch.float32), d, rows, gelu=act, dtype=pwt(gpu, dtype))
            out = off(np.zeros((rows, n), np.float32), DT[dtype])
            f.forward(off(x, DT[dtype]), out=out)
            want, pre = ox.product(q, s, w, ws, None, None, rows, act=act)
            check_product(out, want, pre, dtype, act)


def test_codes_captured_with_a_limit_that_changes(gpu):
    rng = np.random.default_rng(13)
    x = rows_of(rng, 900, 300, "bf16")
    wq, ws = ox.quant(x)
    X, limit = dev(x, torch.bfloat16), torch.zeros(1, dtype=torch.int64, device="cuda")
    f = gpu.RowQuant(900, 300)
    q, s = f.forward(X, limit=limit)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f.forward(X, limit=limit)
    for n in (5, 900, 0, 77, 1 << 35):
        q.fill_(99)
        s.fill_(-1.0)
        limit.fill_(n)
        g.replay()
        n = min(n, 900)
        assert np.array_equal(q.cpu().numpy()[:n], wq[:n]) and np.array_equal(s.cpu().numpy()[:n], ws[:n])
        assert bool((q[n:] == 99).all()) and bool((s[n:] == -1).all())
