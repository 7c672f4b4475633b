"""GPU parity of the router balance (loss, counts, gradient of the logits)
against the oracle in 64 bits.

Bars, with u = 2^-24 (an fp32 rounding) and D the widest row of logits (its
maximum minus a logit): exp of a rounded difference is off by (D + 4) u, a
row's sum of E terms in lanes of 4 and a tree by 12 more, so p by
(2 D + 32) u of itself; a lane adds at most 512 rows before the partial sums
are joined in double; lse is off by u (|lse| + 2 D + 32).
"""
import numpy as np
import pytest
import torch

from oracle import block as ob

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BAL, Z = 0.7, 0.05

CASES = [(1, 2, 1, None), (1, 64, 2, None), (7, 3, 2, None), (48, 8, 2, "some"), (999, 5, 2, "some"), (2048, 64, 2, None),
         (2049, 64, 2, "some"), (5000, 16, 4, None), (3001, 65, 8, "some"), (513, 256, 8, "some"), (2500, 256, 2, None),
         (257, 130, 3, None), (300, 17, 1, "none valid"), (40000, 64, 2, "some"), (70001, 7, 3, "some")]


def make(T, E, k, masked, seed=0):
    rng = np.random.default_rng([T, E, k, seed])
    l = (rng.standard_normal((T, E)) * 2 + np.linspace(1, -1, E)).astype(np.float32)
    ex = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    kept = np.exp(np.take_along_axis(l, ex, 1).astype(np.float64))
    g = (kept / kept.sum(1, keepdims=True)).astype(np.float32)
    dg = rng.standard_normal((T, k)).astype(np.float32)
    valid = None if masked is None else (rng.random(T) < 0.8) if masked == "some" else np.zeros(T, bool)
    return l, ex, g, dg, valid, (rng.random(2) + 0.5).astype(np.float32)


def dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


def width(l):
    return float((l.max(axis=1) - l.min(axis=1)).max())


def check_loss(got, l, ex, valid):
    counts, mean, loss = (t.cpu().numpy() for t in got)
    c, m, want, p, lse = ob.balance(l, ex, valid, BAL, Z)
    assert np.array_equal(counts, c)
    D = width(l)
    rel = (2 * D + 32 + 512 + 16) * U
    assert np.all(np.abs(mean - m) <= rel * m + 1e-38)
    assert abs(loss[0] - want[0]) <= (rel + 8 * U) * want[0]
    e = U * (np.abs(lse) + 2 * D + 32)
    bound = Z * ((2 * np.abs(lse) * e + e * e).mean() + 600 * U * (lse ** 2).mean()) if lse.size else 0
    assert abs(loss[1] - want[1]) <= bound


def check_grad(d, l, ex, counts, g, dg, valid, u):
    want, size = ob.router_grad(l, ex, counts, g, dg, valid, u, BAL, Z)
    safe = l if valid is None else np.where(valid[:, None], l, 0)
    assert np.all(np.abs(d - want) <= (4 * width(safe) + 64) * U * size + 1e-38)


@pytest.mark.parametrize("T,E,k,masked", CASES)
def test_loss_counts_and_gradient(gpu, T, E, k, masked):
    print(f"balance T={T} E={E} k={k} {masked}", flush=True)
    l, ex, g, dg, valid, u = make(T, E, k, masked)
    f = gpu.RouterBalance(T, E, k, BAL, Z)
    L, X, V = dev(l), dev(ex), dev(valid)
    got = f.loss(L, X, valid=V)
    check_loss(got, l, ex, valid)
    counts = got[0].cpu().numpy()
    d = f.grad(L, X, gates=dev(g), dgates=dev(dg), valid=V, grad_loss=dev(u)).cpu().numpy()
    check_grad(d, l, ex, counts, g, dg, valid, u)
    # the losses alone, upstream gradients of one
    check_grad(f.grad(L, valid=V).cpu().numpy(), l, ex, counts, None, None, valid, None)
    # equal inputs, equal bits
    again = [t.clone() for t in f.loss(L, X, valid=V)]
    assert all(torch.equal(a, b) for a, b in zip(again, f.loss(L, X, valid=V)))


def test_logits_that_are_not_16_byte_aligned(gpu):
    T, E, k = 300, 64, 2
    l, ex, g, dg, _, u = make(T, E, k, None)
    flat = torch.zeros(T * E + 1, device="cuda")
    L = flat[1:].view(T, E)
    L.copy_(dev(l))
    f = gpu.RouterBalance(T, E, k, BAL, Z)
    check_loss(f.loss(L, dev(ex)), l, ex, None)
    d = f.grad(L, dev(ex), gates=dev(g), dgates=dev(dg), grad_loss=dev(u)).cpu().numpy()
    check_grad(d, l, ex, f.loss(L, dev(ex))[0].cpu().numpy(), g, dg, None, u)


def test_masked_rows_hold_anything(gpu):
    """NaN, infinities and foreign expert ids in padding; all -inf and lowest-value rows, unrouted tuples in valid rows."""
    T, E, k = 64, 8, 2
    l, ex, g, dg, _, u = make(T, E, k, None)
    valid = np.ones(T, bool)
    valid[[3, 9, 63]] = False
    l[3], l[9], l[63] = np.nan, np.inf, -np.inf
    g[3], dg[9] = np.nan, np.inf
    ex[3] = 1 << 30
    l[5] = -np.inf                                # nothing to choose from
    l[6] = np.finfo(np.float32).min               # a mask of the lowest value: an even row
    l[7, :4] = -np.inf
    ex[20] = -1, 8                                # no tuples
    ex[21] = 4, 4                                 # one expert twice
    f = gpu.RouterBalance(T, E, k, BAL, 0.0)      # the lowest value squared is no fp32 number
    counts, mean, loss = (t.cpu().numpy() for t in f.loss(dev(l), dev(ex), valid=dev(valid)))
    c, m, want, _, _ = ob.balance(l, ex, valid, BAL, 0.0)
    assert np.array_equal(counts, c) and counts[:E].sum() == 2 * (T - 3) - 2
    assert np.all(np.abs(mean - m) <= 700 * U * m) and abs(loss[0] - want[0]) <= 800 * U * want[0] and loss[1] == 0
    d = f.grad(dev(l), dev(ex), gates=dev(g), dgates=dev(dg), valid=dev(valid)).cpu().numpy()
    want, size = ob.router_grad(np.where(np.isnan(l), 0, l), ex, counts, g, dg, valid, None, BAL, 0.0)
    assert np.all(d[[3, 9, 63]] == 0)
    assert np.all(np.abs(d - want) <= 200 * U * size)


def test_offsets_past_32_bits(gpu):
    """More than 2^32 logits: the last tokens alone are valid."""
    T, E, k, n = 17000000, 256, 2, 300
    assert T * E > 1 << 32
    l, ex, g, dg, _, u = make(n, E, k, None)

    def long(a, dtype):
        t = torch.zeros(T, a.shape[1], dtype=dtype, device="cuda")
        t[-n:] = dev(a)
        return t

    f = gpu.RouterBalance(T, E, k, BAL, Z)
    L, X = long(l, torch.float32), long(ex, torch.int32)
    valid = torch.zeros(T, dtype=torch.bool, device="cuda")
    valid[-n:] = True
    got = f.loss(L, X, valid=valid)
    check_loss(got, l, ex, None)
    d = f.grad(L, X, gates=long(g, torch.float32), dgates=long(dg, torch.float32), valid=valid, grad_loss=dev(u))
    check_grad(d[-n:].cpu().numpy(), l, ex, got[0].cpu().numpy(), g, dg, None, u)
    assert not d[:T - n].any()


def test_no_tokens(gpu):
    f = gpu.RouterBalance(0, 4, 2)
    e = torch.empty((0, 4), device="cuda")
    i = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    for t in f.loss(e, i):
        assert not t.any()
    assert f.grad(e, i).shape == (0, 4)


def test_another_stream_and_a_replayed_graph(gpu):
    T, E, k = 9000, 64, 2
    f = gpu.RouterBalance(T, E, k, BAL, Z)
    data = [make(T, E, k, "some", seed) for seed in range(4)]
    L, X, G, DG, V, UP = (dev(a).clone() for a in data[0])
    f.grad(L, X, counts=f.loss(L, X, valid=V)[0], gates=G, dgates=DG, valid=V, grad_loss=UP)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = f.loss(L, X, valid=V)
        d = f.grad(L, X, gates=G, dgates=DG, valid=V, grad_loss=UP)
    for l, ex, g, dg, valid, u in data[1:] + data[:1]:
        for t, a in zip((L, X, G, DG, V, UP), (l, ex, g, dg, valid, u)):
            t.copy_(dev(a))
        graph.replay()
        torch.cuda.synchronize()
        check_loss(got, l, ex, valid)
        check_grad(d.cpu().numpy(), l, ex, got[0].cpu().numpy(), g, dg, valid, u)
    other = gpu.RouterBalance(T, E, k, BAL, Z)
    side.wait_stream(torch.cuda.current_stream())
    out = other.loss(L, X, valid=V, stream=side)
    side.synchronize()
    check_loss(out, l, ex, valid)


def test_two_objects_on_two_streams_at_once(gpu):
    """Nothing is shared between objects."""
    sets = [make(60000, 64, 2, "some", seed) for seed in (11, 12)]
    streams = [torch.cuda.Stream() for _ in sets]
    objs = [gpu.RouterBalance(60000, 64, 2, BAL, Z) for _ in sets]
    data = [[dev(a) for a in s] for s in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for f, (L, X, G, DG, V, UP), st in zip(objs, data, streams):
            f.loss(L, X, valid=V, stream=st)
            f.grad(L, X, gates=G, dgates=DG, valid=V, grad_loss=UP, stream=st)
    torch.cuda.synchronize()
    for f, (l, ex, g, dg, valid, u) in zip(objs, sets):
        check_loss((f._counts, f._buffers["prob_mean"], f._buffers["loss"]), l, ex, valid)
        check_grad(f._buffers["dlogits"].cpu().numpy(), l, ex, f._counts.cpu().numpy(), g, dg, valid, u)


def test_a_first_call_under_capture_is_refused(gpu):
    f = gpu.RouterBalance(16, 8, 2)
    l, x = torch.zeros(16, 8, device="cuda"), torch.zeros(16, 2, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = l + 1
        with pytest.raises(gpu.PwError) as e:
            f.loss(l, x)
    assert e.value.code == gpu.PW_ERR_STATE
    graph.replay()
    torch.cuda.synchronize()
    assert bool((y == 1).all())


def test_buffers_belong_to_the_stream_of_the_first_call(gpu):
    """Memory that was just freed on the current stream may still be in use
    there: a call on another stream gets none of it."""
    T, E = 50000, 64
    f = gpu.RouterBalance(T, E, 2)
    l, x = torch.zeros(T, E, device="cuda"), torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (4 * T * E, 256 * (E + 1) * 8, 4 * E, 8, 4 * (E + 1))]
    spans = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in freed]
    torch.cuda.synchronize()
    del freed
    side = torch.cuda.Stream()
    f.loss(l, x, stream=side)
    f.grad(l, x, stream=side)
    side.synchronize()
    assert set(f._buffers) == {"counts", "prob_mean", "loss", "dlogits", "workspace"}
    for name, b in f._buffers.items():
        lo, hi = b.data_ptr(), b.data_ptr() + b.numel() * b.element_size()
        assert all(hi <= s or e <= lo for s, e in spans), name


def test_refusals(gpu):
    f = gpu.RouterBalance(16, 8, 2)
    l, x = torch.zeros(16, 8, device="cuda"), torch.zeros(16, 2, dtype=torch.int32, device="cuda")
    for bad in ((l.half(), x), (l[:15], x), (l.cpu(), x), (l.t().contiguous().t(), x), (l, x.long()), (l, x[:, :1])):
        with pytest.raises(gpu.PwError):
            f.loss(*bad)
    with pytest.raises(gpu.PwError):
        f.loss(None, x)
    with pytest.raises(gpu.PwError):
        f.grad(l, x)                      # no counts yet
    with pytest.raises(gpu.PwError):
        gpu.RouterBalance(16, 1)


@pytest.mark.parametrize("T,E", [(1 << 25, 65), (1 << 28, 2)])
def test_long_batches_of_equal_tokens(gpu, T, E):
    """Thousands of equal rows a lane, where fp32 additions err to the same side:
    a lane adds them in runs of 256, and then the runs, here at most 32. Bar: p by
    (2 D + 32) u, these additions, 40 more across lanes, waves and partial sums; lse
    as above."""
    row = np.linspace(0.5, -0.5, E).astype(np.float32)[None]
    l = dev(row).expand(T, E).contiguous()
    ex = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    counts, mean, loss = (t.cpu().numpy() for t in gpu.RouterBalance(T, E, 1, BAL, Z).loss(l, ex))
    assert counts[0] == counts[E] == T and not counts[1:E].any()
    p, lse = (a[0] for a in ob.softmax_lse(row))
    rel = (2 * width(row) + 32 + 256 + 32 + 40) * U
    assert np.all(np.abs(mean - p) <= rel * p)
    assert abs(loss[0] - BAL * E * p[0]) <= (rel + 8 * U) * BAL * E * p[0]
    e = U * (abs(lse) + 2 * width(row) + 32)
    assert abs(loss[1] - Z * lse ** 2) <= Z * (2 * abs(lse) * e + e * e + 330 * U * lse ** 2)


@pytest.mark.parametrize("T,E,k,masked", [(300, 61, 2, None), (20000, 61, 2, "some"), (40000, 18, 3, "some"), (70001, 35, 8, None),
                                          (3000, 3, 2, "some"), (70001, 2, 1, None), (140000, 3, 3, "some"), (9, 2, 2, None)])
def test_expert_counts_that_fill_no_lane(gpu, T, E, k, masked):
    """17 to 64 experts that are no multiple of 4 (a lane moved back to the row's
    last four) and fewer than 4, in one launch and in two, and with one and with four
    rows of the logit gradient in flight."""
    test_loss_counts_and_gradient(gpu, T, E, k, masked)
