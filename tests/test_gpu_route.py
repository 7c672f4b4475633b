"""GPU parity of the routing to experts and its gradient against the oracle in
64 bits. The chosen experts are equal.

Bars, with u = 2^-24 (an fp32 rounding) and D the widest difference of two
logits, or the largest one for a sigmoid: the exponential of a rounded
difference is off by (D + 4) u, a sum of E terms in lanes of 4 and a tree by 12 u
more, and a weight is the quotient of two such, times the scale: (2 D + 40) u.
A gradient's terms are products of three of these: (4 D + 96) u of their
absolute values.
"""
import numpy as np
import pytest
import torch

from oracle import experts as ox

pytestmark = pytest.mark.gpu
U = ox.U
SCALE = 2.5

# tokens, experts, k, sigmoid, bias, groups, top_groups, group_best, renorm, masked
CASES = [(1, 2, 1, False, False, 1, 1, 2, True, False), (1, 256, 8, True, True, 8, 4, 2, True, False),
         (3, 8, 8, False, False, 2, 1, 2, True, False), (5, 5, 2, False, True, 5, 3, 2, False, True),
         (33, 64, 6, True, True, 1, 1, 2, True, True), (48, 8, 2, False, False, 1, 1, 2, True, False),
         (64, 60, 8, False, False, 4, 2, 1, False, True), (100, 17, 3, True, False, 1, 1, 2, False, True),
         (129, 65, 8, True, True, 13, 2, 2, True, False), (250, 256, 8, False, True, 16, 3, 1, True, True),
         (255, 130, 1, True, True, 2, 1, 2, False, False), (300, 16, 4, False, False, 16, 5, 2, True, True),
         (999, 5, 2, False, False, 1, 1, 2, False, True), (1000, 128, 6, True, True, 4, 2, 2, True, True),
         (1500, 33, 7, True, False, 3, 2, 2, True, False), (2000, 64, 2, False, False, 1, 1, 2, True, True),
         (4099, 12, 5, True, True, 6, 4, 1, True, False), (5000, 3, 3, True, True, 1, 1, 2, True, True),
         (70, 2, 1, True, True, 2, 1, 2, False, False), (90, 3, 2, False, False, 3, 2, 1, True, True),
         (16384, 64, 6, True, True, 1, 1, 2, True, True), (34000, 64, 4, False, False, 1, 1, 2, False, True),
         (40000, 60, 1, True, True, 4, 2, 2, True, False), (33000, 64, 8, False, True, 8, 2, 2, False, False), (17001, 30, 3, False, False, 5, 2, 2, False, False),
         (16500, 9, 1, True, True, 1, 1, 2, True, False), (3000, 7, 7, True, False, 1, 1, 2, True, True), (777, 16, 8, False, True, 1, 1, 2, False, True), (20001, 200, 8, True, True, 8, 3, 2, True, True),
         (16999, 256, 4, False, True, 1, 1, 2, True, False), (16400, 13, 7, True, False, 1, 1, 2, False, True)]


def make(T, E, k, bias, masked, seed=0):
    rng = np.random.default_rng([T, E, k, seed])
    l = (rng.standard_normal((T, E)) * 1.5 + np.linspace(0.7, -0.7, E)).astype(np.float32)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32) if bias else None
    valid = rng.random(T) < 0.8 if masked else None
    return l, b, valid, rng.standard_normal((T, k)).astype(np.float32), rng.standard_normal((T, E)).astype(np.float32)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def width(l, sigmoid):
    l = l[np.isfinite(l)] if l.ndim == 1 else l
    f = np.where(np.isfinite(l), l, 0)
    return float(np.abs(f).max()) if sigmoid else float((f.max(axis=-1) - f.min(axis=-1)).max())


def router(gpu, T, E, k, sigmoid, groups=1, top_groups=1, group_best=2, renorm=True, scale=SCALE):
    return gpu.Router(T, E, k, "sigmoid" if sigmoid else "softmax", groups, top_groups, group_best, renorm, scale)


def check_route(got, l, b, valid, k, sigmoid, groups=1, top_groups=1, group_best=2, renorm=True, scale=SCALE, D=None):
    ids, w = ox.route(l, b, valid, k, sigmoid, groups, top_groups, group_best, renorm, scale)
    D = width(l, sigmoid) if D is None else D
    experts, weights = got[0].cpu().numpy(), got[1].cpu().numpy().astype(np.float64)
    assert np.array_equal(experts, ids), np.flatnonzero((experts != ids).any(1))[:10]
    assert np.all(np.abs(weights - w) <= (2 * D + 40) * U * np.abs(w) + 1e-37)
    return ids


def check_grad(got, l, ids, dw, valid, add, sigmoid, renorm, scale=SCALE, D=None):
    want, size = ox.route_grad(l, ids, dw, valid, add, sigmoid, renorm, scale)
    D = width(l, sigmoid) if D is None else D
    d = got.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(d - want) <= (4 * D + 96) * U * size + 1e-37)


@pytest.mark.parametrize("T,E,k,sigmoid,bias,groups,top_groups,group_best,renorm,masked", CASES)
def test_choice_weights_and_gradient(gpu, T, E, k, sigmoid, bias, groups, top_groups, group_best, renorm, masked):
    print(f"route T={T} E={E} k={k} sigmoid={sigmoid} bias={bias} groups={groups}/{top_groups}", flush=True)
    l, b, valid, dw, add = make(T, E, k, bias, masked)
    f = router(gpu, T, E, k, sigmoid, groups, top_groups, group_best, renorm)
    L, V = dev(l), dev(valid)
    got = f.forward(L, bias=dev(b), valid=V)
    ids = check_route(got, l, b, valid, k, sigmoid, groups, top_groups, group_best, renorm)
    check_grad(f.grad(L, got[0], dev(dw), valid=V), l, ids, dw, valid, None, sigmoid, renorm)
    check_grad(f.grad(L, got[0], dev(dw), valid=V, add=dev(add)), l, ids, dw, valid, add, sigmoid, renorm)
    # equal inputs, equal bits
    again = [t.clone() for t in got]
    assert all(torch.equal(x, y) for x, y in zip(again, f.forward(L, bias=dev(b), valid=V)))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E,groups,top_groups", [(8, 1, 1), (64, 8, 3), (256, 16, 5), (100, 4, 2)])
@pytest.mark.parametrize("T", [40, 3000, 34000])
def test_equal_scores_take_the_lowest_index(gpu, sigmoid, E, groups, top_groups, T):
    rng = np.random.default_rng(E)
    k = min(8, E // groups * top_groups)
    l = rng.integers(-1, 2, (T, E)).astype(np.float32)
    b = (rng.integers(0, 2, E) * 0.25).astype(np.float32)
    for bias in (None, b, np.zeros(E, np.float32)):
        f = router(gpu, T, E, k, sigmoid, groups, top_groups)
        check_route(f.forward(dev(l), bias=dev(bias)), l, bias, None, k, sigmoid, groups, top_groups)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("E", [6, 64, 200])
@pytest.mark.parametrize("T", [50, 2500, 33000])
def test_scores_that_differ_in_their_last_bits(gpu, sigmoid, E, T):
    """Neighbouring fp32 logits and biases: sums that fp32 cannot tell apart."""
    rng = np.random.default_rng([E, sigmoid])
    l = np.nextafter(np.float32(0.5), np.float32(1)) + np.zeros((T, E), np.float32)
    l += rng.integers(-3, 4, (T, E)).astype(np.float32) * np.float32(2.0 ** -24)
    b = (0.1 + rng.integers(-3, 4, E) * 2.0 ** -27).astype(np.float32)
    k = min(8, E)
    for bias in (None, b):
        for groups, top in ((1, 1), (2, 1)):
            if k > E // groups * top:
                continue
            f = router(gpu, T, E, k, sigmoid, groups, top)
            got = f.forward(dev(l), bias=dev(bias))
            rows = np.ones(T, bool)
            if groups == 2:
                rows = ~other_group(got[0].cpu().numpy(), l, bias, k, sigmoid)
            check_route([t[dev(rows)] for t in got], l[rows], bias, None, k, sigmoid, groups, top)


def other_group(experts, l, b, k, sigmoid):
    """Rows that take the other one of two groups, right if their marks are equal in 64 bits.

    Of logits x + i h on a grid of h = 2^-24, the pairs (i, j) and (i + 1, j - 1) have sums of scores that differ by
    s'' h^2 (1 + |i - j|) at most, with |s''| at most s and |i - j| at most 7: by 8 x 2^-48 = 2^-45 of a score as a bound, and
    by nothing in most pairs (softmax: s'' h^2 = s 2^-48). A sum of two scores and two biases is rounded four times, by up to
    2^-53 of itself each, and the exponentials behind it by as much again. Marks that are 2^-49 of themselves apart or less
    have no order that 64 bits could tell."""
    want, _ = ox.route(l, b, None, k, sigmoid, 2, 1)
    rows = np.flatnonzero((experts != want).any(1))
    c = ox.scores(l, sigmoid)[0] + (0 if b is None else b.astype(np.float64))
    half = l.shape[1] // 2
    marks = np.sort(c.reshape(len(l), 2, half), axis=2)[:, :, -2:].sum(2)
    for t in rows:
        assert abs(marks[t, 0] - marks[t, 1]) <= 2.0 ** -49 * marks[t].max()
        other = np.arange(2 * half) // half != want[t, 0] // half
        assert np.array_equal(experts[t], np.lexsort((np.arange(2 * half), -np.where(other, c[t], -np.inf)))[:k])
    out = np.zeros(len(l), bool)
    out[rows] = True
    return out


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,pad", [(8, 0), (8, 2500), (96, 0), (96, 2500), (8, 16384), (40, 60000), (96, 22000)])
def test_masked_and_infinite_logits(gpu, sigmoid, renorm, E, pad):
    """Rows whose mask leaves nothing, or fewer than k; the lowest value; NaN and infinities; padding that holds anything."""
    k, inf, low = 3, np.inf, np.finfo(np.float32).min
    rng = np.random.default_rng(E)
    l = rng.standard_normal((12 + pad, E)).astype(np.float32)
    l[0] = -inf
    l[1, 1:] = -inf
    l[2] = low
    l[3, 2:] = low
    l[4] = np.nan
    l[5, ::2] = np.nan
    l[6, :2] = inf
    l[7] = inf
    l[8] -= 150.0                                  # scores that fp32 cannot hold
    l[9], l[10] = np.nan, inf
    valid = np.ones(len(l), bool)
    valid[[9, 10]] = False
    b = np.zeros(E, np.float32)
    b[0], b[3], b[5] = -inf, np.nan, 0.5
    dw = rng.standard_normal((len(l), k)).astype(np.float32)
    f = router(gpu, len(l), E, k, sigmoid, renorm=renorm)
    for bias in (None, b):
        got = f.forward(dev(l), bias=dev(bias), valid=dev(valid))
        ids = check_route(got, l, bias, valid, k, sigmoid, renorm=renorm, D=160)
        assert np.all(ids[[0, 4, 9, 10]] == E) and np.all(got[1].cpu().numpy()[[0, 4, 9, 10]] == 0)
        d = f.grad(dev(l), got[0], dev(dw), valid=dev(valid))
        check_grad(d, l, ids, dw, valid, None, sigmoid, renorm, D=160)
        d = f.grad(dev(l), got[0], dev(dw), valid=dev(valid), add=dev(np.full_like(l, np.nan)))
        assert np.all(d.cpu().numpy()[[9, 10]] == 0)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_logits_of_few_bits(gpu, sigmoid):
    """bf16 logits: many equal ones among the best, none in doubt."""
    T, E, k = 40000, 64, 6
    l, b, _, _, _ = make(T, E, k, True, False)
    l = torch.from_numpy(l).bfloat16().float().numpy()
    f = router(gpu, T, E, k, sigmoid, renorm=False)
    for bias in (None, b):
        check_route(f.forward(dev(l), bias=dev(bias)), l, bias, None, k, sigmoid, renorm=False)


def test_a_group_without_experts_is_not_kept(gpu):
    l = np.tile(np.array([[0.0, 0.1, 3.0, -np.inf, -np.inf, -np.inf, -1.0, -2.0]], np.float32), (70, 1))
    for best in (1, 2):
        f = router(gpu, 70, 8, 4, True, 4, 2, best)
        check_route(f.forward(dev(l)), l, None, None, 4, True, 4, 2, best, D=4)
    f = router(gpu, 70, 8, 4, True, 4, 4)
    check_route(f.forward(dev(l)), l, None, None, 4, True, 4, 4, D=4)


def test_negative_scores_and_large_biases(gpu):
    T, E, k = 300, 24, 4
    l, _, _, _, _ = make(T, E, k, False, False)
    rng = np.random.default_rng(8)
    for s in (-1.0, 1e3, 1e-6, 3e38):
        b = (rng.standard_normal(E) * s).clip(-3e38, 3e38).astype(np.float32)
        for groups in (1, 4):
            f = router(gpu, T, E, k, True, groups, max(1, groups // 2))
            check_route(f.forward(dev(l), bias=dev(b)), l, b, None, k, True, groups, max(1, groups // 2))


def test_gradient_of_foreign_and_repeated_ids(gpu):
    T, E, k = 40, 20, 4
    l, _, _, dw, _ = make(T, E, k, False, False)
    ids = np.tile(np.array([3, 3, -1, 1 << 30], np.int32), (T, 1))
    ids[1] = 7
    ids[2] = E
    for sigmoid in (False, True):
        for renorm in (False, True):
            f = router(gpu, T, E, k, sigmoid, renorm=renorm)
            check_grad(f.grad(dev(l), dev(ids), dev(dw)), l, ids, dw, None, None, sigmoid, renorm)


@pytest.mark.parametrize("T,E,k", [(7, 64, 2), (3000, 64, 6), (300, 256, 8), (300, 10, 2), (40000, 63, 3)])
def test_buffers_that_are_not_16_byte_aligned(gpu, T, E, k):
    l, b, _, dw, add = make(T, E, k, True, False)

    def off(a):
        flat = torch.zeros(a.size + 1, device="cuda")
        t = flat[1:].view(a.shape)
        t.copy_(dev(a))
        return t

    f = router(gpu, T, E, k, True)
    got = f.forward(off(l), bias=off(b))
    ids = check_route(got, l, b, None, k, True)
    check_grad(f.grad(off(l), got[0], off(dw), add=off(add)), l, ids, dw, None, add, True, True)


def test_add_may_be_the_result(gpu):
    T, E, k = 200, 64, 2
    l, _, _, dw, add = make(T, E, k, False, False)
    f = router(gpu, T, E, k, False)
    ids, _ = f.forward(dev(l))
    out = f.grad(dev(l), ids, dev(dw))
    out.copy_(dev(add))
    check_grad(f.grad(dev(l), ids, dev(dw), add=out), l, ids.cpu().numpy(), dw, None, add, False, True)


def test_offsets_past_32_bits(gpu):
    """More than 2^32 logits: the last tokens alone are looked at."""
    T, E, k, n = 17000000, 256, 2, 300
    l, _, _, dw, _ = make(n, E, k, False, False)
    L = torch.zeros(T, E, device="cuda")
    L[-n:] = dev(l)
    valid = torch.zeros(T, dtype=torch.bool, device="cuda")
    valid[-n:] = True
    f = router(gpu, T, E, k, True)
    got = f.forward(L, valid=valid)
    ids = check_route([t[-n:] for t in got], l, None, None, k, True)
    assert int((got[0][:-n] != E).sum()) == 0
    DW = torch.zeros(T, k, device="cuda")
    DW[-n:] = dev(dw)
    d = f.grad(L, got[0], DW, valid=valid)
    check_grad(d[-n:], l, ids, dw, None, None, True, True)
    assert float(d[:-n].abs().max()) == 0


def test_no_tokens_and_refusals(gpu):
    f = router(gpu, 0, 8, 2, False)
    ids, w = f.forward(torch.empty(0, 8, device="cuda"))
    assert ids.shape == (0, 2) and w.shape == (0, 2)
    assert f.grad(torch.empty(0, 8, device="cuda"), ids, w).shape == (0, 8)
    f = router(gpu, 4, 8, 2, False)
    l = torch.zeros(4, 8, device="cuda")
    ids, w = f.forward(l)
    for bad in (l.double(), l.cpu(), l[:3], torch.zeros(8, 4, device="cuda").t()):
        with pytest.raises(gpu.PwError):
            f.forward(bad)
    with pytest.raises(gpu.PwError):
        f.forward(l, bias=torch.zeros(4, device="cuda"))
    with pytest.raises(gpu.PwError):
        f.grad(l, ids.long(), w)
    with pytest.raises(gpu.PwError):
        gpu.Router(4, 8, 2, score="relu")
    with pytest.raises(gpu.PwError):
        gpu.Router(4, 8, 9).forward(l)


@pytest.mark.parametrize("T,E,k", [(500, 64, 4), (36000, 64, 4), (9000, 256, 8)])
def test_on_another_stream_and_captured(gpu, T, E, k):
    l, b, _, dw, _ = make(T, E, k, True, False)
    L, B, DW = dev(l), dev(b), dev(dw)
    f = router(gpu, T, E, k, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ids, w = f.forward(L, bias=B)
        f.grad(L, ids, DW)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ids, w = f.forward(L, bias=B)
        d = f.grad(L, ids, DW)
    for seed in range(1, 4):
        l2, _, _, dw2, _ = make(T, E, k, True, False, seed)
        L.copy_(dev(l2))
        DW.copy_(dev(dw2))
        g.replay()
        torch.cuda.synchronize()
        i = check_route((ids, w), l2, b, None, k, True)
        check_grad(d, l2, i, dw2, None, None, True, True)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,E,groups", [(3000, 16, 8), (20000, 16, 8), (4000, 32, 16), (40000, 64, 16), (1000, 128, 16), (20000, 128, 16)])
def test_groups_whose_best_cancel(gpu, sigmoid, T, E, groups):
    """Marks of a large bias and its negative: what fp32 loses of the two is far more than what tells the marks apart."""
    rng = np.random.default_rng([T, E, sigmoid])
    l = (rng.standard_normal((T, E)) * 1e-2).astype(np.float32)
    for size in (100.0, 1000.0, 30000.0):
        b = np.full((groups, E // groups), -4 * size, np.float32)
        b[:, 0], b[:, 1] = size, -size
        for top in (1, 3):
            f = router(gpu, T, E, 2, sigmoid, groups, top)
            got = f.forward(dev(l), bias=dev(b.reshape(-1)))
            check_route(got, l, b.reshape(-1), None, 2, sigmoid, groups, top)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,E,groups", [(50, 16, 8), (20000, 16, 8), (40000, 64, 16), (300, 128, 16), (20000, 128, 16)])
def test_marks_below_the_least_number(gpu, sigmoid, T, E, groups):
    """Two biases near the type's lowest value, whose sum fp32 cannot hold: the groups' order is that of the sums."""
    rng = np.random.default_rng(E)
    l = rng.standard_normal((T, E)).astype(np.float32)
    b = np.full((groups, E // groups), -3.4e38, np.float32)
    b[:, 0] = b[:, 1] = -(3.3e38 - 1e37 * np.arange(groups))   # the last group is the best
    b = b.reshape(-1)
    for best in (1, 2):
        f = router(gpu, T, E, 4, sigmoid, groups, 3, best)
        check_route(f.forward(dev(l), bias=dev(b)), l, b, None, 4, sigmoid, groups, 3, best)
    b[2 * (E // groups)] = 0.0                                  # one group of an ordinary and a lowest value
    f = router(gpu, T, E, 4, sigmoid, groups, 2)
    check_route(f.forward(dev(l), bias=dev(b)), l, b, None, 4, sigmoid, groups, 2)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("T,E,k", [(200, 8, 4), (20000, 16, 8), (300, 64, 6), (40000, 64, 8), (500, 256, 8), (20000, 200, 7)])
def test_weights_of_far_logits(gpu, sigmoid, renorm, T, E, k):
    """Weights keep their bits far from zero. An exponential (of one ulp at most) is off by 2 u, and by D u for the
    rounding of a difference of logits that are D apart; 1 + e by 3 u at most and its quotient by u: a sigmoid's score by 6 u,
    and D u with renorm. A sum's terms e^-D carry D u of themselves, at most 0.37 u of the largest each, and as much besides as
    one score; adding k of them rounds 3 times, all E up to 21 times (16 in a lane, 6 levels), the quotient and the scale once each."""
    rng = np.random.default_rng([T, E, k])
    l = rng.uniform(-80, -10, (T, E)).astype(np.float32)
    f = router(gpu, T, E, k, sigmoid, renorm=renorm)
    ids, w = f.forward(dev(l))
    want_ids, want = ox.route(l, None, None, k, sigmoid, renorm=renorm, scale=SCALE)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    chosen = np.take_along_axis(l, want_ids, 1).astype(np.float64)
    apart = chosen.max(1, keepdims=True) - chosen  # (without a bias the best has the highest logit of all)
    if sigmoid:
        bar = apart + 6 + (0.37 * k + 6) + 3 + 2 if renorm else np.full(want.shape, 6.0 + 2)
    else:
        bar = apart + 2 + (0.37 * (k if renorm else E) + 2) + (3 if renorm else 21) + 2
    ok = np.abs(w.cpu().numpy().astype(np.float64) - want) <= bar * U * want + 1e-44 * SCALE
    assert ok.all(), (int((~ok).sum()), ok.size)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("T,E,groups", [(60, 8, 4), (20000, 8, 4), (60, 64, 8), (34000, 64, 8), (50, 200, 10), (12000, 200, 10)])
def test_infinite_biases(gpu, sigmoid, T, E, groups):
    """An infinite bias is above every score, of several the lowest index comes first; a group that holds one is kept."""
    rng = np.random.default_rng([T, E])
    l = rng.standard_normal((T, E)).astype(np.float32)
    b = (rng.standard_normal(E) * 0.1).astype(np.float32)
    b[[1, E // 2, E - 1]] = np.inf
    b[[0, E // 2 + 1]] = -np.inf
    for g, top in ((1, 1), (groups, 2), (groups, 3)):
        f = router(gpu, T, E, 4, sigmoid, g, top)
        check_route(f.forward(dev(l), bias=dev(b)), l, b, None, 4, sigmoid, g, top)
