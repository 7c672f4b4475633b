"""The oracle of the routing, its gradient, the 8-bit codes and products against
independent forms, and the refusals of the operators' entry points (host only)."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

import sparse_shard_exchange_amd as pw
from oracle import experts as ox


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_weights_and_gradient_against_autograd_and_differences(sigmoid, renorm):
    rng = np.random.default_rng(5)
    T, E, k, scale = 20, 12, 3, 1.7
    l = rng.standard_normal((T, E))
    bias = rng.standard_normal(E) * 0.1
    ids, w = ox.route(l, bias, None, k, sigmoid, 4, 2, 2, renorm, scale)
    t = torch.from_numpy(l).requires_grad_(True)
    s = torch.sigmoid(t) if sigmoid else torch.softmax(t, 1)
    c = (s.detach() + torch.from_numpy(bias)).view(T, 4, 3)
    keep = c.topk(2, dim=2).values.sum(2).topk(2, dim=1).indices
    mask = torch.zeros(T, 4, dtype=torch.bool).scatter_(1, keep, True)
    want = torch.where(mask.unsqueeze(2), c, torch.full_like(c, -9)).view(T, E).topk(k, dim=1).indices
    assert np.array_equal(ids, want.numpy())
    got = torch.gather(s, 1, want)
    got = scale * (got / got.sum(1, keepdim=True) if renorm else got)
    assert np.allclose(got.detach().numpy(), w, rtol=1e-13)
    dw = rng.standard_normal((T, k))
    (d,) = torch.autograd.grad(got, t, torch.from_numpy(dw))
    mine, size = ox.route_grad(l, ids, dw, None, None, sigmoid, renorm, scale)
    assert np.allclose(mine, d.numpy(), rtol=1e-11, atol=1e-13) and np.all(np.abs(mine) <= size + 1e-15)
    # differences, in random directions
    for _ in range(4):
        dl, h = rng.standard_normal(l.shape), 1e-5
        up, down = (ox._weights(l + f * h * dl, ids, sigmoid, renorm) * scale for f in (1, -1))
        assert abs(((up - down) * dw).sum() / (2 * h) - (mine * dl).sum()) < 1e-7


def test_route_places_without_an_expert():
    inf = np.inf
    l = np.array([[0.0, -inf, -inf, 1.0], [np.nan, -inf, -inf, -inf], [2.0, 2.0, 2.0, 2.0], [inf, 0.0, inf, 0.0]])
    ids, w = ox.route(l, None, None, 3, False)
    assert ids.tolist() == [[3, 0, 4], [4, 4, 4], [0, 1, 2], [0, 2, 1]]
    assert np.all(w[1] == 0) and w[0, 2] == 0 and np.allclose(w[3], [0.5, 0.5, 0])
    ids, _ = ox.route(l, np.array([0, 0, -inf, np.nan]), np.array([1, 1, 1, 0]), 2, True)
    assert ids.tolist() == [[0, 4], [4, 4], [0, 1], [4, 4]]
    # one member left in a group: its own value is the mark; a group of none is never kept
    ids, _ = ox.route(np.array([[0.0, 0.1, 3.0, -inf, -inf, -inf]]), None, None, 3, True, 3, 2)
    assert ids.tolist() == [[2, 1, 0]]
    # scores that underflow keep their ratio
    _, w = ox.route(np.array([[-2000.0, -2001.0]]), None, None, 2, True)
    assert np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.e)]])


def test_codes():
    x = np.array([[127, 63.5, -0.5, 1.5], [0, 0, 0, 0], [1, np.inf, 2, 3], [np.nan, 0, 0, 0], [1e-45, 0, 0, -1e-45]], np.float32)
    q, s = ox.quant(x)
    assert q[0, :4].tolist() == [127, 64, 0, 2] and s[0] == 1 and q.shape == (5, 64)
    assert not q[1:4].any() and s[1] == 0 and np.isnan(s[2:4]).all() and s[4] == 0 and not q[4].any()


def test_product_and_combine():
    rng = np.random.default_rng(3)
    T, k, E, d, n = 7, 2, 3, 10, 5
    x, w = rng.standard_normal((T, d)).astype(np.float32), rng.standard_normal((E, n, d)).astype(np.float32)
    q, s = ox.quant(x)
    wq, ws = ox.quant(w.reshape(E * n, d))
    wq, ws = wq.reshape(E, n, -1), ws.reshape(E, n)
    dest = rng.integers(0, E, T * k)
    src = np.argsort(dest, kind="stable").astype(np.int32)
    off = np.concatenate([[0], np.cumsum(np.bincount(dest, minlength=E))])
    y, _ = ox.product(q, s, wq, ws, off, src, T * k, gather=k, scatter=True, act=True)
    for g in range(T * k):
        z = (q[g // k, :d].astype(float) * s[g // k]) @ (wq[dest[g], :, :d].astype(float) * ws[dest[g]][:, None]).T
        assert np.allclose(y[g], torch.nn.functional.gelu(torch.from_numpy(z)).numpy())
        assert np.allclose(z, x[g // k] @ w[dest[g]].T, atol=0.15)
    wt = rng.standard_normal((T, k))
    wt[2, 1] = 0
    y[5] = np.nan  # the tuple of weight 0
    out, _ = ox.combine(y, wt, x[:, :n])
    assert np.allclose(out[0], x[0, :n] + wt[0, 0] * y[0] + wt[0, 1] * y[1]) and np.isfinite(out[2]).all()


# ---- refusals: none of these calls reaches the device -------------------------

P = 4096  # an aligned address that is never looked at


def code(fn, d, io, *more):
    return fn(C.byref(d) if d is not None else None, C.byref(io) if io is not None else None, *more)


def route_desc(**kw):
    base = dict(tokens=4, num_experts=16, top_k=2, score=0, groups=4, top_groups=2, group_best=2, renorm=1, scale=1.0)
    return pw.pw_route_desc(**{**base, **kw})


@pytest.mark.parametrize("bad", [dict(tokens=(1 << 28) + 1), dict(num_experts=1, groups=1, top_groups=1, top_k=1),
                                 dict(num_experts=260), dict(top_k=0), dict(top_k=9), dict(num_experts=4, top_k=5),
                                 dict(tokens=1 << 28, top_k=8), dict(score=2), dict(groups=0), dict(groups=5),
                                 dict(groups=32, num_experts=64), dict(top_groups=0), dict(top_groups=5), dict(group_best=0),
                                 dict(group_best=3), dict(renorm=2), dict(scale=float("inf")), dict(scale=float("nan"))])
@pytest.mark.parametrize("fn", ["pw_route", "pw_route_grad"])
def test_route_descriptors_are_refused(fn, bad):
    io = pw.pw_route_io(logits=P, experts=P, weights=P, dweights=P, dlogits=P)
    assert code(getattr(pw.lib, fn), route_desc(**bad), io, None) == pw.PW_ERR_INVALID
    assert pw.lib.pw_last_error()


def test_route_buffers_are_refused():
    full = dict(logits=P, experts=P, weights=P, dweights=P, dlogits=P)
    for fn, needs in ((pw.lib.pw_route, ("logits", "experts", "weights")),
                      (pw.lib.pw_route_grad, ("logits", "experts", "dweights", "dlogits"))):
        assert code(fn, None, pw.pw_route_io(**full), None) == pw.PW_ERR_INVALID
        assert code(fn, route_desc(), None, None) == pw.PW_ERR_INVALID
        for n in needs:
            assert code(fn, route_desc(), pw.pw_route_io(**{**full, n: None}), None) == pw.PW_ERR_INVALID
            assert code(fn, route_desc(), pw.pw_route_io(**{**full, n: P + 2}), None) == pw.PW_ERR_INVALID
        assert code(fn, route_desc(tokens=0), pw.pw_route_io(), None) == pw.PW_OK


def q8_desc(**kw):
    base = dict(rows=8, x_rows=8, d=100, n=32, num_experts=4, dtype=1, gather=0, scatter=0, gelu=0)
    return pw.pw_q8_desc(**{**base, **kw})


@pytest.mark.parametrize("bad", [dict(rows=1 << 31, x_rows=1 << 31), dict(x_rows=7), dict(gather=2, x_rows=0), dict(d=0), dict(d=65537),
                                 dict(n=0), dict(n=65537), dict(num_experts=0), dict(num_experts=257), dict(dtype=2),
                                 dict(gather=257), dict(scatter=2), dict(gelu=2)])
def test_q8_descriptors_are_refused(bad):
    need = C.c_size_t(0)
    assert pw.lib.pw_q8_product_workspace(C.byref(q8_desc(**bad)), C.byref(need)) == pw.PW_ERR_INVALID
    io = pw.pw_q8_io(x=P, w=P, w_scale=P, offsets=P, src_index=P, out=P)
    assert code(pw.lib.pw_q8_product, q8_desc(**bad), io, P, 1 << 30, None) == pw.PW_ERR_INVALID


def test_q8_buffers_are_refused():
    full = dict(x=P, w=P, w_scale=P, offsets=P, out=P)
    run = lambda d, ws=P, size=1 << 20, **kw: code(pw.lib.pw_q8_product, d, pw.pw_q8_io(**{**full, **kw}), ws, size, None)  # noqa: E731
    for n in ("w", "w_scale", "out", "offsets", "x"):
        assert run(q8_desc(), **{n: None}) == pw.PW_ERR_INVALID
        assert run(q8_desc(), **{n: P + 1}) == pw.PW_ERR_INVALID
    assert run(q8_desc(), w=P + 8) == pw.PW_ERR_INVALID                         # codes: 16 bytes
    assert run(q8_desc(), q=P, q_scale=P) == pw.PW_ERR_INVALID                  # both forms of x
    assert run(q8_desc(), x=None, q=P) == pw.PW_ERR_INVALID                     # codes without scales
    assert run(q8_desc(), src_index=P) == pw.PW_ERR_INVALID                     # an index that nothing reads
    assert run(q8_desc(gather=2)) == pw.PW_ERR_INVALID                          # gather without an index
    assert run(q8_desc(scatter=1)) == pw.PW_ERR_INVALID
    assert run(q8_desc(), ws=None) == pw.PW_ERR_INVALID
    assert run(q8_desc(), ws=P + 16) == pw.PW_ERR_INVALID
    assert run(q8_desc(), size=512) == pw.PW_ERR_NOMEM
    need = C.c_size_t(0)
    assert pw.lib.pw_q8_product_workspace(C.byref(q8_desc()), C.byref(need)) == pw.PW_OK and need.value == 8 * 128 + 256
    assert pw.lib.pw_q8_product_workspace(C.byref(q8_desc()), None) == pw.PW_ERR_INVALID
    assert run(q8_desc(rows=0, x_rows=0), w=None) == pw.PW_OK


def test_quant_and_combine_are_refused():
    q = lambda d, **kw: code(pw.lib.pw_quant_rows, pw.pw_quant_desc(*d), pw.pw_quant_io(**{**dict(x=P, q=P, scale=P), **kw}), None)  # noqa: E731
    for d in ((1 << 31, 8, 1), (4, 0, 1), (4, 65537, 1), (4, 8, 2)):
        assert q(d) == pw.PW_ERR_INVALID
    for kw in (dict(x=None), dict(q=None), dict(scale=None), dict(q=P + 8), dict(x=P + 1), dict(limit=P + 4)):
        assert q((4, 8, 1), **kw) == pw.PW_ERR_INVALID
    assert q((0, 8, 1), x=None) == pw.PW_OK
    c = lambda d, **kw: code(pw.lib.pw_topk_combine, pw.pw_combine_desc(*d), pw.pw_topk_combine_io(**{**dict(y=P, weights=P, out=P), **kw}), None)  # noqa: E731
    for d in ((1 << 31, 8, 2, 1), (4, 0, 2, 1), (4, 65537, 2, 1), (4, 8, 0, 1), (4, 8, 9, 1), (4, 8, 2, 3)):
        assert c(d) == pw.PW_ERR_INVALID
    for kw in (dict(y=None), dict(weights=None), dict(out=None), dict(y=P + 1), dict(weights=P + 2), dict(add=P + 1)):
        assert c((4, 8, 2, 1), **kw) == pw.PW_ERR_INVALID
    assert c((0, 8, 2, 1), y=None) == pw.PW_OK


def test_the_gradient_takes_the_descriptors_that_the_routing_takes():
    """What the header says of pw_route_grad: group fields that pw_route refuses are refused, here with every buffer there."""
    full = pw.pw_route_io(logits=P, experts=P, weights=P, dweights=P, dlogits=P)
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pw.h")).read()
    assert "not looked at). */\nint pw_route_grad" not in text
    for bad in (dict(groups=0), dict(top_groups=0), dict(group_best=0), dict(groups=0, top_groups=0, group_best=0)):
        d = route_desc(tokens=0, **bad)
        assert code(pw.lib.pw_route, d, full, None) == code(pw.lib.pw_route_grad, d, full, None) == pw.PW_ERR_INVALID


def test_gelu_of_infinities():
    got = ox.gelu(np.array([-np.inf, np.inf, np.nan, -1e300, 0.0, 1.0]))
    assert got[0] == 0 and got[1] == np.inf and np.isnan(got[2]) and got[3] == 0 and got[4] == 0
    assert abs(got[5] - 0.8413447460685429) < 1e-15
