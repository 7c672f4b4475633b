"""The oracle's gradients of the operators around an MoE step against central
differences of their own forward definitions, in 64 bits on the CPU, and the
argument errors of the entry points, which need no device."""
import ctypes as C

import numpy as np
import pytest

import sparse_shard_exchange_amd as pw
from oracle import block as ob

STEP = 1e-5   # central differences: error STEP^2 f''' / 6 + 2^-52 f / STEP, both below 1e-8 here


def difference(f, x, weight):
    """d/dx of sum(weight * f(x)) by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + STEP
        hi = (weight * f()).sum()
        x[i] = keep - STEP
        lo = (weight * f()).sum()
        x[i] = keep
        g[i] = (hi - lo) / (2 * STEP)
    return g


def close(a, b):
    assert np.all(np.abs(a - b) <= 1e-7 * (1 + np.abs(b))), np.abs(a - b).max()


def test_router_gradient_matches_differences():
    rng = np.random.default_rng(1)
    T, E, k = 7, 5, 2
    l = rng.standard_normal((T, E))
    valid = np.array([1, 1, 0, 1, 1, 1, 1], bool)
    ex = np.argsort(-l, axis=1)[:, :k]
    dg, u = rng.standard_normal((T, k)), rng.random(2)
    counts = ob.balance(l, ex, valid, 0.7, 0.3)[0]

    def gates():
        kept = np.exp(np.take_along_axis(l, ex, axis=1))
        return kept / kept.sum(axis=1, keepdims=True) * valid[:, None]

    d, _ = ob.router_grad(l, ex, counts, gates() + 0.0, dg, valid, u, 0.7, 0.3)
    want = difference(lambda: ob.balance(l, ex, valid, 0.7, 0.3)[2], l, u) + difference(gates, l, dg)
    close(d, want)
    assert np.all(d[2] == 0)


@pytest.mark.parametrize("norm_y,gates,pre", [(True, 2, True), (False, 3, True), (True, 0, False), (False, 0, True)])
def test_norm_gradients_match_differences(norm_y, gates, pre):
    rng = np.random.default_rng(2)
    T, d, ax, ay, eps = 6, 5, 0.9, 0.6, 1e-3
    x, y = rng.standard_normal((T, d)), rng.standard_normal((T, d))
    w_y = rng.standard_normal(d) if norm_y else None
    gate = rng.standard_normal((gates, d)) if gates else None
    w_r = rng.standard_normal(d) if pre else None
    dr, dh = rng.standard_normal((T, d)), rng.standard_normal((T, d))

    def f():
        r, h, _ = ob.block_norm(x, y, w_y, gate, w_r, ax, ay, eps)
        return np.stack([r, h if pre else np.zeros_like(r)])

    r = f()[0]
    out, _ = ob.block_norm_grad(dr, dh if pre else None, r, y, w_y, gate, w_r, ax, ay, eps)
    weight = np.stack([dr, dh])
    for name, leaf in (("dx", x), ("dy", y), ("dw_y", w_y), ("dgate", gate), ("dw_r", w_r)):
        if leaf is not None:
            close(out[name], difference(f, leaf, weight))


def test_combine_and_dispatch_gradients_match_differences():
    rng = np.random.default_rng(3)
    T, d, E = 5, 4, 3
    src = np.array([0, 3, 9, 2, 5, 6, 8], np.int64)   # three tuples of ten dropped
    kept = src.size
    y, g, dout = rng.standard_normal((kept, d)), rng.random((T, 2)), rng.standard_normal((T, d))

    def combine():
        out = np.zeros((T, d))
        np.add.at(out, src // 2, g[src // 2, src % 2][:, None] * y)
        return out

    dy, dg, _ = ob.combine_grad(dout, y, g, src, kept)
    close(dy, difference(combine, y, dout))
    close(dg, difference(combine, g, dout))
    slot_of = ob.slots(src, kept, T)
    x, w = rng.standard_normal((T, d)), rng.standard_normal((d, E))
    dxd, dl = rng.standard_normal((kept, d)), rng.standard_normal((T, E))
    dx, _, _, dw, _ = ob.dispatch_grad(dxd, dl, w, x, slot_of)
    close(dx, difference(lambda: x[src // 2], x, dxd) + difference(lambda: x @ w, x, dl))
    close(dw, difference(lambda: x @ w, w, dl))


# ---- argument errors (include/pw.h), before any device call ------------------------

INV, NOMEM, UNS = pw.PW_ERR_INVALID, pw.PW_ERR_NOMEM, pw.PW_ERR_UNSUPPORTED
P = 1 << 20   # never dereferenced


def test_struct_sizes_match_the_header():
    assert C.sizeof(pw.pw_balance_desc) == 24 and C.sizeof(pw.pw_balance_io) == 80
    assert C.sizeof(pw.pw_moe_grad_desc) == 32
    assert C.sizeof(pw.pw_combine_grad_io) == 72 and C.sizeof(pw.pw_dispatch_grad_io) == 64
    assert C.sizeof(pw.pw_norm_desc) == 32 and C.sizeof(pw.pw_norm_io) == 120


def bal(**kw):
    base = dict(tokens=4096, num_experts=64, top_k=2, balance_coef=0.1, z_coef=0.0)
    base.update(kw)
    return pw.pw_balance_desc(*base.values())


@pytest.mark.parametrize("bad", [
    dict(tokens=(1 << 28) + 1), dict(num_experts=1), dict(num_experts=257), dict(top_k=0), dict(top_k=9),
    dict(num_experts=3, top_k=4), dict(tokens=1 << 28, top_k=8), dict(balance_coef=float("nan")),
    dict(z_coef=float("inf"))])
def test_balance_descriptor_errors(bad):
    n, io = C.c_size_t(0), pw.pw_balance_io()
    assert pw.lib.pw_router_balance_workspace(C.byref(bal(**bad)), C.byref(n)) == INV
    assert pw.lib.pw_last_error()
    assert pw.lib.pw_router_balance(C.byref(bal(**bad)), C.byref(io), None, 0, None) == INV
    assert pw.lib.pw_router_grad(C.byref(bal(**bad)), C.byref(io), None) == INV


def test_balance_buffer_errors():
    n = C.c_size_t(0)
    assert pw.lib.pw_router_balance_workspace(None, C.byref(n)) == INV
    assert pw.lib.pw_router_balance_workspace(C.byref(bal()), None) == INV
    assert pw.lib.pw_router_balance_workspace(C.byref(bal()), C.byref(n)) == 0 and n.value > 0
    io = pw.pw_balance_io()
    d = bal()
    call = lambda ws, b: pw.lib.pw_router_balance(C.byref(d), C.byref(io), ws, b, None)  # noqa: E731
    assert pw.lib.pw_router_balance(C.byref(d), None, P, n.value, None) == INV
    assert call(P, n.value) == INV                      # no buffers
    io.logits = io.experts = io.counts = P
    assert call(P, n.value) == INV                      # no loss
    io.loss = P
    assert call(None, 0) == INV                         # no workspace
    assert call(P + 8, n.value) == INV                  # not aligned
    assert call(P, n.value - 1) == NOMEM
    assert pw.lib.pw_router_grad(C.byref(d), C.byref(io), None) == INV   # no dlogits
    io.dlogits = io.gates = P
    assert pw.lib.pw_router_grad(C.byref(d), C.byref(io), None) == INV   # gates without dgates
    io.dgates, io.experts = P, None
    assert pw.lib.pw_router_grad(C.byref(d), C.byref(io), None) == INV   # gates without experts


@pytest.mark.parametrize("name", ["logits", "experts", "counts", "loss", "gates", "dgates", "grad_loss", "dlogits"])
def test_balance_refuses_split_elements(name):
    io = pw.pw_balance_io(*([P] * 10))
    io.valid = None
    setattr(io, name, P + 2)
    assert pw.lib.pw_router_balance(C.byref(bal()), C.byref(io), P, 1 << 30, None) == INV
    assert pw.lib.pw_router_grad(C.byref(bal()), C.byref(io), None) == INV


def moe(**kw):
    base = dict(tokens=512, rows=1024, d=512, num_experts=8, top_k=2, dtype=pw.PW_BF16)
    base.update(kw)
    return pw.pw_moe_grad_desc(*base.values())


@pytest.mark.parametrize("bad,code", [
    (dict(tokens=(1 << 28) + 1), INV), (dict(rows=1025), INV), (dict(d=0), INV), (dict(d=320), INV), (dict(d=1536), INV),
    (dict(num_experts=1), INV), (dict(num_experts=65), INV), (dict(top_k=1), UNS), (dict(dtype=pw.PW_F32), INV)])
def test_moe_grad_descriptor_errors(bad, code):
    n = C.c_size_t(0)
    c, s = pw.pw_combine_grad_io(), pw.pw_dispatch_grad_io()
    assert pw.lib.pw_moe_dispatch_grad_workspace(C.byref(moe(**bad)), C.byref(n)) == code
    assert pw.lib.pw_moe_combine_grad(C.byref(moe(**bad)), C.byref(c), None) == code
    assert pw.lib.pw_moe_dispatch_grad(C.byref(moe(**bad)), C.byref(s), None, 0, None) == code


@pytest.mark.parametrize("name", ["dout", "y", "gates", "src_index", "offsets", "dy", "dgates", "slot_of"])
def test_combine_grad_buffer_errors(name):
    io = pw.pw_combine_grad_io(*([P] * 5), None, P, P, P)
    setattr(io, name, None)
    assert pw.lib.pw_moe_combine_grad(C.byref(moe()), C.byref(io), None) == INV
    if name in ("dout", "y", "dy", "gates", "dgates", "slot_of"):
        setattr(io, name, P + 4)
        assert pw.lib.pw_moe_combine_grad(C.byref(moe()), C.byref(io), None) == INV


def test_dispatch_grad_buffer_errors():
    d, n = moe(), C.c_size_t(0)
    assert pw.lib.pw_moe_dispatch_grad_workspace(C.byref(d), C.byref(n)) == 0 and n.value > 0
    names = [f for f, _ in pw.pw_dispatch_grad_io._fields_ if f != "valid"]
    for name in names[:-1]:
        io = pw.pw_dispatch_grad_io(P, P, P, P, P, None, P, P)
        setattr(io, name, None)
        assert pw.lib.pw_moe_dispatch_grad(C.byref(d), C.byref(io), P, n.value, None) == INV, name
    io = pw.pw_dispatch_grad_io(P, P, P, P, P, None, P, P)
    for ws, b, code in ((None, 0, INV), (P + 64, n.value, INV), (P, n.value - 256, NOMEM)):
        assert pw.lib.pw_moe_dispatch_grad(C.byref(d), C.byref(io), ws, b, None) == code
    io.x = P + 8
    assert pw.lib.pw_moe_dispatch_grad(C.byref(d), C.byref(io), P, n.value, None) == INV


def norm(**kw):
    base = dict(rows=64, d=256, dtype=pw.PW_BF16, gates=0, x_scale=1.0, y_scale=1.0, eps=1e-6)
    base.update(kw)
    return pw.pw_norm_desc(*base.values())


@pytest.mark.parametrize("bad", [
    dict(rows=1 << 31), dict(d=0), dict(d=8193), dict(dtype=2), dict(gates=3), dict(x_scale=float("inf")),
    dict(y_scale=float("nan")), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan"))])
def test_norm_descriptor_errors(bad):
    n, io = C.c_size_t(0), pw.pw_norm_io()
    assert pw.lib.pw_block_norm_grad_workspace(C.byref(norm(**bad)), C.byref(n)) == INV
    assert pw.lib.pw_block_norm(C.byref(norm(**bad)), C.byref(io), None) == INV
    assert pw.lib.pw_block_norm_grad(C.byref(norm(**bad)), C.byref(io), None, 0, None) == INV


@pytest.mark.parametrize("given,gates", [
    ("x", 0), ("x w_y w_r h", 0), ("x gate w_r h", 2), ("x y r gate", 0), ("x y r", 2), ("x y", 0), ("x w_r", 0),
    ("x y r h", 0), ("y w_y r", 0)])
def test_norm_buffer_errors(given, gates):
    io = pw.pw_norm_io()
    for f in given.split():
        setattr(io, f, P)
    assert pw.lib.pw_block_norm(C.byref(norm(gates=gates)), C.byref(io), None) == INV


@pytest.mark.parametrize("drop", ["dw_y", "dgate", "dw_r", "dh", "r", "dx", "dy"])
def test_norm_grad_buffer_errors(drop):
    io = pw.pw_norm_io(*([P] * 15))
    io.valid = None
    setattr(io, drop, None)
    assert pw.lib.pw_block_norm_grad(C.byref(norm(gates=2)), C.byref(io), P, 1 << 30, None) == INV


@pytest.mark.parametrize("name,dtype,off", [("x", pw.PW_BF16, 1), ("w_r", pw.PW_F32, 2), ("dh", pw.PW_F32, 2),
                                            ("dw_y", pw.PW_BF16, 2), ("dx", pw.PW_BF16, 1)])
def test_norm_refuses_split_elements(name, dtype, off):
    io = pw.pw_norm_io(*([P] * 15))
    io.valid = None
    setattr(io, name, P + off)
    assert pw.lib.pw_block_norm_grad(C.byref(norm(gates=2, dtype=dtype)), C.byref(io), P, 1 << 30, None) == INV
    assert pw.lib.pw_block_norm(C.byref(norm(gates=2, dtype=dtype)), C.byref(io), None) == INV


def test_norm_grad_workspace_errors():
    d, n = norm(rows=4096), C.c_size_t(0)
    assert pw.lib.pw_block_norm_grad_workspace(C.byref(d), C.byref(n)) == 0 and n.value > 0
    io = pw.pw_norm_io()
    io.w_r = io.dw_r = io.dh = io.r = io.dx = P
    for ws, b, code in ((None, 0, INV), (P + 128, n.value, INV), (P, n.value - 1, NOMEM)):
        assert pw.lib.pw_block_norm_grad(C.byref(d), C.byref(io), ws, b, None) == code
    io.w_r = io.dr = None                                # neither part
    assert pw.lib.pw_block_norm_grad(C.byref(d), C.byref(io), P, n.value, None) == INV


def test_missing_dispatched_rows_are_refused():
    """The number of rows comes from y and dxd: without them, or from scalars, there is none."""
    import torch
    f = pw.MoEGrad(4, 256, 2, device="cuda:0")
    for call in (lambda t: f.combine(None, t, None, None, None), lambda t: f.dispatch(t, None, None)):
        for t in (None, torch.zeros(()), torch.zeros(8)):
            with pytest.raises(pw.PwError) as e:
                call(t)
            assert e.value.code == INV
