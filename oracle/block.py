"""Oracle of the operators around an MoE step (test infrastructure only), in
64 bits, from their definitions in include/pw.h: the router's balance loss
with counts and gradient, the norms around a block with gate and residual
scale, and the gradients of the gated combine and of dispatch and router.

Each function also returns, where a test needs it, the sum of the absolute
values of the terms behind each output: what a rounding error is relative to.
"""
from __future__ import annotations

import numpy as np


def softmax_lse(logits):
    """(p, lse) of each row; a row of -inf alone has zeros."""
    l = logits.astype(np.float64)
    m = l.max(axis=1, keepdims=True)
    m = np.where(m == -np.inf, 0.0, m)
    z = np.exp(l - m)
    s = z.sum(axis=1, keepdims=True)
    empty = s == 0
    return np.where(empty, 0.0, z / np.where(empty, 1.0, s)), np.where(empty, 0.0, m + np.log(np.where(empty, 1.0, s)))[:, 0]


def balance(logits, experts, valid, balance_coef, z_coef):
    """(counts [E + 1], prob_mean [E], loss [2], p, lse) over the valid tokens."""
    E, k = logits.shape[1], experts.shape[1]
    v = np.ones(logits.shape[0], bool) if valid is None else valid.astype(bool)
    n = int(v.sum())
    ids = experts[v].reshape(-1)
    counts = np.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
    p, lse = softmax_lse(logits[v])
    if n == 0:
        return np.zeros(E + 1, np.int64), np.zeros(E), np.zeros(2), p, lse
    mean = p.sum(axis=0) / n
    loss = np.array([balance_coef * E * (counts / (k * n) * mean).sum(), z_coef * (lse ** 2).mean()])
    return np.concatenate([counts, [n]]), mean, loss, p, lse


def router_grad(logits, experts, counts, gates, dgates, valid, grad_loss, balance_coef, z_coef):
    """dlogits, and a bound on the absolute values of its terms per element."""
    T, E = logits.shape
    k = experts.shape[1]
    v = np.ones(T, bool) if valid is None else valid.astype(bool)
    n = int(counts[E])
    inv = 1.0 / n if n else 0.0
    u = np.ones(2) if grad_loss is None else grad_loss.astype(np.float64)
    safe = np.where(v[:, None], logits, 0.0)
    p, lse = softmax_lse(safe)
    c = counts[:E].astype(np.float64) * inv - k / E
    cb, cz = u[0] * balance_coef * E / k * inv, u[1] * 2 * z_coef * inv
    d = p * (cb * (c - (p * c).sum(axis=1, keepdims=True)) + cz * lse[:, None])
    size = p * (abs(cb) * (np.abs(c) + (p * np.abs(c)).sum(axis=1, keepdims=True)) + abs(cz) * (np.abs(lse[:, None]) + 1))
    if gates is not None:
        g, dg = np.where(v[:, None], gates, 0).astype(np.float64), np.where(v[:, None], dgates, 0).astype(np.float64)
        dot, adot = (g * dg).sum(axis=1), np.abs(g * dg).sum(axis=1)
        for s in range(k):
            e = experts[:, s]
            t = np.flatnonzero((e >= 0) & (e < E))
            d[t, e[t]] += g[t, s] * (dg[t, s] - dot[t])
            size[t, e[t]] += np.abs(g[t, s]) * (np.abs(dg[t, s]) + adot[t])
    d[~v] = 0
    size[~v] = 0
    return d, size


def rstd(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def _gate_rows(gate, rows):
    return np.repeat(gate.astype(np.float64), rows // gate.shape[0], axis=0)


def block_norm(x, y, w_y, gate, w_r, x_scale, y_scale, eps):
    """(r, h or None, size of r's terms)."""
    r = x_scale * x.astype(np.float64)
    size = np.abs(r)
    if y is not None:
        n = y.astype(np.float64)
        if w_y is not None:
            n = n * rstd(n, eps) * w_y.astype(np.float64)
        if gate is not None:
            n = n * _gate_rows(gate, x.shape[0])
        r = r + y_scale * n
        size = size + np.abs(y_scale * n)
    h = None if w_r is None else r * rstd(r, eps) * w_r.astype(np.float64)
    return r, h, size


def block_norm_grad(dr, dh, r, y, w_y, gate, w_r, x_scale, y_scale, eps, valid=None, u=0.0):
    """Gradients {dx, dy, dw_y, dgate, dw_r}, and for each the largest error of an
    fp32 evaluation whose every term is off by at most u of its value (before
    the results are rounded to their type)."""
    rows, d = (dr if dr is not None else dh).shape
    v = np.ones(rows, bool) if valid is None else valid.astype(bool)

    def take(t):
        return None if t is None else np.where(v[:, None], t, 0).astype(np.float64)

    dr, dh, r, y = take(dr), take(dh), take(r), take(y)
    out, err = {}, {}
    D = np.zeros((rows, d)) if dr is None else dr.copy()
    size = np.abs(D)
    if w_r is not None:
        s, G = rstd(r, eps), dh * w_r.astype(np.float64)
        D = D + s * (G - r * s * s * (G * r).mean(axis=1, keepdims=True))
        size = size + s * (np.abs(G) + np.abs(r) * s * s * np.abs(G * r).mean(axis=1, keepdims=True))
        out["dw_r"], err["dw_r"] = (dh * r * s).sum(axis=0), u * np.abs(dh * r * s).sum(axis=0)
    eD = u * size
    out["dx"], err["dx"] = x_scale * D, abs(x_scale) * eD
    if y is not None:
        wy = np.ones(d) if w_y is None else w_y.astype(np.float64)
        gr = np.ones((rows, d)) if gate is None else _gate_rows(gate, rows)
        t = np.ones((rows, 1)) if w_y is None else rstd(y, eps)
        q = y_scale * D * gr * wy
        eq = np.abs(y_scale * gr * wy) * eD + u * np.abs(q)
        Q, eQ = D * y * t, eD * np.abs(y * t) + u * np.abs(D * y * t)
        if w_y is None:
            out["dy"], err["dy"] = q, eq
        else:
            out["dy"] = t * (q - y * t * t * (q * y).mean(axis=1, keepdims=True))
            err["dy"] = t * (eq + u * np.abs(q) + np.abs(y) * t * t * ((eq * np.abs(y)).mean(axis=1, keepdims=True)
                                                                     + u * np.abs(q * y).mean(axis=1, keepdims=True)))
            out["dw_y"] = (y_scale * gr * Q).sum(axis=0)
            err["dw_y"] = np.abs(y_scale * gr * eQ).sum(axis=0)
        if gate is not None:
            n = gate.shape[0]
            out["dgate"] = (y_scale * wy * Q).reshape(n, rows // n, d).sum(axis=1)
            err["dgate"] = np.abs(y_scale * wy * eQ).reshape(n, rows // n, d).sum(axis=1)
    return out, err


def slots(src_index, kept, tokens):
    """slot_of [T, 2] of an index whose first `kept` rows hold tuples."""
    s = np.full(2 * tokens, -1, np.int64)
    s[src_index[:kept]] = np.arange(kept)
    return s.reshape(tokens, 2)


def combine_grad(dout, y, gates, src_index, kept, valid=None):
    """(dy [kept, d], dgates [T, 2], sum of |terms| of dgates)."""
    T = dout.shape[0]
    v = np.ones(T, bool) if valid is None else valid.astype(bool)
    t, s = src_index[:kept] // 2, src_index[:kept] % 2
    rows = np.where(v[t][:, None], dout[t], 0).astype(np.float64)
    g = np.where(v[t], gates[t, s], 0).astype(np.float64)
    yk = np.where(v[t][:, None], y[:kept], 0).astype(np.float64)
    dg, size = np.zeros((T, 2)), np.zeros((T, 2))
    dg[t, s] = (rows * yk).sum(axis=1)
    size[t, s] = np.abs(rows * yk).sum(axis=1)
    return g[:, None] * rows, dg, size


def dispatch_grad(dxd, dlogits, w_router, x, slot_of, valid=None):
    """(dx, size of its product's terms, size of its rows' terms, dW, size of dW's terms)."""
    T = dlogits.shape[0]
    v = np.ones(T, bool) if valid is None else valid.astype(bool)
    dl, w = dlogits.astype(np.float64), w_router.astype(np.float64)
    dx = dl @ w.T
    size = np.abs(dl) @ np.abs(w).T
    rows = np.zeros_like(dx)
    for s in range(2):
        have = slot_of[:, s] >= 0
        add = dxd[slot_of[have, s]].astype(np.float64)
        dx[have] += add
        rows[have] += np.abs(add)
    dx[~v] = 0
    xv = np.where(v[:, None], x, 0).astype(np.float64)
    dlv = np.where(v[:, None], dl, 0)
    return dx, size, rows, xv.T @ dlv, np.abs(xv).T @ np.abs(dlv)
