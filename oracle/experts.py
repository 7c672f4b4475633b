"""Oracle of the operators that serve a mixture of experts with any top-k (test
infrastructure only), in 64 bits, from their definitions in include/pw.h: the
routing and its gradient, rows as 8-bit codes, the products and the combine.
"""
from __future__ import annotations

import math

import numpy as np

U = 2.0 ** -24  # an fp32 rounding


def _usable(logits):
    """Logits as they count: NaN is none, +infinity the largest finite value."""
    l = np.where(np.isnan(logits), -np.inf, logits).astype(np.float64)
    return np.minimum(l, float(np.finfo(np.float32).max))


def scores(logits, sigmoid):
    """(s [T][E], log s up to one constant a row): rows without a logit have zeros."""
    l = _usable(logits)
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        if sigmoid:
            return 1.0 / (1.0 + np.exp(-l)), -np.logaddexp(0.0, -l)
        m = l.max(axis=1, keepdims=True)
        m = np.where(m == -np.inf, 0.0, m)
        z = np.exp(l - m)
        total = z.sum(axis=1, keepdims=True)
        return np.where(total == 0, 0.0, z / np.where(total == 0, 1.0, total)), l


def _weights(logits, experts, sigmoid, renorm):
    """Scores of the chosen experts (0 where there is none), divided by their sum if renorm."""
    T, E = logits.shape
    s, ls = scores(logits, sigmoid)
    live = (experts >= 0) & (experts < E)
    at = np.where(live, experts, 0)
    if not renorm:
        return np.where(live, np.take_along_axis(s, at, 1), 0.0)
    l = np.where(live, np.take_along_axis(ls, at, 1), -np.inf)
    m = l.max(axis=1, keepdims=True)
    v = np.exp(l - np.where(m == -np.inf, 0.0, m))
    total = v.sum(axis=1, keepdims=True)
    return np.where(total == 0, 0.0, v / np.where(total == 0, 1.0, total))


def route(logits, bias, valid, k, sigmoid, groups=1, top_groups=1, group_best=2, renorm=True, scale=1.0):
    """(experts [T][k], weights [T][k] in 64 bits)."""
    T, E = logits.shape
    s, _ = scores(logits, sigmoid)
    b = np.zeros(E) if bias is None else np.where(np.isnan(bias), -np.inf, bias).astype(np.float64)
    l = _usable(logits)
    # scores grow with their logits: alone, their order is that of the logits, also where they round to one value
    c = l.copy() if bias is None and top_groups == groups else s + b
    c[(l == -np.inf) | (b == -np.inf)] = -np.inf
    if valid is not None:
        c[~np.asarray(valid, bool)] = -np.inf
    if top_groups < groups:
        best = -np.sort(-c.reshape(T, groups, E // groups), axis=2)[:, :, :group_best]
        mark = np.where(best[:, :, 0] == -np.inf, -np.inf, np.where(best == -np.inf, 0, best).sum(axis=2))
        order = np.argsort(-mark, axis=1, kind="stable")[:, :top_groups]
        kept = np.zeros((T, groups), bool)
        np.put_along_axis(kept, order, True, axis=1)
        c[~np.repeat(kept, E // groups, axis=1)] = -np.inf
    experts = np.argsort(-c, axis=1, kind="stable")[:, :k]
    experts = np.where(np.take_along_axis(c, experts, 1) == -np.inf, E, experts)
    return experts, scale * _weights(logits, experts, sigmoid, renorm)


def route_grad(logits, experts, dweights, valid, add, sigmoid, renorm=True, scale=1.0):
    """(dlogits [T][E], the absolute values of its terms)."""
    T, E = logits.shape
    v = np.ones(T, bool) if valid is None else valid.astype(bool)
    l = np.where(v[:, None], logits, 0)
    live = (experts >= 0) & (experts < E) & v[:, None]
    live &= _usable(np.take_along_axis(l, np.where(live, experts, 0), 1)) > -np.inf
    ids = np.where(live, experts, -1)
    g = np.where(live, dweights, 0).astype(np.float64) * scale
    s, _ = scores(l, sigmoid)
    w = _weights(l, ids, sigmoid, renorm)
    d, size = np.zeros((T, E)), np.zeros((T, E))
    dot, adot = (w * g).sum(1, keepdims=True), np.abs(w * g).sum(1, keepdims=True)
    with np.errstate(over="ignore"):
        q = 1.0 / (1.0 + np.exp(_usable(np.take_along_axis(l, np.where(live, experts, 0), 1))))  # 1 - s for sigmoid
    if renorm:
        part, apart = w * (g - dot), w * (np.abs(g) + adot)
        if sigmoid:
            part, apart = part * q, apart * q
    elif sigmoid:
        part = w * g * q
        apart = np.abs(part)
    else:
        part, apart = w * g, np.abs(w * g)
        d -= s * dot
        size += s * adot
    for j in range(experts.shape[1]):
        t = np.flatnonzero(live[:, j])
        d[t, experts[t, j]] += part[t, j]
        size[t, experts[t, j]] += apart[t, j]
    if add is not None:
        a = np.where(v[:, None], add, 0).astype(np.float64)
        d, size = d + a, size + np.abs(a)
    d[~v], size[~v] = 0, 0
    return d, size


def q8_row(d):
    return (d + 63) // 64 * 64


def quant(x):
    """(codes [rows][q8_row(d)] int8, scale [rows] fp32), bit for bit."""
    rows, d = x.shape
    x = x.astype(np.float32)
    with np.errstate(all="ignore"):
        scale = np.abs(x).max(axis=1) * (np.float32(1) / np.float32(127))
        scale = np.where(np.isfinite(x).all(axis=1), scale, np.float32(np.nan)).astype(np.float32)
        some = scale > 0
        z = np.rint(x / np.where(some, scale, np.float32(1))[:, None]).clip(-127, 127)
    q = np.zeros((rows, q8_row(d)), np.int8)
    q[some, :d] = z[some].astype(np.int8)
    return q, scale


def gelu(z):
    """z Phi(z), 0 of -infinity."""
    erfc = np.frompyfunc(math.erfc, 1, 1)
    return np.maximum(z, -np.finfo(np.float64).max) * 0.5 * erfc(-z / math.sqrt(2.0)).astype(np.float64)


def product(q, q_scale, w, w_scale, offsets, src_index, rows, gather=0, scatter=False, act=False, out=None):
    """(out [rows][n] in 64 bits, z before the activation); rows that nothing names hold `out`'s."""
    E, n, _ = w.shape
    out = np.zeros((rows, n)) if out is None else out.astype(np.float64).copy()
    pre = np.zeros((rows, n))
    bounds = [0, rows] if offsets is None else np.maximum.accumulate(np.clip(offsets, 0, min(rows, max(0, offsets[E]))))
    most = min(rows, 1 << 31) if not gather else q.shape[0] * gather if not scatter else min(rows, q.shape[0] * gather)
    for e in range(E):
        i = np.arange(bounds[e], bounds[e + 1])
        g = i if src_index is None else src_index[i].astype(np.int64)
        ok = np.ones(i.shape, bool) if src_index is None else (g >= 0) & (g < most)
        i, g = i[ok], g[ok]
        a, o = (g // gather if gather else i), (g if scatter else i)
        z = (q[a].astype(np.float64) @ w[e].astype(np.float64).T) * q_scale[a].astype(np.float64)[:, None]
        pre[o] = z * w_scale[e].astype(np.float64)
        out[o] = gelu(pre[o]) if act else pre[o]
    return out, pre


def combine(y, weights, add):
    """(out, the absolute values of its terms)."""
    T, k = weights.shape
    on = (weights != 0)[:, :, None]
    terms = np.where(on, weights.astype(np.float64)[:, :, None] * np.where(on, y.reshape(T, k, -1), 0), 0)
    a = 0 if add is None else add.astype(np.float64)
    return terms.sum(1) + a, np.abs(terms).sum(1) + np.abs(a)
