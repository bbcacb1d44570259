"""fp64 reference of differential attention, the distance-bucket bias and counter-based dropout.

Rows are taken one at a time and every gradient is the textbook formula of its
own step (softmax, difference of maps, weighted sum).  ``attention_bounds``
gives, beside each output, a first-order bound on how far a computation in
32-bit floats may be off: it carries the rounding of each step through the
formulas, u = 2^-24 for each rounding of a value to nearest.
"""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24   # unit roundoff of fp32


# ---------------------------------------------------------------- generator

def philox4x32(counter, key, rounds=10):
    """Philox4x32 words [n, 4] of uint32 counters [n, 4] under a key of two words."""
    c = [np.asarray(counter[..., i], np.uint64) for i in range(4)]
    k0, k1 = (int(k) for k in key)
    low = np.uint64(0xFFFFFFFF)
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & low, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1),
             p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1).astype(np.uint32)


def keep_factors(index, p, seed, step, site):
    """0 or 65536/(65536-t) for each decision index (any shape)."""
    index = np.asarray(index, np.int64)
    t = int(np.floor(p * 65536 + 0.5))
    if t == 0:
        return np.ones(index.shape)
    seed &= (1 << 64) - 1
    j = (index >> 3).reshape(-1)
    ctr = np.stack([j & 0xFFFFFFFF, j >> 32, np.full_like(j, step & 0xFFFFFFFF), np.full_like(j, site)], -1)
    words = philox4x32(ctr, (seed & 0xFFFFFFFF, seed >> 32)).astype(np.int64)
    part = (index & 7).reshape(-1)
    word = words[np.arange(len(j)), part >> 1]
    draw = np.where(part & 1, word >> 16, word & 0xFFFF)
    return np.where(draw >= t, 65536.0 / (65536 - t), 0.0).reshape(index.shape)


def dropout_factors(n_rows, lmax, C, share, p, seed, step, site):
    """Factors [n_rows, K, C]."""
    K = (lmax + 1) ** 2
    row = np.arange(n_rows)[:, None, None]
    deg = np.asarray([l for l in range(lmax + 1) for _ in range(2 * l + 1)])[None, :, None]
    c = np.arange(C)[None, None, :]
    if share == "row":
        idx = np.broadcast_to(row, (n_rows, K, C))
    elif share == "channel":
        idx = np.broadcast_to(row * C + c, (n_rows, K, C))
    else:
        idx = (row * (lmax + 1) + deg) * C + c
    return keep_factors(idx, p, seed, step, site)


# --------------------------------------------------------------------- bias

def buckets(dist, borders):
    with np.errstate(invalid="ignore"):
        return (np.asarray(dist, np.float64)[:, None] >= np.asarray(borders, np.float64)[None, :]).sum(1)


def bias_forward(dist, borders, table):
    return np.asarray(table, np.float64)[buckets(dist, borders)]


def bias_backward(dist, borders, grad_bias):
    g = np.asarray(grad_bias, np.float64)
    out = np.zeros((len(borders) + 1, g.shape[1]))
    np.add.at(out, buckets(dist, borders), g)
    return out


# ---------------------------------------------------------------- attention

def _row(q, k, bias, live, scale):
    """Logits and softmax weights [n, H, 2] of one row, with the roundoff of the logits."""
    prod = q[None] * k
    l = scale * prod.sum(-1) + bias
    l = np.where(live[:, None, None] & (bias != -np.inf), l, -np.inf)
    M = l.max(0, initial=-np.inf)
    M = np.where(np.isfinite(M), M, 0.0)
    e = np.exp(l - M)
    S = e.sum(0)
    a = np.divide(e, S, out=np.zeros_like(e), where=S > 0)
    n, D = len(l), q.shape[-1]
    fin = np.where(np.isfinite(l), l, 0.0)
    finb = np.where(np.isfinite(bias), bias, 0.0)
    # a product sum of D terms in any order, times the scale, plus the bias
    dl = U32 * ((D + 2) * abs(scale) * np.abs(prod).sum(-1) + 2 * np.abs(fin) + np.abs(finb))
    # exp of a rounded argument, the row's sum, the reciprocal
    rel = dl + (a * dl).sum(0) + U32 * (n + 12 + 2 * np.abs(fin - M) + (a * 2 * np.abs(fin - M)).sum(0))
    return l, a, rel


def _attention(row_ptr, src, q, k, v, lam, scale, bias, mask, factors, grad_out):
    row_ptr, src = np.asarray(row_ptr, np.int64), np.asarray(src, np.int64)
    q, k, v, lam = (np.asarray(t, np.float64) for t in (q, k, v, lam))
    n_dst, n_src, E, H = len(row_ptr) - 1, len(v), len(src), len(lam)
    K, C = v.shape[1:]
    Ch = C // H
    bias = np.zeros((E, H, 2)) if bias is None else np.asarray(bias, np.float64).reshape(E, H, 2)
    live = (src >= 0) & (src < n_src)
    if mask is not None:
        live &= np.asarray(mask) != 0
    m = np.ones((E, H)) if factors is None else factors
    at = np.where((src >= 0) & (src < n_src), src, 0)
    out, out_b = np.zeros((n_dst, K, C)), np.zeros((n_dst, K, C))
    res = dict(out=out)
    bnd = dict(out=out_b)
    if grad_out is not None:
        go = np.asarray(grad_out, np.float64).reshape(n_dst, K, H, Ch)
        for name, shape in (("grad_q", q.shape), ("grad_k", k.shape), ("grad_v", (n_src, K, H, Ch)),
                            ("grad_lam", (H,)), ("grad_bias", (E, H, 2))):
            res[name], bnd[name] = np.zeros(shape), np.zeros(shape)
        terms_k, terms_v = np.zeros(k.shape), np.zeros((n_src, K, H, Ch))
    for d in range(n_dst):
        e = np.arange(row_ptr[d], row_ptr[d + 1])
        n = len(e)
        if n == 0:
            continue
        s, ok = at[e], live[e]
        ks = np.where(ok[:, None, None, None], k[s], 0.0)
        b_in = bias[e]
        hidden = b_in == -np.inf
        ks = np.where(hidden[..., None], 0.0, ks)           # a masked place may hold anything
        l, a, rel = _row(q[d], ks, b_in, ok, scale)
        fl = np.stack([np.ones(H), -lam], -1)
        w = m[e] * (fl * a).sum(-1)
        dw = m[e] * (np.abs(fl) * a * (rel + 2 * U32)).sum(-1) + 2 * U32 * np.abs(w)
        used = (a != 0).any(-1) & (m[e] != 0)
        vs = np.where(used[:, None, :, None], v[s].reshape(n, K, H, Ch), 0.0)
        out[d] = (w[:, None, :, None] * vs).sum(0).reshape(K, C)
        out_b[d] = ((dw + (n + 1) * U32 * np.abs(w))[:, None, :, None] * np.abs(vs)).sum(0).reshape(K, C)
        if grad_out is None:
            continue
        alive = (a != 0).any(-1)
        va = np.where(alive[:, None, :, None], v[s].reshape(n, K, H, Ch), 0.0)
        va = np.where((m[e] != 0)[:, None, :, None], va, 0.0)
        u = m[e] * (go[d][None] * va).sum((1, 3))
        du = m[e] * (K * Ch + 2) * U32 * np.abs(go[d][None] * va).sum((1, 3))
        t = (a * u[..., None]).sum(0)
        dt = (a * (rel * np.abs(u)[..., None] + du[..., None] + (n + 1) * U32 * np.abs(u)[..., None])).sum(0)
        g = fl * a * (u[..., None] - t)
        dg = np.abs(fl) * a * ((rel + 4 * U32) * (np.abs(u)[..., None] + np.abs(t)) + du[..., None] + dt)
        res["grad_bias"][e], bnd["grad_bias"][e] = g, dg
        res["grad_q"][d] = scale * (g[..., None] * ks).sum(0)
        bnd["grad_q"][d] = abs(scale) * ((dg + (n + 2) * U32 * np.abs(g))[..., None] * np.abs(ks)).sum(0)
        qd = np.where((a != 0)[..., None], q[d][None], 0.0)
        np.add.at(res["grad_k"], s, scale * g[..., None] * qd)
        np.add.at(bnd["grad_k"], s, abs(scale) * dg[..., None] * np.abs(qd))
        np.add.at(terms_k, s, abs(scale) * np.abs(g)[..., None] * np.abs(qd))
        god = np.where(used[:, None, :, None], go[d][None], 0.0)
        np.add.at(res["grad_v"], s, w[:, None, :, None] * god)
        np.add.at(bnd["grad_v"], s, dw[:, None, :, None] * np.abs(god))
        np.add.at(terms_v, s, np.abs(w)[:, None, :, None] * np.abs(god))
        res["grad_lam"] -= t[:, 1]
        bnd["grad_lam"] += dt[:, 1] + U32 * np.abs(t[:, 1])
    if grad_out is not None:
        deg = np.bincount(at, minlength=n_src).astype(np.float64)
        bnd["grad_k"] += (deg + 2)[:, None, None, None] * U32 * terms_k
        bnd["grad_v"] += (deg + 2)[:, None, None, None] * U32 * terms_v
        bnd["grad_lam"] += U32 * np.abs(res["grad_lam"])
        for r in (res, bnd):
            r["grad_v"] = r["grad_v"].reshape(n_src, K, C)
            r["grad_bias"] = r["grad_bias"].reshape(E, 2 * H)
    return res, bnd


def attention_forward(row_ptr, src, q, k, v, lam, scale, bias=None, mask=None, factors=None):
    """out [n_dst, K, C]; factors [E, H] are the dropout factors of the weights."""
    return _attention(row_ptr, src, q, k, v, lam, scale, bias, mask, factors, None)[0]["out"]


def attention_bounds(row_ptr, src, q, k, v, lam, scale, bias=None, mask=None, factors=None, grad_out=None):
    """(outputs, roundoff bounds) by name: out and, with grad_out, grad_q, grad_k, grad_v, grad_lam, grad_bias."""
    return _attention(row_ptr, src, q, k, v, lam, scale, bias, mask, factors, grad_out)
