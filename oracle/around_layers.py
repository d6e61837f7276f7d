"""Plain fp64 NumPy oracles of the operators around the layers: the embedding lookup and its gradient, the norms before
and after a block with its gate and residual scale, and activation checkpoints in 8 bits (test infrastructure).

Written from the definitions, a row or a group at a time where that is the plainest form; shares no code with the GPU path.
"""
from __future__ import annotations

import numpy as np

F8 = np.float64


# ----------------------------------------------------------------------------
# Embedding
# ----------------------------------------------------------------------------

def embedding_fwd(table, ids, scale, width=None):
    V, dim = table.shape
    out = np.zeros((len(ids), width or dim), F8)
    for t, v in enumerate(ids):
        if 0 <= v < V:
            out[t, :dim] = F8(scale) * table[v].astype(F8)
    return out


def embedding_bwd(dout, ids, V, dim, scale):
    """(gradient [V][dim], sum of |terms| [V][dim], events per item [V])"""
    g, a, n = np.zeros((V, dim), F8), np.zeros((V, dim), F8), np.zeros(V, np.int64)
    for t, v in enumerate(ids):
        if 0 <= v < V:
            row = F8(scale) * dout[t, :dim].astype(F8)
            g[v] += row
            a[v] += np.abs(row)
            n[v] += 1
    return g, a, n


# ----------------------------------------------------------------------------
# Norms before and after a block
# ----------------------------------------------------------------------------

def stats(kind, a, eps):
    """Mean and 1/spread of each row [T][1]; (0, 1) without a norm."""
    a = a.astype(F8)
    T = a.shape[0]
    if kind is None:
        return np.zeros((T, 1)), np.ones((T, 1))
    m = a.mean(1, keepdims=True) if kind == "layer" else np.zeros((T, 1))
    return m, 1.0 / np.sqrt(((a - m) ** 2).mean(1, keepdims=True) + eps)


def act(kind, u):
    """act(u), act'(u)."""
    u = u.astype(F8)
    s = 1.0 / (1.0 + np.exp(-u))
    if kind == "silu":
        return u * s, s * (1.0 + u * (1.0 - s))
    if kind == "sigmoid":
        return s, s * (1.0 - s)
    return u, np.ones_like(u)


def _or(p, other):
    return F8(other) if p is None else p.astype(F8)


def _normed(kind, a, m, r, gamma, beta):
    n = (a.astype(F8) - m) * r
    return n, (n * _or(gamma, 1) + _or(beta, 0) if kind is not None else a.astype(F8))


def block_y(cfg, p, x, b, gate, eps):
    """y and the statistics after the block; cfg: post, pre, gate; p: parameters by name (None: absent)."""
    m, r = stats(cfg["post"], b, eps)
    _, v = _normed(cfg["post"], b, m, r, p.get("post_gamma"), p.get("post_beta"))
    if gate is not None:
        v = v * act(cfg["gate"], gate)[0]
    return x.astype(F8) + _or(p.get("res_scale"), 1) * v, m, r


def block_h(cfg, p, y, eps):
    m, r = stats(cfg["pre"], y, eps)
    return _normed(cfg["pre"], y, m, r, p.get("pre_gamma"), p.get("pre_beta"))[1], m, r


def _norm_bwd(kind, n, r, q):
    if kind is None:
        return q
    level = q.mean(1, keepdims=True) if kind == "layer" else 0.0
    return r * (q - level - n * (q * n).mean(1, keepdims=True))


def block_bwd(cfg, p, y, b, gate, st, dy, dh):
    """Gradients (dx, db, dgate, parameters) from the forward's statistics st [T][4]."""
    m1, r1, m2, r2 = (st[:, i:i + 1].astype(F8) for i in range(4))
    out = {}
    e = np.zeros(st.shape[:1] + ((y if y is not None else b).shape[1],), F8) if dy is None else dy.astype(F8)
    if dh is not None:
        n2 = (y.astype(F8) - m2) * r2
        up = dh.astype(F8)
        if cfg["pre"] is not None:
            out["pre_gamma"], out["pre_beta"] = (up * n2).sum(0), up.sum(0)
            up = up * _or(p.get("pre_gamma"), 1)
        e = e + _norm_bwd(cfg["pre"], n2, r2, up)
    out["dx"] = e
    if b is None:
        return out
    n1, v = _normed(cfg["post"], b, m1, r1, p.get("post_gamma"), p.get("post_beta"))
    a, da = act(cfg["gate"], gate) if gate is not None else (1.0, 0.0)
    out["res_scale"] = (e * v * a).sum(0)
    dv = e * _or(p.get("res_scale"), 1)
    if gate is not None:
        out["dgate"] = dv * v * da
    dp = dv * a
    if cfg["post"] is not None:
        out["post_gamma"], out["post_beta"] = (dp * n1).sum(0), dp.sum(0)
        dp = dp * _or(p.get("post_gamma"), 1)
    out["db"] = _norm_bwd(cfg["post"], n1, r1, dp)
    return out


# ----------------------------------------------------------------------------
# 8-bit checkpoints
# ----------------------------------------------------------------------------

def _e4m3_values():
    """All non-negative finite e4m3 values: code c has exponent c >> 3 and fraction c & 7."""
    return np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


E4M3 = _e4m3_values()


def nearest(fmt, q):
    """q to the nearest whole number or e4m3 value, ties to the even code."""
    if fmt == "int8":
        return np.round(q)                               # NumPy rounds halves to even
    a = np.abs(q)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)       # first value >= a
    lo = np.maximum(hi - 1, 0)
    up, down = E4M3[hi] - a, a - E4M3[lo]
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return np.copysign(E4M3[pick], q)


def hold(fmt, x):
    """x [rows][w] held in 8 bits with a scale for every 32 values: (values in units of the scale, scale exponents k, the
    values they stand for).  k is the smallest with max |x| <= top 2^k, at least -126 and at most the largest with top 2^k in
    fp32's range (larger magnitudes are held as top 2^k); 128 marks a group with a non-finite value."""
    top, last = (127.0, 121) if fmt == "int8" else (448.0, 119)
    x = np.asarray(x, F8)
    rows, w = x.shape
    q, k, back = np.zeros_like(x), np.zeros((rows, w // 32), np.int64), np.zeros_like(x)
    for r in range(rows):
        for g in range(w // 32):
            v = x[r, 32 * g:32 * g + 32]
            at = np.s_[r, 32 * g:32 * g + 32]
            if not np.all(np.isfinite(v)):
                k[r, g], back[at] = 128, np.nan
                continue
            e = -126
            while np.max(np.abs(v)) > top * 2.0 ** e and e < last:
                e += 1
            k[r, g] = e
            q[at] = nearest(fmt, np.clip(v / 2.0 ** e, -top, top))
            back[at] = q[at] * 2.0 ** e
    return q, k, back
