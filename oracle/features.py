"""fp64 definitions (numpy) of the feature stage in front of the output layer:
embedding bags, feature projections and the norms around a block.  TEST
INFRASTRUCTURE ONLY, like the rest of the oracle; it shares no code with the
library."""
from __future__ import annotations

import numpy as np


# ---------------------------------------------------------------- embedding
def entries(n, B, V, tokens, row_ptr=None):
    """Row of every entry, and which entries' tokens are in the table."""
    row = np.arange(n) if row_ptr is None else np.repeat(np.arange(B), np.diff(row_ptr))
    tokens = np.asarray(tokens, dtype=np.int64)
    return row, (tokens >= 0) & (tokens < V)


def embed_fwd(tokens, E, B, row_ptr=None, weights=None, scale=1.0):
    """y, and the sum of the sizes of its terms."""
    E = np.asarray(E, dtype=np.float64)
    y, size = np.zeros((B, E.shape[1])), np.zeros((B, E.shape[1]))
    row, live = entries(len(tokens), B, len(E), tokens, row_ptr)
    for e in np.flatnonzero(live):
        t = scale * (1.0 if weights is None else weights[e]) * E[tokens[e]]
        y[row[e]] += t
        size[row[e]] += np.abs(t)
    return y, size


def embed_bwd(tokens, dy, V, E=None, row_ptr=None, weights=None, scale=1.0):
    """dE, the sizes of its sums; dweights and theirs (None without E)."""
    dy = np.asarray(dy, dtype=np.float64)
    B, D = dy.shape
    dE, size = np.zeros((V, D)), np.zeros((V, D))
    row, live = entries(len(tokens), B, V, tokens, row_ptr)
    dw, dsize = (None, None) if E is None else (np.zeros(len(tokens)), np.zeros(len(tokens)))
    for e in np.flatnonzero(live):
        t = scale * (1.0 if weights is None else weights[e]) * dy[row[e]]
        dE[tokens[e]] += t
        size[tokens[e]] += np.abs(t)
        if E is not None:
            p = scale * np.asarray(E[tokens[e]], dtype=np.float64) * dy[row[e]]
            dw[e], dsize[e] = p.sum(), np.abs(p).sum()
    return dE, size, dw, dsize


# -------------------------------------------------------------- projections
ACTS = ("none", "relu", "gelu", "silu")


def act(name, z):
    """The activation and its derivative."""
    if name == "none":
        return z, np.ones_like(z)
    if name == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    c = 2.0 * np.sqrt(2.0 / np.pi)
    t, dt = (z, 1.0) if name == "silu" else (c * (z + 0.044715 * z ** 3), c * (1.0 + 3 * 0.044715 * z ** 2))
    s = 0.5 * (1.0 + np.tanh(0.5 * t))
    return z * s, s + z * s * (1.0 - s) * dt


def linear_fwd(x, W, bias=None, name="none", residual=None):
    """y, z."""
    z = np.asarray(x, np.float64) @ np.asarray(W, np.float64).T
    if bias is not None:
        z = z + bias
    y = act(name, z)[0]
    return (y if residual is None else y + residual), z


def linear_bwd(x, W, dy, z, name="none", add=None):
    """dx, dW, dbias, dz."""
    dz = np.asarray(dy, np.float64) * act(name, np.asarray(z, np.float64))[1]
    dx = dz @ W
    return (dx if add is None else dx + add), dz.T @ x, dz.sum(0), dz


# ------------------------------------------------- the norms around a block
def _norm(x, eps):
    m = x.mean(1)
    return m, 1.0 / np.sqrt(((x - m[:, None]) ** 2).mean(1) + eps)


def addnorm_fwd(o, r, gate=None, alpha=1.0, post=None, norm=None, eps=1e-5, keep=None, scale=1.0):
    """post, norm: (gamma, beta) or None.  Returns r_out, y (or None), stats
    (rows of a norm that is not there: 0, 1)."""
    o, r = np.asarray(o, np.float64), np.asarray(r, np.float64)
    B = len(o)
    stats = np.stack([np.zeros(B), np.ones(B)] * 2)
    p = o
    if post is not None:
        stats[0], stats[1] = _norm(o, eps)
        p = (o - stats[0][:, None]) * stats[1][:, None] * post[0] + post[1]
    if keep is not None:
        p = np.where(keep, p * scale, 0.0)
    out = r + alpha * (1.0 if gate is None else gate) * p
    if norm is None:
        return out, None, stats
    stats[2], stats[3] = _norm(out, eps)
    return out, (out - stats[2][:, None]) * stats[3][:, None] * norm[0] + norm[1], stats


def addnorm_bwd(o, r_out, stats, dy=None, dr_out=None, gate=None, alpha=1.0, post=None, norm=None, keep=None, scale=1.0):
    """Returns a dict: dr, do, and gate, g1, b1, g2, b2 per element (B x D,
    before the sums over the rows)."""
    o = np.asarray(o, np.float64)
    m1, s1, m2, s2 = (t[:, None] for t in stats)
    out = {}
    dR = np.zeros_like(o) if dr_out is None else np.asarray(dr_out, np.float64)
    if dy is not None:
        h = (r_out - m2) * s2
        u = dy * norm[0]
        dR = dR + s2 * (u - u.mean(1, keepdims=True) - h * (u * h).mean(1, keepdims=True))
        out["g2"], out["b2"] = dy * h, dy
    k = 1.0 if keep is None else np.where(keep, scale, 0.0)
    a = k * alpha * (1.0 if gate is None else gate) * dR
    p = o
    do = a
    if post is not None:
        h = (o - m1) * s1
        p = h * post[0] + post[1]
        v = a * post[0]
        do = s1 * (v - v.mean(1, keepdims=True) - h * (v * h).mean(1, keepdims=True))
        out["g1"], out["b1"] = a * h, a
    out.update(dr=dR, do=do, gate=alpha * dR * k * p)
    return out
