"""fp64 definitions (numpy) of the operators around the output layer: layer
norm, dropout from the counter-based generator, log probabilities of given
labels, 8-bit rows and their product.  TEST INFRASTRUCTURE ONLY, like the
rest of the oracle; it shares no code with the library."""
from __future__ import annotations

import math

import numpy as np


# ------------------------------------------------------------------ dropout
def philox4x32(ctr, key, rounds: int = 10):
    """Philox4x32 (Salmon et al., "Parallel random numbers: as easy as 1, 2,
    3", 2011): ctr four and key two arrays of 32-bit words; returns four."""
    lo = np.uint64(0xFFFFFFFF)
    c = [np.asarray(x, dtype=np.uint64) & lo for x in ctr]
    k = [int(x) & 0xFFFFFFFF for x in key]
    for _ in range(rounds):
        a = c[0] * np.uint64(0xD2511F53)
        b = c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & lo,
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & lo]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def drop_mask(B, D, p, seed, offset):
    """(keep, scale): B x D truth values, and 2^16 / (2^16 - T)."""
    T = int(math.floor(float(np.float32(p)) * 65536.0 + 0.5))
    nv = -(-D // 8)
    col, row = np.meshgrid(np.arange(nv), np.arange(B))
    w = philox4x32((col, row, np.full_like(col, offset & 0xFFFFFFFF), np.full_like(col, offset >> 32)),
                   (seed & 0xFFFFFFFF, seed >> 32))
    half = np.stack([x for v in w for x in (v & np.uint64(0xFFFF), v >> np.uint64(16))], axis=2)
    keep = half.reshape(B, nv * 8)[:, :D].astype(np.int64) >= T
    return keep, (65536.0 / (65536 - T) if T < 65536 else 0.0)


# --------------------------------------------------------------- layer norm
def norm_fwd(x, gamma, beta, eps, keep=None, scale=1.0):
    """x: B x D; gamma, beta: D or None.  Returns y, mean, rstd."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + eps)
    y = d * rstd[:, None]
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    if keep is not None:
        y = np.where(keep, y * scale, 0.0)
    return y, mean, rstd


def norm_bwd(x, gamma, mean, rstd, dy, keep=None, scale=1.0):
    """Returns dx, dgamma, dbeta."""
    a = np.where(keep, dy * scale, 0.0) if keep is not None else np.asarray(dy, dtype=np.float64)
    h = (x - mean[:, None]) * rstd[:, None]
    g = a if gamma is None else a * gamma
    dx = rstd[:, None] * (g - g.mean(1)[:, None] - h * (g * h).mean(1)[:, None])
    return dx, (a * h).sum(0), a.sum(0)


# -------------------------------------------------------- log probabilities
def logprob_rows(z):
    """Row statistics of B x N logits: lse, entropy and the B x N log
    probabilities (-inf where the logit is).  Rows with no logit above -inf:
    lse = -inf, entropy 0."""
    z = np.asarray(z, dtype=np.float64)
    lse = np.full(z.shape[0], -np.inf)
    ent = np.zeros(z.shape[0])
    lp = np.full(z.shape, -np.inf)
    for b, r in enumerate(z):
        if np.isnan(r).any() or np.isposinf(r).any():
            lse[b] = ent[b] = np.nan
            lp[b] = np.nan
            continue
        f = r > -np.inf
        if not f.any():
            continue
        m = r[f].max()
        lse[b] = m + math.log(math.fsum(np.exp(r[f] - m)))
        lp[b, f] = r[f] - lse[b]
        p = np.exp(lp[b])
        ent[b] = -math.fsum(p[p > 0] * lp[b, p > 0])
    return lse, ent, lp


def logprob_given(lp, row_ptr, labels, offset=0):
    """Log probability of every entry (label outside the range: -inf)."""
    out = np.full(len(labels), -np.inf)
    for b in range(lp.shape[0]):
        for e in range(row_ptr[b], row_ptr[b + 1]):
            j = int(labels[e]) - offset
            if 0 <= j < lp.shape[1]:
                out[e] = lp[b, j]
    return out


def logprob_top(z, lp, K, offset=0):
    """Top-K of every row by (logit descending, label ascending) over logits
    above -inf (NaN not listed), padded with (-inf, -1)."""
    B, N = z.shape
    val = np.full((B, K), -np.inf)
    idx = np.full((B, K), -1, dtype=np.int64)
    for b in range(B):
        j = np.flatnonzero(z[b] > -np.inf)
        j = j[np.lexsort((j, -z[b, j]))][:K]
        val[b, :len(j)] = lp[b, j]
        idx[b, :len(j)] = j + offset
    return val, idx


def logprob_bwd(z, lse, ent, row_ptr, labels, dlogp, dent=None, offset=0):
    """Gradient of sum_e dlogp[e] logp[e] + sum_b dent[b] entropy[b]."""
    B, N = z.shape
    dz = np.zeros((B, N))
    for b in range(B):
        if np.isneginf(lse[b]):
            continue
        hot = np.zeros(N)
        G = 0.0
        for e in range(row_ptr[b], row_ptr[b + 1]):
            j = int(labels[e]) - offset
            if 0 <= j < N:
                hot[j] += dlogp[e]
                G += dlogp[e]
        lp = z[b] - lse[b]
        p = np.exp(lp)
        n = 0.0 if dent is None else dent[b]
        plp = np.where(p > 0, p * np.where(np.isneginf(lp), 0.0, lp), 0.0)
        dz[b] = hot - p * G - n * (plp + (0.0 if n == 0.0 else p * ent[b]))
    return dz


# ------------------------------------------------------------- 8-bit rows
def quantize_rows(x):
    """fp32 definition: scale = max|x| * fl(1/127), q = x / scale to nearest even."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(invalid="ignore"):
        s = (np.abs(x).max(1) * (np.float32(1) / np.float32(127))).astype(np.float32)
    ok = (s > 0)[:, None]
    t = np.divide(x, s[:, None], out=np.zeros_like(x), where=ok)
    return np.clip(np.rint(t), -127, 127).astype(np.int8), s


def head_i8(q, s, wq, ws):
    """Exact integer sums, scaled in fp64."""
    return (q.astype(np.int64) @ wq.astype(np.int64).T).astype(np.float64) * s[:, None].astype(np.float64) * \
        ws[None, :].astype(np.float64)
