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
