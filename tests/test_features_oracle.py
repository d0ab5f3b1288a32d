"""The oracle of the feature stage against torch's automatic differentiation
in fp64 on the CPU, and against values worked by hand."""
import numpy as np
import torch

from oracle import features as ft


def t64(a, grad=False):
    return torch.tensor(np.asarray(a), dtype=torch.float64, requires_grad=grad)


def test_embedding_by_hand():
    E = np.array([[1.0, 2.0], [3.0, 5.0], [7.0, 11.0]])
    y, size = ft.embed_fwd([2, 0, -1, 1, 3], E, 3, [0, 3, 3, 5], [2.0, -1.0, 9.0, 0.5, 4.0], 10.0)
    assert np.array_equal(y, [[130.0, 200.0], [0.0, 0.0], [15.0, 25.0]])
    assert np.array_equal(size, [[150.0, 240.0], [0.0, 0.0], [15.0, 25.0]])


def test_embedding_gradients():
    r = np.random.default_rng(1)
    B, n, V, D = 7, 60, 9, 5
    tok = r.integers(-1, V + 1, n)
    rp = np.concatenate([[0], np.sort(r.integers(0, n + 1, B - 1)), [n]])
    E, w, dy = t64(r.standard_normal((V, D)), True), t64(r.standard_normal(n), True), r.standard_normal((B, D))
    row, live = ft.entries(n, B, V, tok, rp)
    k = np.flatnonzero(live)
    y = torch.zeros(B, D, dtype=torch.float64).index_add(0, torch.tensor(row[k]), 0.3 * w[k, None] * E[tok[k]])
    assert np.allclose(ft.embed_fwd(tok, E.detach().numpy(), B, rp, w.detach().numpy(), 0.3)[0], y.detach().numpy())
    (y * t64(dy)).sum().backward()
    dE, _, dw, _ = ft.embed_bwd(tok, dy, V, E.detach().numpy(), rp, w.detach().numpy(), 0.3)
    assert np.allclose(dE, E.grad.numpy()) and np.allclose(dw, w.grad.numpy())
    z = ft.embed_fwd(tok, E.detach().numpy(), n, None, None, 1.0)[0]
    assert np.array_equal(z[live], E.detach().numpy()[tok[live]]) and (z[~live] == 0).all()
