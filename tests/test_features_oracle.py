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


def test_norms_around_a_block():
    r = np.random.default_rng(2)
    B, D = 5, 13
    keep = r.random((B, D)) > 0.3
    o, x, dy, dro = (r.standard_normal((B, D)) for _ in range(4))
    for gate in (None, r.standard_normal(D), r.standard_normal((B, D))):
        for post in (None, (r.standard_normal(D), r.standard_normal(D))):
            for norm in (None, (r.standard_normal(D), r.standard_normal(D))):
                kw = dict(gate=gate, alpha=0.3, post=post, norm=norm, keep=keep, scale=1 / 0.7)
                t = [t64(v, True) for v in (o, x, np.ones(D) if gate is None else gate, *(post or (np.ones(D), np.zeros(D))),
                                            *(norm or (np.ones(D), np.zeros(D))))]
                ln = torch.nn.functional.layer_norm
                p = ln(t[0], (D,), t[3], t[4], 1e-5) if post else t[0]
                out = t[1] + 0.3 * t[2] * torch.where(torch.tensor(keep), p / 0.7, 0.0)
                y = ln(out, (D,), t[5], t[6], 1e-5) if norm else None
                got, gy, st = ft.addnorm_fwd(o, x, eps=1e-5, **kw)
                assert np.allclose(got, out.detach().numpy())
                loss = (out * t64(dro)).sum()
                if norm:
                    assert np.allclose(gy, y.detach().numpy())
                    loss = loss + (y * t64(dy)).sum()
                loss.backward()
                g = ft.addnorm_bwd(o, got, st, dy if norm else None, dro, **kw)
                assert np.allclose(g["do"], t[0].grad.numpy()) and np.allclose(g["dr"], t[1].grad.numpy())
                if gate is not None:
                    assert np.allclose(g["gate"] if gate.ndim == 2 else g["gate"].sum(0), t[2].grad.numpy())
                for k, i in (("g1", 3), ("b1", 4), ("g2", 5), ("b2", 6)):
                    if k in g:
                        assert np.allclose(g[k].sum(0), t[i].grad.numpy())


def test_projections():
    r = np.random.default_rng(3)
    M, K, N = 6, 5, 7
    F = torch.nn.functional
    fn = {"none": lambda z: z, "relu": torch.relu, "gelu": lambda z: F.gelu(z, approximate="tanh"), "silu": F.silu}
    for name in ft.ACTS:
        x, W, b, res = (t64(r.standard_normal(s), True) for s in ((M, K), (N, K), (N,), (M, N)))
        dy, add = r.standard_normal((M, N)), r.standard_normal((M, K))
        z = x @ W.T + b
        y = fn[name](z) + res
        gy, gz = ft.linear_fwd(x.detach().numpy(), W.detach().numpy(), b.detach().numpy(), name, res.detach().numpy())
        assert np.allclose(gy, y.detach().numpy()) and np.allclose(gz, z.detach().numpy())
        ((y * t64(dy)).sum() + (x * t64(add)).sum()).backward()
        dx, dW, db, _ = ft.linear_bwd(x.detach().numpy(), W.detach().numpy(), dy, gz, name, add)
        assert np.allclose(dx, x.grad.numpy()) and np.allclose(dW, W.grad.numpy()) and np.allclose(db, b.grad.numpy())
