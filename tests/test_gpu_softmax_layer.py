"""The operators together, as examples/softmax_layer.py uses them: one
training step against the fp64 composition, a falling loss, and serving."""
import numpy as np
import pytest
import torch

import workloads as wl
from examples.softmax_layer import SoftmaxLayer
from oracle import ops
from tests._gpu import to_f64

pytestmark = pytest.mark.gpu


def _inputs(**kw):
    return wl.make_inputs(wl.tiny("softmax", **{**dict(B=64, D=128, H=256, L=2000, G=16, F=64, w_std=0.05), **kw}))


def _dense_tail(inp, W):
    """The tail's weights as an L x D matrix."""
    c = inp.cfg
    M = np.zeros((c.n_groups * c.G, c.D))
    for g in range(c.n_groups):
        M[g * c.G:(g + 1) * c.G, inp.idx[g]] = W[g * c.G:(g + 1) * c.G]
    return M[:c.L]


def test_step_matches_the_composition():
    """Loss, dX's norm gradient and the weight gradients of one step.  X, the
    logits and dZ are bf16 between the calls, so they are taken from the
    device; every other quantity follows from them in fp64, within the bf16
    roundings of the results (2^-8) and of dZ's products (2^-8 of the sum of
    their sizes)."""
    inp = _inputs()
    c = inp.cfg
    m = SoftmaxLayer(inp, p=0.2)
    Wh, W = to_f64(m.Wh), _dense_tail(inp, to_f64(m.W))
    gamma, E = to_f64(m.gamma), to_f64(m.E)
    m.step(0.0)
    keep, scale = ops.drop_mask(c.B, c.D, 0.2, 1, 0)
    y, mean, rstd = ops.norm_fwd(E, gamma, to_f64(m.beta), 1e-5, keep, scale)
    X = to_f64(m.X)
    assert np.all(np.abs(X - y) <= 2.0 ** -8 * np.abs(y) + 1e-6)
    z = X @ np.concatenate([Wh, W]).T
    got = np.concatenate([to_f64(m.Zh), to_f64(m.Z)], axis=1)
    assert np.all(np.abs(got - z) <= 2.0 ** -8 * np.abs(z) + 1e-3 * (np.abs(X) @ np.abs(np.concatenate([Wh, W])).T))
    lse, ent, lp = ops.logprob_rows(got)
    logp = ops.logprob_given(lp, inp.row_ptr, inp.labels)
    want = -logp.mean()
    assert abs(m.loss.item() - want) <= 1e-4 * abs(want)
    dz = ops.logprob_bwd(got, lse, ent, inp.row_ptr, inp.labels, np.full(len(logp), -1.0 / len(logp)),
                         np.full(c.B, -0.01 / c.B))
    dzd = np.concatenate([to_f64(m.dZh), to_f64(m.dZ)], axis=1)
    assert np.all(np.abs(dzd - dz) <= 2.0 ** -8 * np.abs(dz) + 1e-4 * np.abs(dz).max())
    dX = dzd @ np.concatenate([Wh, W])
    size = np.abs(dzd) @ np.abs(np.concatenate([Wh, W]))
    assert np.all(np.abs(to_f64(m.dX) - dX) <= 1e-2 * size + 1e-6)
    dWh = dzd[:, :c.H].T @ X
    assert np.all(np.abs(to_f64(m.dWh) - dWh) <= 1e-2 * (np.abs(dzd[:, :c.H]).T @ np.abs(X)) + 1e-6)
    dE, dg, db = ops.norm_bwd(E, gamma, mean, rstd, to_f64(m.dX), keep, scale)
    assert np.all(np.abs(to_f64(m.dE) - dE) <= 2.0 ** -8 * np.abs(dE) + 1e-4 * np.abs(dE).max())
    assert np.allclose(to_f64(m.dgamma), dg, atol=1e-4 * np.abs(dg).max())
    assert np.allclose(to_f64(m.dbeta), db, atol=1e-4 * np.abs(db).max())


def test_training_lowers_the_loss_and_serving_finds_labels():
    inp = _inputs(B=48, pos_per_row=1, zipf_s=0.3)
    m = SoftmaxLayer(inp, p=0.1)
    losses = []
    for _ in range(30):
        m.step(4.0)
        losses.append(m.loss.item())
    print("loss", losses[0], "->", losses[-1], flush=True)
    assert losses[-1] < 0.5 * losses[0]
    val, idx = m.serve(5)
    torch.cuda.synchronize()
    v = to_f64(val)
    assert np.all(v[:, :-1] >= v[:, 1:]) and np.all(np.exp(v).sum(1) <= 1 + 1e-5)
    # the 8-bit head's alternatives against the bf16 head's
    m.logits()
    g = m.given(topk=5)
    from sparse_output_layer_amd import haste as H
    H.haste_logprob_fwd(m.Zh, m.Z, g, m.lse, m.logp)
    same = (g.topk_idx[:, 0] == idx[:, 0]).float().mean().item()
    assert same >= 0.9
