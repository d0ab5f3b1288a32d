"""The oracle's definitions of the operators around the layer, pinned on the
CPU: the generator's published answers, gradients against central
differences, hand-made rows."""
import math

import numpy as np
import pytest

from oracle import ops


def test_generator_known_answers():
    """Known-answer vectors of Philox4x32-10 published with the paper."""
    ff = 0xFFFFFFFF
    for ctr, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((ff, ff, ff, ff), (ff, ff), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        got = ops.philox4x32([np.array([c]) for c in ctr], key)
        assert tuple(int(w[0]) for w in got) == want


def test_mask_counts_and_steps():
    for p in (0.1, 0.5, 0.9):
        keep, scale = ops.drop_mask(64, 1000, p, 12345, 6)
        T = math.floor(float(np.float32(p)) * 65536 + 0.5)
        q = T / 65536
        n = keep.size
        assert abs((~keep).sum() - n * q) < 5 * math.sqrt(n * q * (1 - q))
        assert scale == 65536 / (65536 - T)
    assert ops.drop_mask(3, 9, 0.0, 1, 0)[0].all()
    assert not ops.drop_mask(3, 9, 1.0, 1, 0)[0].any()
    a = ops.drop_mask(5, 40, 0.5, 1, 0)[0]
    assert np.array_equal(a[:, :17], ops.drop_mask(5, 17, 0.5, 1, 0)[0])    # by element, not by shape
    assert not np.array_equal(a, ops.drop_mask(5, 40, 0.5, 1, 1)[0])
    assert not np.array_equal(a, ops.drop_mask(5, 40, 0.5, 1 << 32, 0)[0])


def _central(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        d = np.zeros_like(x)
        d[i] = h
        g[i] = (f(x + d) - f(x - d)) / (2 * h)
    return g


@pytest.mark.parametrize("p", [0.0, 0.4])
def test_norm_gradient_by_differences(p):
    r = np.random.default_rng(3)
    B, D, eps = 3, 7, 1e-3
    x, dy = r.standard_normal((B, D)), r.standard_normal((B, D))
    ga, be = r.standard_normal(D), r.standard_normal(D)
    keep, sc = ops.drop_mask(B, D, p, 9, 2) if p else (None, 1.0)
    _, m, rs = ops.norm_fwd(x, ga, be, eps, keep, sc)
    dx, dg, db = ops.norm_bwd(x, ga, m, rs, dy, keep, sc)
    loss = lambda x_, g_, b_: float((ops.norm_fwd(x_, g_, b_, eps, keep, sc)[0] * dy).sum())  # noqa: E731
    assert np.allclose(dx, _central(lambda t: loss(t, ga, be), x), atol=1e-7)
    assert np.allclose(dg, _central(lambda t: loss(x, t, be), ga), atol=1e-7)
    assert np.allclose(db, _central(lambda t: loss(x, ga, t), be), atol=1e-7)


def test_logprob_gradient_by_differences():
    r = np.random.default_rng(4)
    B, N = 3, 9
    z = r.standard_normal((B, N)) * 2
    z[1, 3] = -np.inf
    rp = np.array([0, 3, 4, 4])
    lab = np.array([11, 15, 11, 99])      # a repeated label, one out of range
    dl, de = r.standard_normal(4), r.standard_normal(B)

    def f(t):
        _, ent, lp = ops.logprob_rows(t)
        lpg = ops.logprob_given(lp, rp, lab, 10)
        return float(dl[:3] @ lpg[:3] + de @ ent)
    lse, ent, _ = ops.logprob_rows(z)
    got = ops.logprob_bwd(z, lse, ent, rp, lab, dl, de, 10)
    want = np.zeros_like(z)
    for i in np.ndindex(B, N):
        if np.isinf(z[i]):
            continue
        d = np.zeros_like(z)
        d[i] = 1e-6
        want[i] = (f(z + d) - f(z - d)) / 2e-6
    assert np.allclose(got, want, atol=1e-7)


def test_logprob_rows_by_hand():
    inf = np.inf
    z = np.array([[0.0, 0.0, -inf, 0.0], [-inf] * 4, [math.log(3), 0.0, -inf, -inf], [1, np.nan, 0, 0], [inf, 0, 0, 0]])
    lse, ent, lp = ops.logprob_rows(z)
    assert np.isclose(lse[0], math.log(3)) and np.isclose(ent[0], math.log(3))
    assert lse[1] == -inf and ent[1] == 0 and np.all(lp[1] == -inf)
    assert np.isclose(lse[2], math.log(4)) and np.isclose(lp[2, 1], math.log(0.25))
    assert np.isnan(lse[3:]).all() and np.isnan(ent[3:]).all()
    v, i = ops.logprob_top(z, lp, 3, 100)
    assert i.tolist() == [[100, 101, 103], [-1, -1, -1], [100, 101, -1], [100, 102, 103], [100, 101, 102]]
    assert v[1].tolist() == [-inf] * 3


def test_quantize_by_hand():
    q, s = ops.quantize_rows(np.array([[127.0, -254.0, 0.0, 1.0, 3.0], [0, 0, 0, 0, 0]]))
    assert s.tolist() == [2.0, 0.0]
    assert q.tolist() == [[64, -127, 0, 0, 2], [0, 0, 0, 0, 0]]     # 63.5 -> 64, 0.5 -> 0, 1.5 -> 2
    assert np.array_equal(ops.head_i8(q[:1], s[:1], q[:1], s[:1]), [[4.0 * (64 * 64 + 127 * 127 + 4)]])
