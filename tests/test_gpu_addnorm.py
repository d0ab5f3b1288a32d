"""GPU parity of the norms around a block (forward, backward) against the
fp64 oracle, through the C ABI.

Bounds are worst-case rounding bounds of the fp32 formulas, u = 2^-24 a
rounding: a layer norm of x known within e, n elements a row, has its mean
within mean(e) + (n + 2) u mean|x|, and so on as written below; every result
is rounded once more to its type."""
import numpy as np
import pytest
import torch

from oracle import features as ft
from oracle import ops
from tests._gpu import DEV, to_f64
from tests.test_gpu_ops import TINY, TT, gen, rand, rounded, u, within

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module")
def H():
    from sparse_output_layer_amd import haste
    haste.lib()
    return haste


CASES = [  # B, D, o, r, y, weights, post, norm, gate, affine, p
    (1, 1, "f32", "f32", "f32", "f32", 0, 1, "none", 1, 0.0), (1, 1024, "bf16", "bf16", "bf16", "f32", 1, 1, "vector", 1, 0.0),
    (5, 3, "bf16", "f32", "f32", "bf16", 1, 1, "rows", 1, 0.3), (33, 768, "bf16", "bf16", "bf16", "f32", 1, 1, "vector", 1, 0.1),
    (33, 768, "bf16", "f32", "f32", "bf16", 1, 0, "rows", 1, 0.1), (17, 1001, "f32", "f32", "f32", "f32", 0, 1, "none", 0, 0.0),
    (17, 1001, "bf16", "f32", "bf16", "f32", 1, 1, "vector", 1, 0.5), (9, 4097, "f32", "bf16", "f32", "f32", 0, 1, "rows", 1, 0.1),
    (300, 64, "bf16", "bf16", "bf16", "f32", 1, 1, "none", 0, 0.0), (3, 8192, "bf16", "f32", "bf16", "bf16", 1, 1, "vector", 1, 0.1),
    (2, 20011, "f32", "f32", "f32", "f32", 1, 1, "rows", 1, 0.1), (700, 1024, "f32", "bf16", "bf16", "f32", 0, 0, "vector", 1, 0.2),
    (1500, 96, "bf16", "f32", "f32", "f32", 1, 1, "vector", 0, 0.0), (4, 30001, "bf16", "bf16", "f32", "f32", 0, 1, "vector", 1, 0.0),
    (2051, 520, "bf16", "f32", "f32", "f32", 1, 1, "vector", 1, 0.1), (64, 2048, "f32", "f32", "bf16", "bf16", 1, 1, "rows", 1, 0.0),
    (520, 200, "f32", "bf16", "f32", "f32", 1, 1, "rows", 1, 1.0), (6, 12000, "bf16", "f32", "bf16", "f32", 1, 0, "none", 1, 0.1),
    (7, 16384, "f32", "bf16", "bf16", "f32", 0, 0, "rows", 1, 0.1), (600, 9000, "bf16", "bf16", "bf16", "f32", 1, 1, "vector", 1, 0.0)]


def norm_bounds(X, e):
    """Of a layer norm of X known within e: bounds of mean, rstd (relative) and
    of the normed elements."""
    D = X.shape[1]
    m = X.mean(1, keepdims=True)
    dm = e.mean(1, keepdims=True) + (D + 2) * u * np.abs(X).mean(1, keepdims=True)
    d = np.abs(X - m)
    ed = e + dm + u * d
    var = (d * d).mean(1, keepdims=True)
    dvar = (2 * d * ed + ed * ed).mean(1, keepdims=True) + (D + 8) * u * var
    rel = dvar / (var + EPS) + 4 * u
    rstd = 1 / np.sqrt(var + EPS)
    return dm[:, 0], rel[:, 0], d * rstd * (rel + 3 * u) + rstd * ed


class Case:
    def __init__(self, H, case, shift=3.0):
        print(f"addnorm {case}", flush=True)
        (self.B, self.D, self.ot, self.rt, self.yt, wt, post, norm, gate, affine, p) = case
        B, D = self.B, self.D
        g = gen(B * 7 + D)
        self.g = g
        self.o, self.r = rand(g, (B, D), self.ot, 1.5, shift), rand(g, (B, D), self.rt, 2.0, -shift)
        self.alpha = 0.7
        self.gate = None if gate == "none" else rand(g, (D,), wt, 0.5, 0.3) if gate == "vector" else rand(g, (B, D), self.ot, 0.5, 0.3)

        def weights():
            return H.NormWeights(rand(g, (D,), wt, 0.3, 1.0), rand(g, (D,), wt, 0.3)) if affine else H.NormWeights()
        self.post = weights() if post else None
        self.norm = weights() if norm else None
        self.drop = H.Dropout(p, 987654321987, 3) if p else None
        self.keep, self.scale = ops.drop_mask(B, D, p, 987654321987, 3) if p else (None, 1.0)
        self.kw = dict(gate=self.gate, alpha=self.alpha, post=self.post, norm=self.norm, dropout=self.drop)
        n64 = lambda w: None if w is None else (np.ones(D), np.zeros(D)) if w.gamma is None else (to_f64(w.gamma), to_f64(w.beta))  # noqa: E731
        self.o64 = to_f64(self.o)
        self.G = 1.0 if self.gate is None else to_f64(self.gate)
        self.kw64 = dict(gate=None if self.gate is None else self.G, alpha=float(np.float32(self.alpha)), post=n64(self.post),
                         norm=n64(self.norm), keep=self.keep, scale=self.scale)
        self.k = np.ones((B, D)) if self.keep is None else np.where(self.keep, self.scale, 0.0)


@pytest.mark.parametrize("case", CASES)
def test_addnorm_fwd(H, case):
    c = Case(H, case)
    B, D = c.B, c.D
    stats = torch.full((4, B), 7.0, device=DEV)
    y = torch.full((B, D), 9.0, dtype=TT[c.yt], device=DEV) if c.norm else None
    r_out, _ = H.haste_addnorm_fwd(c.o, c.r, None, y, stats=stats, eps=EPS, **c.kw)
    want, wy, ws = ft.addnorm_fwd(c.o64, to_f64(c.r), eps=EPS, **c.kw64)
    p, ep = np.abs(c.o64), np.zeros((B, D))
    st = to_f64(stats)
    if c.post:
        dm, rel, dh = norm_bounds(c.o64, np.zeros((B, D)))
        within("mean of o", st[0], ws[0], dm + u * np.abs(ws[0]))
        within("rstd of o", st[1], ws[1], rel * ws[1])
        ga, be = (np.abs(t) for t in c.kw64["post"])
        h = np.abs(c.o64 - ws[0][:, None]) * ws[1][:, None]
        p, ep = ga * h + be, ga * dh
    else:
        assert (st[:2] == 7.0).all()
    size = 0.7 * np.abs(c.G) * c.k
    e = size * (ep + 10 * u * p) + 2 * u * (np.abs(to_f64(c.r)) + size * p)
    within("r_out", to_f64(r_out), want, e + rounded(c.rt, np.abs(want) + e))
    if c.norm:
        dm, rel, dh = norm_bounds(want, e)
        within("mean", st[2], ws[2], dm + u * np.abs(ws[2]))
        within("rstd", st[3], ws[3], rel * ws[3])
        ga, be = (np.abs(t) for t in c.kw64["norm"])
        h = np.abs(want - ws[2][:, None]) * ws[3][:, None]
        b = ga * dh + 4 * u * (ga * h + be)
        within("y", to_f64(y), wy, b + rounded(c.yt, np.abs(wy) + b))
    else:
        assert (st[2:] == 7.0).all()
    # without statistics, and in place: the same bits
    y2 = torch.empty_like(y) if c.norm else None
    r2 = c.r.clone()
    H.haste_addnorm_fwd(c.o, r2, r2, y2, eps=EPS, **c.kw)
    assert torch.equal(r2, r_out) and (y is None or torch.equal(y2, y))


def _bwd(H, c, dr_given=True, check=True):
    B, D = c.B, c.D
    stats = torch.zeros(4, B, device=DEV)
    r_out, _ = H.haste_addnorm_fwd(c.o, c.r, stats=stats, eps=EPS, **c.kw)
    dy = rand(c.g, (B, D), c.yt, 0.7) if c.norm else None
    dro = rand(c.g, (B, D), c.rt, 0.5) if dr_given or not c.norm else None
    grads = dict(dpost=H.NormWeights(*(torch.full((D,), 5.0, device=DEV) for _ in range(2))) if c.post else None,
                 dnorm=H.NormWeights(*(torch.full((D,), 5.0, device=DEV) for _ in range(2))) if c.norm else None,
                 dgate=None if c.gate is None else torch.full((D,), 5.0, device=DEV) if c.gate.dim() == 1 else torch.empty_like(c.gate))
    return r_out, stats, dy, dro, grads


def _vectors(grads):
    out = {}
    if grads["dgate"] is not None and grads["dgate"].dim() == 1:
        out["gate"] = grads["dgate"]
    for k, names in (("dpost", ("g1", "b1")), ("dnorm", ("g2", "b2"))):
        if grads[k] is not None:
            out[names[0]], out[names[1]] = grads[k].gamma, grads[k].beta
    return out


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dr_given", [True, False])
def test_addnorm_bwd(H, case, dr_given):
    c = Case(H, case)
    B, D = c.B, c.D
    r_out, stats, dy, dro, grads = _bwd(H, c, dr_given)
    kw = dict(c.kw, **grads)
    dr, do = H.haste_addnorm_bwd(c.o, r_out, stats, dy, dro, **kw)
    st = to_f64(stats)
    ref = ft.addnorm_bwd(c.o64, to_f64(r_out), st, None if dy is None else to_f64(dy), None if dro is None else to_f64(dro), **c.kw64)

    def back(v, h, s, e):        # bound of a norm's input gradient from v known within e
        m = lambda t: t.mean(1, keepdims=True)  # noqa: E731
        return s * (e + m(e) + h * m(e * h) + 6 * u * v + (D + 9) * u * m(v) + h * (D + 13) * u * m(v * h))
    eR = 2 * u * np.abs(ref["dr"]) + (0 if dro is None else u * np.abs(to_f64(dro)))
    tot = {}
    if c.norm:
        h2 = np.abs(to_f64(r_out) - st[2][:, None]) * st[3][:, None]
        v = np.abs(to_f64(dy) * c.kw64["norm"][0])
        eR = eR + back(v, h2, st[3][:, None], np.zeros((B, D)))
        tot["g2"], tot["b2"] = (B + 8) * u * np.abs(ref["g2"]).sum(0), (B + 4) * u * np.abs(ref["b2"]).sum(0)
    within("dr", to_f64(dr), ref["dr"], eR + rounded(c.rt, np.abs(ref["dr"]) + eR))
    size = 0.7 * np.abs(c.G) * c.k
    a, ea = size * np.abs(ref["dr"]), size * (eR + 4 * u * np.abs(ref["dr"]))
    p, ep, b = np.abs(c.o64), 0, ea
    if c.post:
        h1 = np.abs(c.o64 - st[0][:, None]) * st[1][:, None]
        ga, be = (np.abs(t) for t in c.kw64["post"])
        p, ep = ga * h1 + be, 6 * u * (ga * h1 + be)
        b = back(a * ga, h1, st[1][:, None], ea * ga)
        tot["g1"] = (ea * h1).sum(0) + (B + 8) * u * (a * h1).sum(0)
        tot["b1"] = ea.sum(0) + (B + 4) * u * a.sum(0)
    within("do", to_f64(do), ref["do"], b + rounded(c.ot, np.abs(ref["do"]) + b))
    t = 0.7 * c.k * np.abs(ref["dr"])
    eg = 0.7 * c.k * eR * p + t * ep + 6 * u * t * p
    if c.gate is not None and c.gate.dim() == 2:
        within("dgate", to_f64(grads["dgate"]), ref["gate"], eg + rounded(c.ot, np.abs(ref["gate"]) + eg))
    # a vector's gradient is gamma times sum(t h) plus beta times sum(t): the roundings count by the terms' sizes t p
    tot["gate"] = eg.sum(0) + (B + 8) * u * (t * p).sum(0)
    first = _vectors(grads)
    for k, t in first.items():
        r = ref[k].sum(0)
        within(k, to_f64(t), r, tot[k] + u * np.abs(r) + TINY)
    # added to; in place; without weight gradients: the same bits
    r_, s_, _, _, more = _bwd(H, c, dr_given)
    dro2 = None if dro is None else dro.clone()
    dr2, do2 = H.haste_addnorm_bwd(c.o, r_out, stats, dy, dro2, dr=dro2, accumulate_dw=True, **dict(c.kw, **more))
    assert torch.equal(dr2, dr) and torch.equal(do2, do)
    for k, t in _vectors(more).items():
        assert torch.equal(t, first[k] + 5.0)
    dr3, do3 = H.haste_addnorm_bwd(c.o, r_out, stats, dy, dro, **c.kw)
    assert torch.equal(dr3, dr) and torch.equal(do3, do)


@pytest.mark.parametrize("D", [2, 5, 7, 8, 9, 15, 127, 129, 250, 257, 511, 514, 1023, 1028, 2045, 2049, 4093, 4098, 8190, 8193])
def test_addnorm_row_ends(H, D):
    for ot, rt, gate in (("bf16", "f32", "vector"), ("f32", "bf16", "rows")):
        case = (5, D, ot, rt, ot, "f32", 1, 1, gate, 1, 0.25)
        test_addnorm_fwd(H, case)
        test_addnorm_bwd(H, case, True)


@pytest.mark.parametrize("B", [1, 2, 31, 33, 511, 513, 4100])
@pytest.mark.parametrize("D", [40, 200, 777, 1300])
def test_addnorm_row_counts(H, B, D):
    test_addnorm_bwd(H, (B, D, "bf16", "f32", "f32", "f32", 1, 1, "vector", 1, 0.1), True)


def test_addnorm_nan_and_dropped(H):
    """A NaN or infinity stays in its row; where it is dropped it is not seen."""
    B, D = 8, 200
    keep, _ = ops.drop_mask(B, D, 0.5, 9, 9)
    o, r = rand(gen(1), (B, D), "bf16"), rand(gen(2), (B, D), "f32")
    o[~torch.from_numpy(keep).to(DEV)] = float("nan")
    o[2, int(np.flatnonzero(keep[2])[0])] = float("nan")
    r[5, 3] = float("inf")
    st = torch.zeros(4, B, device=DEV)
    norm, dr = H.NormWeights(), H.Dropout(0.5, 9, 9)
    r_out, y = H.haste_addnorm_fwd(o, r, norm=norm, stats=st, dropout=dr)
    bad = np.zeros(B, bool)
    bad[[2, 5]] = True
    assert np.isnan(to_f64(y)[bad]).all() and np.isfinite(to_f64(y)[~bad]).all()
    dx, do = H.haste_addnorm_bwd(o, r_out, st, torch.ones_like(y), None, norm=norm, dropout=dr)
    assert np.isfinite(to_f64(dx)[~bad]).all() and (to_f64(do)[~keep] == 0).all() and np.isnan(to_f64(dx)[bad]).all()


def test_addnorm_plain_residual(H):
    """No norm at all: r + o in one rounding, its gradients the same."""
    o, r = rand(gen(1), (9, 130), "bf16"), rand(gen(2), (9, 130), "f32")
    r_out, y = H.haste_addnorm_fwd(o, r)
    assert y is None and torch.equal(r_out, r + o.float())
    dr, do = H.haste_addnorm_bwd(o, r_out, None, None, r)
    assert torch.equal(dr, r) and torch.equal(do, r.bfloat16())


def test_addnorm_gradient_by_differences(H):
    """The kernels' gradients against central differences of the oracle's
    forward in fp64 along random directions."""
    r = np.random.default_rng(11)
    B, D, eps, p = 6, 130, 1e-4, 0.2
    t = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(DEV)  # noqa: E731
    o, x, dy, dro, w = t(B, D), t(B, D), t(B, D), t(B, D), [t(D) for _ in range(4)]
    keep, scale = ops.drop_mask(B, D, p, 5, 6)
    for gate in (t(D), t(B, D)):
        kw = dict(gate=gate, alpha=0.5, post=H.NormWeights(*w[:2]), norm=H.NormWeights(*w[2:]), dropout=H.Dropout(p, 5, 6))
        st, g = torch.empty(4, B, device=DEV), [torch.empty(D, device=DEV) for _ in range(4)]
        dg = torch.empty_like(gate)
        r_out, _ = H.haste_addnorm_fwd(o, x, stats=st, eps=eps, **kw)
        dr, do = H.haste_addnorm_bwd(o, r_out, st, dy, dro, dgate=dg, dpost=H.NormWeights(*g[:2]), dnorm=H.NormWeights(*g[2:]), **kw)

        def f(a):
            s, y, _ = ft.addnorm_fwd(a[0], a[1], a[2], 0.5, a[3:5], a[5:7], eps, keep, scale)
            return float((s * to_f64(dro)).sum() + (y * to_f64(dy)).sum())
        at, got = [to_f64(v) for v in (o, x, gate, *w)], [to_f64(v) for v in (do, dr, dg, *g)]
        for _ in range(4):
            v = [r.standard_normal(a.shape) for a in at]
            h = 1e-6
            want = (f([a + h * b for a, b in zip(at, v)]) - f([a - h * b for a, b in zip(at, v)])) / (2 * h)
            have = sum(float((a * b).sum()) for a, b in zip(got, v))
            size = sum(float(np.abs(a * b).sum()) for a, b in zip(got, v))
            assert abs(have - want) <= 400 * u * size + 1e-7 * size


def test_addnorm_captured(H):
    c = Case(H, CASES[14])
    st, y, r_out = torch.empty(4, c.B, device=DEV), torch.empty(c.B, c.D, device=DEV), torch.empty_like(c.r)
    dy = rand(c.g, (c.B, c.D), c.yt, 0.7)
    _, _, _, _, g = _bwd(H, c)
    ws = torch.empty(H.haste_addnorm_bwd_workspace_bytes(c.B, c.D), dtype=torch.uint8, device=DEV)
    dr, do = torch.empty_like(c.r), torch.empty_like(c.o)

    def go(r_out, y, st, dr, do, ws, g):
        H.haste_addnorm_fwd(c.o, c.r, r_out, y, stats=st, **c.kw)
        H.haste_addnorm_bwd(c.o, r_out, st, dy, dr=dr, do=do, workspace=ws, **dict(c.kw, **g))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(r_out, y, st, dr, do, ws, g)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(r_out, y, st, dr, do, ws, g)
    for i in range(4):
        c.o.copy_(rand(gen(i), (c.B, c.D), c.ot))
        graph.replay()
        _, _, _, _, h = _bwd(H, c)
        want = [torch.empty_like(t) for t in (r_out, y, st, dr, do)]
        go(*want, torch.empty_like(ws), h)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((r_out, y, st, dr, do), want)), i
        assert all(torch.equal(a, _vectors(h)[k]) for k, a in _vectors(g).items())
