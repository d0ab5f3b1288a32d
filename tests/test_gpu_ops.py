"""GPU parity of the operators around the layer (layer norm, dropout, log
probabilities, 8-bit head) against the fp64 oracle, through the C ABI.

Bounds are worst-case rounding bounds of the fp32 formulas: u = 2^-24 a
rounding, sums of n terms in any order n * u, the result rounded once more to
its type.  The hardware exponential of an argument v is taken as within
(2 |v| + 4) 2^-23 of it; a thread adds at most 256 logits one after another
and their partial sums are joined in at most 64 levels, each within 5 * 2^-23.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import ops
from tests._gpu import DEV, to_f64

pytestmark = pytest.mark.gpu
u = 2.0 ** -24
TT = {"bf16": torch.bfloat16, "f32": torch.float32}
TINY = 1e-37     # below this a result may have lost bits


@pytest.fixture(scope="module")
def H():
    from sparse_output_layer_amd import haste
    haste.lib()
    return haste


def rand(g, shape, dt, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).to(TT[dt]).to(DEV)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def rounded(dt, v):
    """Half the spacing of the type (8 or 24 significant bits) at |v|."""
    v = np.asarray(v, np.float64)
    return np.ldexp(0.5, np.frexp(np.where(np.isfinite(v), v, 0.0))[1] - (8 if dt == "bf16" else 24)) + TINY


def within(name, got, ref, bound):
    got, ref, bound = np.asarray(got, np.float64), np.asarray(ref, np.float64), np.asarray(bound, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), f"{name}: NaN in other places"
    inf = ~fin & ~np.isnan(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{name}: infinities differ"
    err = np.abs(got - ref, where=fin, out=np.zeros_like(ref))
    bad = fin & ~(err <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, err / np.maximum(bound, 1e-300), 0)), err.shape)
        raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside; worst at {i}: got {got[i]!r} "
                             f"ref {ref[i]!r} bound {np.broadcast_to(bound, err.shape)[i]!r}")


def strided(t, ld):
    """The same rows with stride ld; the gaps hold NaN."""
    base = torch.full((t.shape[0], ld), float("nan"), dtype=t.dtype, device=t.device)
    base[:, :t.shape[1]] = t
    return base[:, :t.shape[1]]


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("B,D,xt,yt,p", [
    (1, 1, "f32", "f32", 0.5), (1, 8, "bf16", "bf16", 0.1), (3, 7, "bf16", "f32", 0.3), (5, 1001, "f32", "bf16", 0.1),
    (64, 768, "bf16", "bf16", 0.1), (130, 1024, "f32", "f32", 0.9), (2, 50000, "bf16", "bf16", 0.25),
    (4099, 9, "bf16", "bf16", 0.5), (7, 96, "f32", "f32", 0.0), (7, 96, "f32", "f32", 1.0), (1000, 1, "bf16", "f32", 0.4)])
def test_dropout_bits(H, B, D, xt, yt, p):
    """Kept elements are x times the fp32 scale, rounded once; the mask is the
    generator's: equal bit for bit."""
    print(f"dropout {B}x{D} {xt}->{yt} p={p}", flush=True)
    seed, off = 0x123456789ABCDEF, (1 << 40) + 5
    x = rand(gen(B + D), (B, D), xt)
    keep, scale = ops.drop_mask(B, D, p, seed, off)
    y = H.haste_dropout_apply(x, H.Dropout(p, seed, off), torch.empty(B, D, dtype=TT[yt], device=DEV))
    k = torch.from_numpy(keep)
    want = torch.where(k, x.float().cpu() * torch.tensor(np.float32(scale)), torch.zeros(())).to(TT[yt])
    assert torch.equal(y.cpu(), want)
    if xt == yt:   # in place
        H.haste_dropout_apply(x, H.Dropout(p, seed, off), x)
        assert torch.equal(x, y)


def test_dropout_drops_nan_and_unaligned(H):
    x = rand(gen(1), (1, 1001), "bf16")
    keep, _ = ops.drop_mask(40, 25, 0.5, 77, 0)
    v = x[0, 1:].reshape(40, 25)            # base two bytes past an aligned one
    x[0, 1:][~torch.from_numpy(keep).reshape(-1).to(DEV)] = float("nan")
    y = torch.empty(1003, dtype=torch.bfloat16, device=DEV)[3:].reshape(40, 25)
    H.haste_dropout_apply(v, H.Dropout(0.5, 77), y)
    assert torch.isfinite(y).all() and (to_f64(y)[~keep] == 0).all()
    assert torch.equal(y.float()[torch.from_numpy(keep).to(DEV)], v.float()[torch.from_numpy(keep).to(DEV)] * 2)


# --------------------------------------------------------------- layer norm
NORMS = [  # B, D, x, y, w, p, row stride beyond D, affine
    (1, 1, "f32", "f32", "f32", 0.0, 0, True), (1, 1024, "bf16", "bf16", "f32", 0.0, 0, True),
    (5, 3, "bf16", "f32", "bf16", 0.0, 2, True), (33, 768, "bf16", "bf16", "f32", 0.1, 0, True),
    (33, 768, "bf16", "f32", "bf16", 0.1, 768 * 3, True), (17, 1001, "f32", "f32", "f32", 0.0, 0, True),
    (17, 1001, "bf16", "bf16", "f32", 0.5, 6, True), (9, 4097, "f32", "bf16", "f32", 0.1, 3, True),
    (300, 64, "bf16", "bf16", "f32", 0.0, 0, False), (3, 8192, "bf16", "bf16", "bf16", 0.0, 0, True),
    (2, 20011, "f32", "f32", "f32", 0.1, 0, True), (700, 1024, "f32", "bf16", "f32", 0.1, 0, True),
    (1500, 96, "bf16", "f32", "f32", 0.0, 0, True), (4, 70001, "bf16", "f32", "f32", 0.0, 1, True),
    (2051, 520, "bf16", "f32", "f32", 0.1, 0, True), (64, 2048, "f32", "f32", "bf16", 0.0, 8, True),
    (40, 16, "bf16", "bf16", "bf16", 0.2, 0, True), (6, 3001, "bf16", "bf16", "f32", 0.0, 0, True)]


def _norm_case(H, case):
    B, D, xt, yt, wt, p, gap, affine = case
    print(f"norm {case}", flush=True)
    g = gen(B * 7 + D)
    x = rand(g, (B, D), xt, 1.5, 3.0)
    if gap:
        x = strided(x, D + gap)
    ga = rand(g, (D,), wt, 0.3, 1.0) if affine else None
    be = rand(g, (D,), wt, 0.3) if affine else None
    seed, off = 987654321987, 3
    dr = H.Dropout(p, seed, off) if p else None
    keep, scale = ops.drop_mask(B, D, p, seed, off) if p else (None, 1.0)
    return g, x, ga, be, dr, keep, scale


@pytest.mark.parametrize("case", NORMS)
def test_norm_fwd(H, case):
    B, D, xt, yt, wt, p, gap, affine = case
    g, x, ga, be, dr, keep, scale = _norm_case(H, case)
    eps = 1e-5
    mean, rstd = (torch.full((B,), 7.0, device=DEV) for _ in range(2))
    y = H.haste_norm_fwd(x, ga, be, torch.empty(B, D, dtype=TT[yt], device=DEV), mean, rstd, eps, dr)
    y2 = H.haste_norm_fwd(x, ga, be, torch.empty(B, D, dtype=TT[yt], device=DEV), eps=eps, dropout=dr)
    assert torch.equal(y, y2)
    X = to_f64(x)
    G, Be = (None if t is None else to_f64(t) for t in (ga, be))
    ry, rm, rr = ops.norm_fwd(X, G, Be, eps, keep, scale)
    dm = (D + 2) * u * np.abs(X).mean(1)
    var = ((X - rm[:, None]) ** 2).mean(1)
    sd = np.sqrt(var)
    dvar = 2 * sd * (dm + u * sd) + (dm + u * sd) ** 2 + (D + 8) * u * var
    rel = dvar / (var + eps) + 4 * u            # of rstd (half of it, with second-order room)
    within("mean", to_f64(mean), rm, dm + u * np.abs(rm))
    within("rstd", to_f64(rstd), rr, rel * rr)
    h = np.abs((X - rm[:, None]) * rr[:, None])
    dh = h * (rel[:, None] + 3 * u) + rr[:, None] * (dm[:, None] + u * np.abs(X - rm[:, None]))
    A = np.abs(G)[None, :] if affine else 1.0
    Ab = np.abs(Be)[None, :] if affine else 0.0
    bound = scale * (A * dh + 4 * u * (A * h + Ab))
    within("y", to_f64(y), ry, bound + rounded(yt, np.abs(ry) + bound))


@pytest.mark.parametrize("case", NORMS)
def test_norm_bwd(H, case):
    B, D, xt, yt, wt, p, gap, affine = case
    g, x, ga, be, dr, keep, scale = _norm_case(H, case)
    dy = rand(g, (B, D), yt, 0.7)
    X, G, DY = to_f64(x), None if ga is None else to_f64(ga), to_f64(dy)
    _, m, r = ops.norm_fwd(X, G, None, 1e-5)
    mean, rstd = (torch.from_numpy(t.astype(np.float32)).to(DEV) for t in (m, r))
    m, r = to_f64(mean), to_f64(rstd)
    rdx, rdg, rdb = ops.norm_bwd(X, G, m, r, DY, keep, scale)
    dg, db = (torch.full((D,), 5.0, device=DEV) for _ in range(2))
    dx = torch.empty(B, D, dtype=TT[xt], device=DEV)
    if gap:
        dx = strided(dx, D + gap + 1)
    H.haste_norm_bwd(x, ga, mean, rstd, dy, dx, dg, db, dr)
    h = np.abs((X - m[:, None]) * r[:, None])
    a = np.abs(DY) * scale * (keep if keep is not None else 1.0)
    gg = a if G is None else a * np.abs(G)
    R = r[:, None]
    bound = R * (6 * u * gg + (D + 8) * u * gg.mean(1)[:, None] + h * (D + 12) * u * (gg * h).mean(1)[:, None])
    within("dx", to_f64(dx), rdx, bound + rounded(xt, np.abs(rdx) + bound))
    bg, bb = (B + 8) * u * (a * h).sum(0), (B + 4) * u * a.sum(0)
    within("dgamma", to_f64(dg), rdg, bg + TINY)
    within("dbeta", to_f64(db), rdb, bb + TINY)
    if gap:   # the gaps are untouched
        assert torch.isnan(dx.as_strided((B - 1, gap + 1), (D + gap + 1, 1), dx.storage_offset() + D)).all()
    # added to; one of them alone; dx alone; equal bits every time
    dg2, db2 = torch.full((D,), 5.0, device=DEV), torch.full((D,), 5.0, device=DEV)
    dx2 = H.haste_norm_bwd(x, ga, mean, rstd, dy, None, dg2, db2, dr, accumulate_dw=True)
    assert torch.equal(dx2, dx) and torch.equal(dg2, dg + 5.0) and torch.equal(db2, db + 5.0)
    dg3 = torch.empty(D, device=DEV)
    dx3 = H.haste_norm_bwd(x, ga, mean, rstd, dy, None, dg3, None, dr)
    assert torch.equal(dx3, dx) and torch.equal(dg3, dg)
    assert torch.equal(H.haste_norm_bwd(x, ga, mean, rstd, dy, None, dropout=dr), dx)


@pytest.mark.parametrize("D", [2, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 127, 129, 250, 257, 259, 511, 514, 767, 771, 1023,
                               1028, 1533, 1537, 2045, 2049, 4093, 4098, 8190, 8193])
def test_row_ends(H, D):
    """Rows that end at every place of a vector of eight, on both sides of the
    widths where the kernels change, through every operator that reads rows."""
    for xt, yt, gap in (("bf16", "f32", 0), ("f32", "bf16", 5)):
        case = (5, D, xt, yt, "f32", 0.25, gap, True)
        test_norm_fwd(H, case)
        test_norm_bwd(H, case)
        test_dropout_bits(H, 5, D, xt, yt, 0.25)
        test_quantize_bits(H, 5, D, xt, gap)


@pytest.mark.parametrize("B", [2, 127, 129, 255, 384, 511, 512, 513])
@pytest.mark.parametrize("D", [40, 200, 333, 777, 1300, 2500, 5001])
def test_norm_bwd_few_rows(H, B, D):
    """Both ways of summing the weight gradient, at row counts around the threads' shares."""
    test_norm_bwd(H, (B, D, "bf16", "f32", "f32", 0.1, 0, True))
    test_norm_bwd(H, (B, D, "f32", "bf16", "bf16", 0.0, 3, True))


def test_norm_nan_stays_in_its_row(H):
    x = rand(gen(5), (6, 200), "bf16")
    x[2, 7], x[4, 0] = float("nan"), float("inf")
    mean, rstd = torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    y = to_f64(H.haste_norm_fwd(x, mean=mean, rstd=rstd))
    bad = np.array([2, 4])
    assert np.isnan(y[bad]).all() and np.isfinite(np.delete(y, bad, 0)).all()
    dx = to_f64(H.haste_norm_bwd(x, None, mean, rstd, torch.ones_like(x)))
    assert np.isnan(dx[bad]).all() and np.isfinite(np.delete(dx, bad, 0)).all()


def test_norm_constant_rows(H):
    x = torch.full((4, 333), 2.5, device=DEV)
    be = torch.arange(333, dtype=torch.float32, device=DEV)
    mean, rstd = torch.empty(4, device=DEV), torch.empty(4, device=DEV)
    y = H.haste_norm_fwd(x, None, be, None, mean, rstd, eps=1e-6)
    # the mean is within its bound of 2.5, so (x - mean) * rstd within 336u * 2.5 * 1000
    assert (y - be).abs().max().item() <= 336 * u * 2.5 * 1000 + 333 * u
    assert abs(rstd[0].item() - 1000.0) <= 1.0


def test_norm_gradient_by_differences(H):
    """The kernels' dx, dgamma and dbeta against central differences of the
    oracle's forward in fp64 along random directions."""
    r = np.random.default_rng(11)
    B, D, eps, p = 6, 130, 1e-4, 0.2
    x, ga, be, dy = (torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(DEV)
                     for s in ((B, D), (D,), (D,), (B, D)))
    dr = H.Dropout(p, 5, 6)
    keep, scale = ops.drop_mask(B, D, p, 5, 6)
    mean, rstd, dg, db = (torch.empty(n, device=DEV) for n in (B, B, D, D))
    H.haste_norm_fwd(x, ga, be, None, mean, rstd, eps, dr)
    dx = H.haste_norm_bwd(x, ga, mean, rstd, dy, None, dg, db, dr)
    X, G, Be, DY = (to_f64(t) for t in (x, ga, be, dy))
    f = lambda a, b, c: float((ops.norm_fwd(a, b, c, eps, keep, scale)[0] * DY).sum())  # noqa: E731
    for _ in range(4):
        vx, vg, vb = r.standard_normal((B, D)), r.standard_normal(D), r.standard_normal(D)
        h = 1e-6
        want = (f(X + h * vx, G + h * vg, Be + h * vb) - f(X - h * vx, G - h * vg, Be - h * vb)) / (2 * h)
        got = float((to_f64(dx) * vx).sum() + (to_f64(dg) * vg).sum() + (to_f64(db) * vb).sum())
        size = float(np.abs(to_f64(dx) * vx).sum() + np.abs(to_f64(dg) * vg).sum() + np.abs(to_f64(db) * vb).sum())
        assert abs(got - want) <= 200 * u * size + 1e-7 * size


# -------------------------------------------------------- log probabilities
LPS = [  # B, H, L, type, given labels a row, K, strides beyond the rows
    (1, 1, 0, "f32", 1, 1, 0), (1, 0, 1, "bf16", 1, 8, 0), (3, 7, 0, "f32", 2, 3, 1), (2, 64, 1000, "bf16", 3, 5, 0),
    (5, 8191, 0, "f32", 3, 8, 0), (4, 0, 40001, "bf16", 4, 5, 7), (4, 129, 20003, "bf16", 5, 8, 0),
    (33, 96, 515, "f32", 2, 1, 3), (2, 8192, 8192, "bf16", 0, 2, 0), (300, 17, 33, "bf16", 1, 0, 0),
    (2, 30, 70003, "f32", 40, 4, 0), (1, 32768, 131072, "bf16", 300, 8, 0)]


def _lp_case(case, seed=0, std=2.0):
    B, Hn, L, dt, P, K, gap = case
    print(f"logprob {case}", flush=True)
    g = gen(B + Hn + L + seed)
    zs = []
    for n in (Hn, L):
        if n == 0:
            zs.append(None)
            continue
        z = rand(g, (B, n), dt, std, -0.5)
        m = torch.rand((B, n), generator=g) < 0.05       # some masked labels
        z[m.to(DEV)] = float("-inf")
        z[:, 0] = 0.25                                    # every row keeps one
        zs.append(strided(z, n + gap) if gap else z)
    off = 50
    r = np.random.default_rng(seed + B)
    cnt = r.integers(0, 2 * P + 1, B) if P else np.zeros(B, dtype=np.int64)
    rp = np.concatenate([[0], np.cumsum(cnt)]).astype(np.int32)
    lab = r.integers(off - 2, off + Hn + L + 2, int(rp[-1])).astype(np.int32)    # repeats, and ids outside
    if len(lab) > 2:
        lab[1] = lab[0]
    return zs, off, rp, lab


def _all(zs):
    return np.concatenate([to_f64(t) for t in zs if t is not None], axis=1)


def _bce(H, rp, lab, off, B, K, loss=False, s=1.0):
    return H.Bce(torch.from_numpy(rp).to(DEV), torch.from_numpy(lab).to(DEV), off, s,
                 torch.full((1,), 3.0, device=DEV) if loss else None,
                 torch.empty(B, K, device=DEV) if K else None,
                 torch.empty(B, K, dtype=torch.int32, device=DEV) if K else None)


def _lp_bounds(z, lse, lp):
    """Bounds of lse and entropy (see the module's note)."""
    p = np.exp(np.where(np.isfinite(lp), lp, -np.inf))
    v = z - np.where(np.isfinite(z), z, -np.inf).max(1, initial=-1e30)[:, None]
    v = np.where(p > 0, np.abs(v), 0.0)
    ev = (p * v).sum(1)
    dS = 2.0 ** -23 * (4 + 2 * ev) + 320 * u + 64 * 5 * 2.0 ** -23
    ev2 = (p * v * (2 * v + 4)).sum(1) * 2.0 ** -23
    dl = dS + 2 * u * np.abs(np.where(np.isfinite(lse), lse, 0)) + 8 * u
    logS = np.log(np.maximum((np.exp(-v) * (p > 0)).sum(1), 1.0))
    dent = dS + ev2 + 2 * dS * ev + 4 * u * (logS + ev)
    return dl, dent


def _lp_check(H, case, zs, off, rp, lab, K, loss=True):
    B = case[0]
    z = _all(zs)
    given = _bce(H, rp, lab, off, B, K, loss, 0.5)
    lse, ent, logp = (torch.full((n,), 9.0, device=DEV) for n in (B, B, len(lab)))
    H.haste_logprob_fwd(zs[0], zs[1], given, lse, logp, ent)
    rl, re, lp = ops.logprob_rows(z)
    rlp = ops.logprob_given(lp, rp, lab, off)
    dl, de = _lp_bounds(z, rl, lp)
    within("lse", to_f64(lse), rl, dl)
    within("entropy", to_f64(ent), re, de)
    row = np.repeat(np.arange(B), np.diff(rp))
    blp = dl[row] + 4 * u * np.abs(np.where(np.isfinite(rlp), rlp, 0)) + 2 * u * np.abs(np.nan_to_num(rl[row], posinf=0, neginf=0))
    within("logp", to_f64(logp), rlp, blp)
    if K:
        rv, ri = ops.logprob_top(z, lp, K, off)
        assert np.array_equal(given.topk_idx.cpu().numpy(), ri)
        within("alternatives", to_f64(given.topk_val), rv,
               dl[:, None] + 4 * u * np.abs(np.where(np.isfinite(rv), rv, 0)) + 2 * u * np.abs(np.nan_to_num(rl, posinf=0, neginf=0))[:, None])
    if loss:
        N = z.shape[1]
        part = rlp[(lab >= off) & (lab < off + N)]
        want = 3.0 - 0.5 * part.sum()
        if math.isfinite(want):
            b = 0.5 * blp[(lab >= off) & (lab < off + N)].sum() + (len(lab) + 300) * u * (3 + 0.5 * np.abs(part).sum())
            assert abs(given.loss.item() - want) <= b
        else:
            within("loss", [given.loss.item()], [want], [0])
    # alone, without labels: the same bits
    lse2 = torch.empty(B, device=DEV)
    H.haste_logprob_fwd(zs[0], zs[1], None, lse2)
    assert torch.equal(lse2.view(torch.int32), lse.view(torch.int32))
    return lse, ent, z


@pytest.mark.parametrize("case", LPS)
def test_logprob_fwd(H, case):
    B, Hn, L, dt, P, K, gap = case
    zs, off, rp, lab = _lp_case(case)
    _lp_check(H, case, zs, off, rp, lab, K)


def test_logprob_hard_rows(H):
    """Masked rows, ties, the type's lowest values, infinities and NaN, wide
    ranges; each in its own row, and -0 equal to 0."""
    inf = float("inf")
    for dt in ("bf16", "f32"):
        low = torch.finfo(TT[dt]).min
        for Hn, L in ((37, 0), (0, 9001), (40, 12000)):
            z = torch.zeros(12, Hn + L)
            z[0] = -inf                          # nothing left
            z[1] = -inf
            z[1, -1] = -5.0                      # one label left
            z[2] = low                           # every logit the lowest value
            z[3, ::2] = low                      # half of them masked by it
            z[4] = torch.linspace(-30, 30, Hn + L)
            z[4, 5] = float("nan")
            z[5, 3] = inf
            z[6, 1::2] = -0.0                    # ties between 0 and -0
            z[7] = 1.5                           # ties everywhere
            z[8] = torch.linspace(-3e4, 3e4, Hn + L)
            z[9, :] = low / 4
            z[9, 20] = torch.finfo(TT[dt]).max / 4   # the widest range whose differences are finite
            z[10] = float("nan")
            z[11, :30] = -inf                    # a masked start
            z = z.to(TT[dt]).to(DEV)
            zs = [z[:, :Hn].contiguous() if Hn else None, z[:, Hn:].contiguous() if L else None]
            rp = (np.arange(13) * 3).astype(np.int32)
            lab = np.tile([0, 20, Hn + L - 1], 12).astype(np.int32)
            case = (12, Hn, L, dt, 3, 8, 0)
            print(case, flush=True)
            lse, ent, zz = _lp_check(H, case, zs, 0, rp, lab, 8, loss=False)
            dzs = [None if t is None else torch.full_like(t, 7.0) for t in zs]
            H.haste_logprob_bwd(zs[0], zs[1], H.Bce(torch.from_numpy(rp).to(DEV), torch.from_numpy(lab).to(DEV)), lse,
                                dzs[0], dzs[1], entropy=ent, dentropy=torch.full((12,), 0.5, device=DEV))
            dz = _all(dzs)
            assert (dz[0] == 0).all()
            assert np.isnan(dz[[4, 10]]).all() and np.isnan(dz[5]).all()
            assert np.isfinite(np.delete(dz, [4, 5, 10], 0)).all()
            # entries -1 each: the masked label keeps its own, the last (p = 1) has -1 + 3
            assert dz[1, 0] == -1 and dz[1, 7] == 0 and dz[1, -1] == 2


@pytest.mark.parametrize("Hn,L,dt", [(0, 70001, "bf16"), (300, 40003, "f32"), (5000, 0, "bf16")])
def test_logprob_many_ties(H, Hn, L, dt):
    """Rows with more equal logits than can be ranked at once: all equal (the
    zero-weight start), equal ones below a few larger, in the second half
    only, every third, rising through one thread's vectors, and with -0."""
    N = Hn + L
    z = torch.zeros(8, N)
    z[1, [7, N // 2, N - 1]] = torch.tensor([2.0, 3.0, 1.0])
    z[2, :N // 2] = -4.0
    z[3] = -1.0
    z[3, ::3] = 0.5
    z[4] = -5.0
    z[4, :4096] = torch.arange(4096) / 512.0
    z[5, ::2] = -0.0
    z[6] = -1e9
    z[7, : N - 3] = -math.inf
    z = z.to(TT[dt]).to(DEV)
    zs = [z[:, :Hn].contiguous() if Hn else None, z[:, Hn:].contiguous() if L else None]
    rp, lab = np.arange(9, dtype=np.int32), np.full(8, N - 1, np.int32)
    for K in (1, 5, 8):
        print(Hn, L, dt, K, flush=True)
        _lp_check(H, (8, Hn, L, dt, 1, K, 0), zs, 0, rp, lab, K)


@pytest.mark.parametrize("N,dt", [(15000, "f32"), (30000, "bf16"), (200001, "bf16")])
def test_logprob_some_ties(H, N, dt):
    """Equal largest logits, in number around what is searched and ranked at a
    time, scattered over the row and in one run."""
    counts = [7, 8, 9, 63, 64, 65, 100, 300, 511, 512, 513, 700, 1500]
    g = gen(N)
    z = torch.rand((2 * len(counts), N), generator=g)
    for i, n in enumerate(counts):
        z[2 * i, torch.randperm(N, generator=g)[:n]] = 4.0
        z[2 * i + 1, N // 3:N // 3 + n] = 4.0
    zs = [z.to(TT[dt]).to(DEV), None]
    B = len(z)
    rp, lab = np.arange(B + 1, dtype=np.int32), np.full(B, N // 3, np.int32)
    for K in (1, 8):
        print(N, dt, K, flush=True)
        _lp_check(H, (B, N, 0, dt, 1, K, 0), zs, 0, rp, lab, K)


def test_logprob_repeats_are_equal(H):
    """Two runs give the same bits, and another stream's run too."""
    case = (7, 100, 50001, "bf16", 3, 5, 0)
    zs, off, rp, lab = _lp_case(case)
    outs = []
    s = torch.cuda.Stream()
    for k in range(3):
        given = _bce(H, rp, lab, off, 7, 5, True)
        lse, ent, logp = (torch.empty(n, device=DEV) for n in (7, 7, len(lab)))
        if k == 2:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                H.haste_logprob_fwd(zs[0], zs[1], given, lse, logp, ent)
            torch.cuda.current_stream().wait_stream(s)
        else:
            H.haste_logprob_fwd(zs[0], zs[1], given, lse, logp, ent)
        outs.append([t.clone() for t in (lse, ent, logp, given.topk_val, given.topk_idx, given.loss)])
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


@pytest.mark.parametrize("case", LPS)
@pytest.mark.parametrize("form", ["loss", "both", "entropy"])
def test_logprob_bwd(H, case, form):
    B, Hn, L, dt, P, K, gap = case
    zs, off, rp, lab = _lp_case(case, seed=1)
    z = _all(zs)
    rl, re, lp = ops.logprob_rows(z)
    lse, ent = (torch.from_numpy(t.astype(np.float32)).to(DEV) for t in (rl, re))
    r = np.random.default_rng(8)
    dl = None if form == "loss" else torch.from_numpy(r.standard_normal(len(lab)).astype(np.float32)).to(DEV)
    de = None if form == "loss" else torch.from_numpy(r.standard_normal(B).astype(np.float32)).to(DEV)
    given = None if form == "entropy" else _bce(H, rp, lab, off, B, 0, False, 0.25)
    if form == "entropy":
        dl, rp, lab = None, np.zeros(B + 1, np.int32), np.zeros(0, np.int32)
    dzs = [None if t is None else torch.full((B, t.shape[1]), 7.0, dtype=t.dtype, device=DEV) for t in zs]
    H.haste_logprob_bwd(zs[0], zs[1], given, lse, dzs[0], dzs[1], entropy=ent, dlogp=dl, dentropy=de)
    g = np.full(len(lab), -0.25) if dl is None else to_f64(dl)
    n = None if de is None else to_f64(de)
    l32, e32 = to_f64(lse), to_f64(ent)
    ref = ops.logprob_bwd(z, l32, e32, rp, lab, g, n, off)
    N = z.shape[1]
    lp = z - l32[:, None]
    p = np.exp(lp)
    al = np.where(p > 0, np.abs(lp), 0.0)
    Ga = np.zeros(B)
    hot = np.zeros((B, N))
    for b in range(B):
        for e in range(rp[b], rp[b + 1]):
            j = int(lab[e]) - off
            if 0 <= j < N:
                Ga[b] += abs(g[e])
                hot[b, j] += abs(g[e])
    na = np.zeros(B) if n is None else np.abs(n)
    coef = Ga[:, None] + na[:, None] * (al + np.abs(e32)[:, None])
    cnt = np.diff(rp)[:, None]
    bound = p * coef * (2.0 ** -23 * (2 * al + 4) + (al + 16 + cnt) * u) + (cnt + 2) * u * hot + 1e-36 * (coef + 1)
    within("dz", _all(dzs), ref, bound + rounded(dt, np.abs(ref) + bound))


def test_logprob_gradient_by_differences(H):
    r = np.random.default_rng(21)
    B, N = 4, 700
    z = torch.from_numpy((2 * r.standard_normal((B, N))).astype(np.float32)).to(DEV)
    rp = np.array([0, 2, 2, 5, 6], np.int32)
    lab = np.array([3, 699, 0, 0, 77, 5], np.int32)
    dl, de = (torch.from_numpy(r.standard_normal(k).astype(np.float32)).to(DEV) for k in (6, B))
    given = _bce(H, rp, lab, 0, B, 0)
    lse, ent, dz = torch.empty(B, device=DEV), torch.empty(B, device=DEV), torch.empty_like(z)
    H.haste_logprob_fwd(z, None, given, lse, entropy=ent)
    H.haste_logprob_bwd(z, None, given, lse, dz, None, entropy=ent, dlogp=dl, dentropy=de)
    Z, DL, DE = to_f64(z), to_f64(dl), to_f64(de)

    def f(t):
        _, e, lp = ops.logprob_rows(t)
        return float(DL @ ops.logprob_given(lp, rp, lab) + DE @ e)
    for _ in range(4):
        v = r.standard_normal((B, N))
        want = (f(Z + 1e-5 * v) - f(Z - 1e-5 * v)) / 2e-5
        size = float(np.abs(to_f64(dz) * v).sum())
        assert abs(float((to_f64(dz) * v).sum()) - want) <= 400 * u * size + 1e-6 * size


# -------------------------------------------------------------- 8-bit head
@pytest.mark.parametrize("rows,D,dt,gap", [(1, 1, "f32", 0), (3, 63, "bf16", 0), (5, 64, "bf16", 1), (7, 65, "f32", 2),
                                           (33, 768, "bf16", 0), (4, 1001, "bf16", 0), (2, 20011, "f32", 0),
                                           (1030, 96, "f32", 0), (9, 1024, "f32", 3), (300, 1024, "bf16", 0)])
def test_quantize_bits(H, rows, D, dt, gap):
    print(f"quantize {rows}x{D} {dt} gap {gap}", flush=True)
    x = rand(gen(rows + D), (rows, D), dt, 3.0)
    if rows > 2:
        x[1] = 0.0
        x[2] = x[2] * 1e-36          # scale below the smallest normal number
    if gap:
        x = strided(x, D + gap)
    q, s = H.haste_quantize_rows(x)
    rq, rs = ops.quantize_rows(to_f64(x).astype(np.float32))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy()[:, :D], rq) and (q.cpu().numpy()[:, D:] == 0).all()


def test_quantize_agrees_with_tensor_arithmetic(H):
    """Features on a coarse grid, where x / scale is often a tie but for the
    scale's last bit: the same scales and integers as tensors give."""
    x = (torch.randint(-255, 256, (4096, 256), generator=gen(9), dtype=torch.int32).float() / 64).to(DEV)
    s = x.abs().amax(1) / 127.0
    want = torch.round(x / s[:, None]).clamp(-127, 127).to(torch.int8)
    q, scale = H.haste_quantize_rows(x)
    assert torch.equal(scale, s) and torch.equal(q, want)


def test_quantize_ties_and_bad_rows(H):
    x = torch.zeros(4, 70)
    x[0, :6] = torch.tensor([127.0, 0.5, 1.5, -2.5, -127.0, 126.5])     # ties to even
    x[1, 3], x[2, 69] = float("nan"), float("-inf")
    q, s = H.haste_quantize_rows(x.to(DEV))
    assert q[0, :6].tolist() == [127, 0, 2, -2, -127, 126] and s[0] == 1.0
    assert math.isnan(s[1]) and math.isinf(s[2])
    Z = torch.empty(4, 4, device=DEV)
    H.haste_head_fwd_i8(q, s, q, s, 70, Z)
    z = to_f64(Z)
    assert np.isnan(z[1:3]).all() and np.isnan(z[:, 1:3]).all()
    assert z[0, 0] == 127 * 127 * 2 + 4 + 4 + 126 * 126 and (z[3, [0, 3]] == 0).all()


@pytest.mark.parametrize("B,D,N,zt", [
    (1, 1, 1, "f32"), (1, 1024, 32768, "f32"), (1, 768, 1000, "bf16"), (2, 65, 17, "bf16"), (5, 63, 33, "f32"),
    (16, 768, 8192, "bf16"), (17, 128, 129, "bf16"), (33, 1001, 257, "f32"), (64, 256, 512, "bf16"),
    (100, 64, 100, "bf16"), (128, 1024, 4096, "bf16"), (130, 1030, 1031, "f32"), (512, 768, 8192, "bf16"),
    (255, 2000, 383, "bf16"), (1000, 320, 1001, "bf16"), (300, 4096, 600, "f32"), (8, 20011, 70, "f32")])
def test_head_i8(H, B, D, N, zt):
    """The integer sum is exact (int32; exact in fp32 below 2^24, else one
    rounding), scaled by two fp32 factors, rounded to the type."""
    print(f"head i8 {B}x{D}x{N} {zt}", flush=True)
    g = gen(B + D + N)
    Xq, xs = H.haste_quantize_rows(rand(g, (B, D), "bf16"))
    Wq, ws = H.haste_quantize_rows(rand(g, (N, D), "f32", 0.02))
    Z = torch.full((B, N), 7.0, dtype=TT[zt], device=DEV)
    H.haste_head_fwd_i8(Xq, xs, Wq, ws, D, Z)
    ref = _i8_ref(Xq, xs, Wq, ws)
    within("Zh", to_f64(Z), ref, 4 * u * np.abs(ref) + rounded(zt, np.abs(ref) * (1 + 4 * u)))


def _i8_ref(Xq, xs, Wq, ws):
    """Exact in fp64 (the sums stay below 2^53)."""
    x, w = (t.cpu().numpy().astype(np.float64) for t in (Xq, Wq))
    return (x @ w.T) * xs.cpu().numpy().astype(np.float64)[:, None] * ws.cpu().numpy().astype(np.float64)[None, :]


def test_head_i8_extremes(H):
    """Every product at its largest: the sum 127 * 127 * D stays in 32 bits."""
    D = 131072
    q = torch.full((2, D), 127, dtype=torch.int8, device=DEV)
    q[1] = -127
    s = torch.ones(2, device=DEV)
    Z = torch.empty(2, 2, device=DEV)
    H.haste_head_fwd_i8(q, s, q, s, D, Z)
    want = 127 * 127 * D
    within("Zh", to_f64(Z), [[want, -want], [-want, want]], u * want)


# ------------------------------------------- capture, and past 32 bits
def test_replayed_graph_equals_eager(H):
    """Every operator captured into one graph, replayed three times with
    eager work between, each replay bit for bit the eager result."""
    g = gen(31)
    x, dy = rand(g, (70, 300), "bf16"), rand(g, (70, 300), "f32")
    ga, be = rand(g, (300,), "f32"), rand(g, (300,), "f32")
    Zh, Z = rand(g, (70, 100), "bf16"), rand(g, (70, 5001), "bf16")
    rp, lab = np.arange(71, dtype=np.int32) * 2, np.tile(np.array([5, 3000], np.int32), 70)
    Wq, ws = H.haste_quantize_rows(rand(g, (200, 300), "f32"))
    given = _bce(H, rp, lab, 0, 70, 4, True)
    dr = H.Dropout(0.3, 5, 9)
    o = dict(y=torch.empty_like(x), mean=torch.empty(70, device=DEV), rstd=torch.empty(70, device=DEV), dx=torch.empty_like(x),
             dg=torch.empty(300, device=DEV), db=torch.empty(300, device=DEV), dp=torch.empty_like(dy),
             lse=torch.empty(70, device=DEV), ent=torch.empty(70, device=DEV), logp=torch.empty(140, device=DEV),
             dzh=torch.empty_like(Zh), dz=torch.empty_like(Z), q=torch.empty(70, 320, dtype=torch.int8, device=DEV),
             s=torch.empty(70, device=DEV), zi=torch.empty(70, 200, device=DEV),
             tv=given.topk_val, ti=given.topk_idx, loss=given.loss)
    space = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)

    def step():
        o["loss"].zero_()
        H.haste_norm_fwd(x, ga, be, o["y"], o["mean"], o["rstd"], dropout=dr)
        H.haste_norm_bwd(x, ga, o["mean"], o["rstd"], dy, o["dx"], o["dg"], o["db"], dr, workspace=space)
        H.haste_dropout_apply(dy, dr, o["dp"])
        H.haste_logprob_fwd(Zh, Z, given, o["lse"], o["logp"], o["ent"], workspace=space)
        H.haste_logprob_bwd(Zh, Z, given, o["lse"], o["dzh"], o["dz"], entropy=o["ent"], dentropy=o["ent"])
        H.haste_quantize_rows(o["y"], o["q"], o["s"])
        H.haste_head_fwd_i8(o["q"], o["s"], Wq, ws, 300, o["zi"])
    step()
    torch.cuda.synchronize()
    want = {k: v.clone() for k, v in o.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for v in o.values():
            v.fill_(3)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, v in o.items():
            assert torch.equal(v, want[k]), k


def test_logprob_past_32_bits(H):
    """255 rows of 8,600,001 logits (more than 2^31 of them), all the same row:
    every row's results equal the first's, and the first's the oracle's."""
    B, N = 255, 8_600_001
    g = gen(40)
    row = (torch.randn(N, generator=g) * 1.5).to(torch.bfloat16).to(DEV)
    z = torch.empty(B, N, dtype=torch.bfloat16, device=DEV)
    z.copy_(row.expand(B, N))
    rp, lab = np.arange(B + 1, dtype=np.int32), np.full(B, N - 1, np.int32)
    given = _bce(H, rp, lab, 0, B, 5)
    lse, ent, logp = (torch.empty(B, device=DEV) for _ in range(3))
    H.haste_logprob_fwd(None, z, given, lse, logp, ent)
    dz = torch.empty_like(z)
    H.haste_logprob_bwd(None, z, given, lse, None, dz)
    # a row's vectors start where its address says, so sums may round
    # differently from row to row; each is within its own bound of the oracle
    zr = to_f64(row)[None, :]
    rl, re, lp = ops.logprob_rows(zr)
    dl, de = _lp_bounds(zr, rl, lp)
    within("lse", to_f64(lse), np.full(B, rl[0]), np.full(B, dl[0]))
    within("entropy", to_f64(ent), np.full(B, re[0]), np.full(B, de[0]))
    rv, ri = ops.logprob_top(zr, lp, 5)
    assert (given.topk_idx.cpu().numpy() == ri).all()
    for b in (0, 249, 254):      # row 249 holds element 2^31
        ref = ops.logprob_bwd(zr, np.array([lse[b].item()]), re, [0, 1], lab[:1], [-1.0])[0]
        p = np.exp(zr[0] - lse[b].item())
        bound = p * (2.0 ** -23 * (2 * np.abs(np.log(p)) + 4) + (np.abs(np.log(p)) + 16) * u) + 2 * u
        bound[:-1] -= 2 * u
        within("dz", to_f64(dz[b]), ref, bound + rounded("bf16", np.abs(ref) + bound))


def test_norm_and_dropout_past_32_bits(H):
    """2,100,000 rows of 1,024 (more than 2^31 elements) of one row's values."""
    B, D = 2_100_000, 1024
    row = rand(gen(41), (1, D), "bf16")
    x = torch.empty(B, D, dtype=torch.bfloat16, device=DEV)
    x.copy_(row.expand(B, D))
    one = H.haste_norm_fwd(row)
    y = H.haste_norm_fwd(x)
    assert all(torch.equal(y[b:b + 1], one) for b in (0, 2_097_151, 2_097_152, B - 1))
    assert bool((y[2_000_000:] == one).all())
    H.haste_dropout_apply(x, H.Dropout(0.5, 3, 1), x)
    for b in (0, 2_097_152, B - 1):
        w = ops.philox4x32((np.arange(128), np.full(128, b), np.full(128, 1), np.zeros(128)), (3, 0))
        half = np.stack([t for v in w for t in (v & np.uint64(0xFFFF), v >> np.uint64(16))], axis=1).reshape(-1)
        keep = torch.from_numpy(half.astype(np.int64) >= 32768).to(DEV)
        assert torch.equal(x[b], torch.where(keep, row[0] * 2, torch.zeros_like(row[0])))


def test_head_i8_past_32_bits(H):
    """65,600 rows x 32,769 labels (more than 2^31 logits): the last rows equal
    those computed alone."""
    B, D, N = 65_600, 64, 32_769
    g = gen(42)
    Xq, xs = H.haste_quantize_rows(rand(g, (B, D), "bf16"))
    Wq, ws = H.haste_quantize_rows(rand(g, (N, D), "f32"))
    Z = torch.empty(B, N, dtype=torch.bfloat16, device=DEV)
    H.haste_head_fwd_i8(Xq, xs, Wq, ws, D, Z)
    for a, b in ((0, 3), (65_534, 65_537), (B - 3, B)):
        part = torch.empty(b - a, N, dtype=torch.bfloat16, device=DEV)
        H.haste_head_fwd_i8(Xq[a:b].contiguous(), xs[a:b].contiguous(), Wq, ws, D, part)
        assert torch.equal(Z[a:b], part)


# ---------------------------------------------------------------- refusals
def test_binding_refusals(H):
    x = torch.zeros(4, 16, device=DEV)
    with pytest.raises(ValueError):
        H.haste_norm_fwd(x.T)                                        # rows not dense
    with pytest.raises(ValueError):
        H.haste_norm_fwd(x[:1].expand(4, 16))                        # overlapping rows
    with pytest.raises(ValueError):
        H.haste_norm_fwd(x, torch.zeros(15, device=DEV))
    with pytest.raises(ValueError):
        H.haste_norm_fwd(x.cpu())
    with pytest.raises(TypeError):
        H.haste_norm_fwd(x.half())
    with pytest.raises(H.HasteError):
        H.haste_norm_fwd(x, y=x)                                     # in place
    with pytest.raises(H.HasteError):
        H.haste_dropout_apply(x, H.Dropout(1.5))
    with pytest.raises(H.HasteError):
        H.haste_dropout_apply(x, H.Dropout(float("nan")))
    with pytest.raises(ValueError):
        H.haste_logprob_fwd(None, None, None, torch.empty(4, device=DEV))
    with pytest.raises(ValueError):
        H.haste_logprob_fwd(x, x.bfloat16(), None, torch.empty(4, device=DEV))
    with pytest.raises(H.HasteError):
        H.haste_logprob_bwd(x, None, None, torch.empty(4, device=DEV), torch.empty_like(x))
    with pytest.raises(ValueError):
        H.haste_quantize_rows(x, torch.empty(4, 16, dtype=torch.int8, device=DEV))
    with pytest.raises(ValueError):
        H.haste_head_fwd_i8(torch.empty(4, 64, dtype=torch.int8, device=DEV), torch.ones(4, device=DEV),
                            torch.empty(5, 64, dtype=torch.int8, device=DEV), torch.ones(5, device=DEV), 65,
                            torch.empty(4, 5, device=DEV))
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    assert H.haste_logprob_workspace_bytes(x, None) <= ws.numel()
    r = H.lib().haste_logprob_fwd(H._logprob_desc(x, None), ctypes.c_void_p(x.data_ptr()), None, None, None,
                                  torch.empty(4, device=DEV).data_ptr(), None, ctypes.c_void_p(ws.data_ptr()), 8, None)
    assert r == H.HASTE_ERR_WORKSPACE
