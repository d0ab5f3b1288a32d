"""GPU checks of the operators around the layer where their kernels, chunks
or number formats change: the widths and row counts at which a row is cut
otherwise, and values and sizes at the ends of their ranges.  The references
are the definitions in 64 bits; the bounds are those that tests/test_gpu_ops.py
derives (u = 2^-24 a rounding, hardware exponential within (2 |v| + 4) 2^-23)."""
import numpy as np
import pytest
import torch

from oracle import ops
from tests._gpu import DEV, to_f64
from tests.test_gpu_ops import TT, gen, rounded, u, within

pytestmark = pytest.mark.gpu
f64 = torch.float64


@pytest.fixture(scope="module")
def H():
    from sparse_output_layer_amd import haste
    haste.lib()
    return haste


# -------------------------------------------------------- log probabilities
def _rows64(z):
    """lse, entropy and their bounds, in 64 bits on the device, of finite rows."""
    z = z.to(f64)
    m = z.amax(1)
    v = z - m[:, None]
    e = torch.exp(v)
    S = e.sum(1)
    p = e / S[:, None]
    del e
    ev, ev2 = -(p * v).sum(1), (p * v * (2 * v - 4)).sum(1) * 2.0 ** -23
    dS = 2.0 ** -23 * (4 + 2 * ev) + 320 * u + 64 * 5 * 2.0 ** -23
    lse = m + torch.log(S)
    dl = dS + 2 * u * lse.abs() + 8 * u
    dent = dS + ev2 + 2 * dS * ev + 4 * u * (torch.log(S) + ev)
    return lse, torch.log(S) + ev, dl, dent


def _check_rows(H, Zh, Z, K):
    """lse, entropy, the last label's log probability, the loss and the K best
    of one part's rows against the definition."""
    z = Z if Zh is None else Zh
    B, N = z.shape
    rp = torch.arange(B + 1, dtype=torch.int32, device=DEV)
    lab = torch.full((B,), N - 1, dtype=torch.int32, device=DEV)
    val, idx = torch.empty(B, K, device=DEV), torch.empty(B, K, dtype=torch.int32, device=DEV)
    given = H.Bce(rp, lab, grad_scale=1.0 / B, loss=torch.zeros(1, device=DEV), topk_val=val, topk_idx=idx)
    lse, ent, logp = (torch.full((B,), 9.0, device=DEV) for _ in range(3))
    H.haste_logprob_fwd(Zh, Z, given, lse, logp, ent)
    rl, re, dl, de = _rows64(z)
    within("lse", to_f64(lse), to_f64(rl), to_f64(dl))
    within("entropy", to_f64(ent), to_f64(re), to_f64(de))
    rp_ = z[:, -1].to(f64) - rl
    dp = dl + 4 * u * rp_.abs() + 2 * u * rl.abs()
    within("logp", to_f64(logp), to_f64(rp_), to_f64(dp))
    assert abs(given.loss.item() + rp_.mean().item()) <= dp.mean().item() + (B + 300) * u * rp_.abs().mean().item()
    order = torch.sort(z.to(f64), dim=1, descending=True, stable=True).indices[:, :K]
    assert torch.equal(idx.long(), order)
    rv = z.gather(1, order).to(f64) - rl[:, None]
    within("best", to_f64(val), to_f64(rv), to_f64(dl[:, None] + 4 * u * rv.abs() + 2 * u * rl.abs()[:, None]))


@pytest.mark.parametrize("N,dt", [(32761, "bf16"), (32762, "bf16"), (32768, "bf16"), (50001, "bf16"), (65529, "bf16"),
                                  (65530, "bf16"), (16381, "f32"), (16382, "f32"), (30000, "f32"), (32765, "f32"),
                                  (32766, "f32")])
def test_logprob_where_the_cut_changes(H, N, dt):
    """A single part on both sides of the widths at which its rows are one
    chunk or several, for numbers of rows at which the chunks' size changes.
    The largest logits and the given label end the row, so that nothing that
    is left out goes unseen; odd widths start rows at every place of a vector."""
    for B, shift, tail in ((511, 0, False), (512, 1, True), (513, 0, True), (1024, 3, False)):
        print(f"cut {B} x {N} {dt} shift {shift}", flush=True)
        base = (torch.randn(B * N + shift, generator=gen(N + B)) * 2.0).to(TT[dt]).to(DEV)
        z = base[shift:].view(B, N)
        z[:, -1], z[:, -2], z[:, N // 2], z[:, 0] = 16.0, 14.0, 15.0, 13.0
        z[3], z[4, ::2] = 0.25, 20.0          # all equal, and many equal largest ones
        _check_rows(H, None if tail else z, z if tail else None, 5)


@pytest.mark.parametrize("N", [2, 700, 20003, 90001])
def test_logprob_of_rows_far_from_zero(H, N):
    """The logits' differences count, not where they lie: rows of the same
    differences around 0 and up to 5 * 10^5 either way, in steps of 1/32 that
    fp32 holds there, in one batch of a thread and in several."""
    near = torch.randint(-160, 1, (N,), generator=gen(N)) / 32.0
    z = torch.stack([near + c for c in (0.0, 100.0, -1000.0, 5000.0, 60_000.0, -60_001.0, 250_000.0, 499_999.0, -500_000.0)])
    z[:, -1] += 7.0
    print("far from zero", N, flush=True)
    _check_rows(H, z.to(DEV), None, min(N, 5))


@pytest.mark.parametrize("N", [1, 700, 3000, 40003])
def test_logprob_around_a_million(H, N):
    """Rows whose logits lie on both sides of +-10^6, where the sums change
    their form: a largest one just above or at the bound and the others, in
    other threads, below it."""
    z = torch.empty(10, N)
    g = gen(N)
    near = torch.randint(0, 64, (N,), generator=g) / 16.0        # 0 to 4 in steps that fp32 holds at 2^20
    z[0] = -1e6 - 1.0 - near
    z[1] = -1e6 - 0.5
    z[2] = 1e6 - near
    z[3] = -1e6 + 2.0 - near
    z[4] = 1e6 + 2.0 - near
    z[5] = -1e6 - 0.25 - near
    z[6] = -999_872.0 - 64.0 * near
    z[7] = -1e6 - near
    z[8] = 1e6 - 1.0 - near
    z[9] = -2e6 - near
    z[:, N // 3] = torch.tensor([-1e6 + 0.5, -1e6, 1e6 + 0.5, -1e6 + 2.0, 1e6, -1e6 + 4.0, -999_871.0, -999_870.0, 1e6, -999_999.0])
    print("around a million", N, flush=True)
    _check_rows(H, z.to(DEV), None, min(N, 5))


@pytest.mark.parametrize("N,dt", [(40, "bf16"), (3000, "bf16"), (40003, "bf16"), (60001, "bf16"), (40, "f32"), (3000, "f32"),
                                  (40003, "f32")])
def test_logprob_signalling_nan(H, N, dt):
    """A NaN of either kind and sign makes the row's numbers NaN and is not
    listed itself; the best of the other logits are."""
    it, quiet, loud, sign = ((torch.int16, 0x7fc1, 0x7f81, -0x8000) if dt == "bf16" else
                             (torch.int32, 0x7fc00001, 0x7f800001, -0x80000000))
    z = torch.randn(8, N, generator=gen(N)).to(TT[dt])
    i = z.view(it)
    for r, bits in enumerate((quiet, loud, quiet + sign, loud + sign)):
        i[r, 7] = i[r, N - 1] = bits
        i[4 + r, r % 3::3] = bits
    ref = z.double()
    ref = torch.where(ref.isnan(), torch.full_like(ref, -float("inf")), ref)
    z = z.to(DEV)
    for K in (1, 5, 8):
        print("NaN", N, dt, K, flush=True)
        val, idx = torch.empty(8, K, device=DEV), torch.empty(8, K, dtype=torch.int32, device=DEV)
        given = H.Bce(torch.zeros(9, dtype=torch.int32, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV),
                      topk_val=val, topk_idx=idx)
        lse, ent = torch.empty(8, device=DEV), torch.empty(8, device=DEV)
        H.haste_logprob_fwd(z, None, given, lse, entropy=ent)
        assert lse.isnan().all() and ent.isnan().all() and val.isnan().all()
        assert torch.equal(idx.long().cpu(), torch.sort(ref, dim=1, descending=True, stable=True).indices[:, :K])


# --------------------------------------------------------------- layer norm
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [1, 3, 8, 9, 12, 24, 40, 72, 100, 130, 300, 513, 777, 1030, 2050, 3001, 4100, 8000, 8001, 9001])
def test_norm_bwd_of_a_large_mean(H, D, dt):
    """Rows of 2^121 with that mean and rstd 316: h is 0 for every element, though
    mean * rstd is past fp32.  The last row is an ordinary one."""
    B, big = 5, 2.0 ** 121
    g = gen(D)
    x = torch.full((B, D), big)
    x[B - 1] = torch.randn(D, generator=g)
    x = x.to(TT[dt]).to(DEV)
    dy, ga = (torch.randn(s, generator=g).to(DEV) for s in ((B, D), (D,)))
    mean, rstd = torch.full((B,), big, device=DEV), torch.full((B,), 316.0, device=DEV)
    mean[B - 1], rstd[B - 1] = 0.25, 1.5
    print("large mean", D, dt, flush=True)
    for rows in (B, 700):        # both forms of the weight gradient
        k = -(-rows // B)
        X, DY, m, r = (t.repeat(k, *(1,) * (t.dim() - 1))[:rows].contiguous() for t in (x, dy, mean, rstd))
        dg, db = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
        dx = H.haste_norm_bwd(X, ga, m, r, DY, None, dg, db)
        xx, gg, mm, rr = to_f64(X), to_f64(DY) * to_f64(ga), to_f64(m)[:, None], to_f64(r)[:, None]
        h = (xx - mm) * rr
        ref = rr * (gg - gg.mean(1, keepdims=True) - h * (gg * h).mean(1, keepdims=True))
        ag, ah = np.abs(gg), np.abs(h)
        bound = rr * (6 * u * ag + (D + 8) * u * ag.mean(1, keepdims=True) + ah * (D + 12) * u * (ag * ah).mean(1, keepdims=True))
        within("dx", to_f64(dx), ref, bound + rounded(dt, np.abs(ref) + bound))
        a = np.abs(to_f64(DY))
        within("dgamma", to_f64(dg), (to_f64(DY) * h).sum(0), (rows + 8) * u * (a * ah).sum(0) + 1e-37)
        within("dbeta", to_f64(db), to_f64(DY).sum(0), (rows + 4) * u * a.sum(0) + 1e-37)


# ------------------------------------------------- the widest rows there are
def test_rows_of_two_to_the_31_minus_1(H):
    """One row whose last vector of eight ends past 2^31 - 1: the mask of its
    first and last elements, and a constant row's mean and rstd (2^20 is exact in
    every sum; an element counted from past the end would add 2^9 to the variance)."""
    D = 2 ** 31 - 1
    x = torch.full((1, D), 2.0 ** 20, dtype=torch.bfloat16, device=DEV)
    print("widest dropout", flush=True)
    y = H.haste_dropout_apply(x, H.Dropout(0.5, 9, 4))
    for v in (0, 1, D // 16, D // 8 - 1, D // 8):
        w = ops.philox4x32(tuple(np.array([t]) for t in (v, 0, 4, 0)), (9, 0))
        half = np.array([int(t[0]) for word in w for t in (word & np.uint64(0xFFFF), word >> np.uint64(16))])
        want = np.where(half >= 32768, 2.0 ** 21, 0.0)[:min(8, D - 8 * v)]
        assert np.array_equal(to_f64(y[0, 8 * v:8 * v + 8]), want), v
    print("widest norm", flush=True)
    mean, rstd = torch.empty(1, device=DEV), torch.empty(1, device=DEV)
    H.haste_norm_fwd(x, y=y, mean=mean, rstd=rstd, eps=2.0 ** -20)
    assert mean.item() == 2.0 ** 20 and abs(rstd.item() - 1024.0) <= 8 * u * 1024.0
    assert not y.any()


# ----------------------------------------------------------------- refusals
def test_norm_bwd_into_the_gaps_of_x(H):
    """dx may be rows between x's in one allocation; rows that share an element
    with x's are refused."""
    B, D = 37, 24
    for dt in ("bf16", "f32"):
        buf = torch.randn(B, 3 * D, generator=gen(3)).to(TT[dt]).to(DEV)
        dy, mean, rstd = (torch.randn(s, generator=gen(4)).to(DEV).abs() for s in ((B, D), (B,), (B,)))
        for at, to in ((0, D), (D, 0), (2 * D, D), (0, 2 * D)):
            both = buf.clone()
            want = H.haste_norm_bwd(buf[:, at:at + D].contiguous(), None, mean, rstd, dy)
            H.haste_norm_bwd(both[:, at:at + D], None, mean, rstd, dy, both[:, to:to + D])
            assert torch.equal(both[:, to:to + D], want)
            rest = torch.ones(3 * D, dtype=torch.bool, device=DEV)
            rest[to:to + D] = False
            assert torch.equal(both[:, rest], buf[:, rest])
        for at, to in ((0, 0), (0, D - 1), (D, 1), (1, 0)):
            with pytest.raises(H.HasteError, match="overlaps"):
                H.haste_norm_bwd(buf[:, at:at + D], None, mean, rstd, dy, buf[:, to:to + D])
        # the last row's gap is past x's reach; other strides are refused by reach
        with pytest.raises(H.HasteError, match="overlaps"):
            H.haste_norm_bwd(buf[:, :D], None, mean, rstd, dy, buf.view(-1)[D:D + B * 2 * D].view(B, 2 * D)[:, :D])
