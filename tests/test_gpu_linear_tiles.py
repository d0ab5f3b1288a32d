"""Every tile of the feature projections' product, with results that end with a
tile and results that end inside one, with everything the epilogue has and with
nothing, against products in 64 bits on the device; and what a NaN and an
infinity reach.

Small integers are exact through every product, sum and split, so that the
results are equal; for the activations with an exponential the bounds are those
of test_gpu_linear.py."""
import math

import pytest
import torch

from tests._gpu import DEV
from tests.test_gpu_ops import TINY, TT, u

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H():
    from sparse_output_layer_amd import haste
    haste.lib()
    return haste


def seeded(s):
    g = torch.Generator(device=DEV)
    g.manual_seed(s)
    return g


def ints(g, shape, dt, most):
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV).to(TT[dt])


def normal(g, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(TT[dt])


def half_step(dt, v):
    return torch.ldexp(torch.full_like(v, 0.5), torch.frexp(v)[1] - (8 if dt == "bf16" else 24)) + TINY


def act64(name, z):
    """The activation, and how far the kernel's may be from it at z known exactly."""
    t = z if name == "silu" else 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)
    s = torch.sigmoid(t)
    es = s * ((1 - s) * (12 * t.abs().clamp(max=200.0) + 8) + 4) * u
    return z * s, z.abs() * (es + 4 * u * s)


def close(name, got, ref, bound):
    err = (got.double() - ref).abs()
    assert (err <= bound).all(), (name, float((err / bound).max()))


# rows and columns of results, whole tiles and ragged ones
TILES = {("bf16", 256): [(3584, 3584), (3500, 3700)], ("bf16", 128): [(1536, 1536), (1500, 1601)],
         ("bf16", 64): [(192, 320), (190, 301)],
         ("f32", 128): [(1792, 1792), (1750, 1901)], ("f32", 64): [(192, 320), (190, 301)]}


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("xt,tile,yt", [(x, t, y) for x, t in TILES for y in (("bf16", "f32") if x == "bf16" else ("f32",))])
def test_linear_fwd_tiles(H, xt, tile, yt, act):
    print(f"tiles {xt} {tile} {yt} {act}", flush=True)
    exact = act in ("none", "relu")
    code = {"none": H.HASTE_ACT_NONE, "relu": H.HASTE_ACT_RELU, "gelu": H.HASTE_ACT_GELU, "silu": H.HASTE_ACT_SILU}[act]
    for M, N in TILES[xt, tile]:
        for K, full in ((136, True), (77, False), (77, True)):
            g = seeded(M + K)
            if exact:
                x, W, b, res = ints(g, (M, K), xt, 3), ints(g, (N, K), xt, 3), ints(g, (N,), "f32", 9), ints(g, (M, N), yt, 9)
            else:
                x, W, b, res = (normal(g, (M, K), xt), normal(g, (N, K), xt, 1.5 * K ** -0.5), normal(g, (N,), "f32", 0.5),
                                normal(g, (M, N), yt))
            y = torch.full((M, N), 9.0, dtype=TT[yt], device=DEV)
            z = torch.full_like(y, 9.0) if full and act != "none" else None
            H.haste_linear_fwd(x, W, y, bias=b if full else None, act=code, residual=res if full else None, z=z)
            x, W = x.double(), W.double()
            rz = x @ W.T + (b.double() if full else 0.0)
            if exact:
                if z is not None:
                    assert torch.equal(z, rz.to(TT[yt])), (M, N, K)
                ry = rz.clamp(min=0) if act == "relu" else rz
                assert torch.equal(y, (ry + (res.double() if full else 0.0)).to(TT[yt])), (M, N, K)
                continue
            ez = (K + 4) * u * (x.abs() @ W.abs().T + (b.double().abs() if full else 0.0))
            if z is not None:
                close("z", z, rz, ez + half_step(yt, rz.abs() + ez))
            ry, ea = act64(act, rz)
            e = 1.13 * ez + ea + TINY
            if full:
                ry = ry + res.double()
                e = e + u * (res.double().abs() + ry.abs())
            close("y", y, ry, e + half_step(yt, ry.abs() + e))


# batch, K, N of dx = dz W (batch x K) and dW = dz^T x (N x K): every tile of
# both, weight gradients in one run and in several
BACK = {"bf16": [(3584, 3584, 72), (3500, 3700, 77), (1536, 1536, 136), (1500, 1601, 40), (192, 320, 200), (190, 301, 77),
                 (300, 3584, 3584), (301, 3700, 3500), (600, 1536, 1536), (601, 1601, 1500),
                 (45056, 768, 1024), (45001, 777, 1000), (8192, 1024, 1024), (8191, 1001, 1023), (2560, 128, 128), (2500, 130, 131)],
        "f32": [(1792, 1792, 72), (1750, 1901, 77), (192, 320, 200), (190, 301, 77), (300, 1792, 1792), (301, 1901, 1750),
                (2048, 128, 128), (2001, 130, 131)]}


@pytest.mark.parametrize("dt,B,K,N", [(dt, *c) for dt in BACK for c in BACK[dt]])
def test_linear_bwd_tiles(H, dt, B, K, N):
    print(f"backward tiles {dt} {B} {K} {N}", flush=True)
    g = seeded(B + K + N)
    x, W, dy, z = ints(g, (B, K), dt, 2), ints(g, (N, K), dt, 3), ints(g, (B, N), dt, 1), ints(g, (B, N), dt, 2)
    add, base = ints(g, (B, K), dt, 9), ints(g, (N, K), dt, 9)
    for act in (H.HASTE_ACT_NONE, H.HASTE_ACT_RELU):
        dz = dy.double() * (z > 0) if act else dy.double()
        rx, rw = dz @ W.double(), dz.T.contiguous() @ x.double()
        dx, dW, db = torch.empty_like(x), torch.empty_like(W), torch.empty(N, device=DEV)
        H.haste_linear_bwd(x, W, dy, act, z if act else None, dx, dW, db)
        assert torch.equal(dx, rx.to(TT[dt])) and torch.equal(dW, rw.to(TT[dt])) and torch.equal(db.double(), dz.sum(0))
        dx, dW = add.clone(), base.clone()
        H.haste_linear_bwd(x, W, dy, act, z if act else None, dx, dW, dx_add=dx, accumulate_dw=True)
        assert torch.equal(dx, (rx + add.double()).to(TT[dt])) and torch.equal(dW, (rw + base.double()).to(TT[dt]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(12, 40, 72), (300, 40, 71), (1600, 1601, 72), (3500, 3700, 77)])
def test_linear_reach_of_nan_and_infinity(H, M, N, K, dt):
    """A NaN in x makes its row, an infinity in W's last used place its column:
    what the formulas give there, finite everywhere else."""
    print(f"reach {M} {N} {K} {dt}", flush=True)
    g = seeded(K)
    x, W = normal(g, (M, K), dt), normal(g, (N, K), dt, K ** -0.5)
    x[x == 0] = 1.0
    x[3, K - 1], W[5, K - 1], W[7, 0] = float("nan"), float("inf"), -float("inf")
    row = torch.arange(M, device=DEV) != 3
    col = torch.ones(N, dtype=torch.bool, device=DEV)
    col[[5, 7]] = False
    inf = float("inf")
    for act, neg in ((H.HASTE_ACT_NONE, -inf), (H.HASTE_ACT_RELU, 0.0), (H.HASTE_ACT_GELU, float("nan")), (H.HASTE_ACT_SILU, float("nan"))):
        y = H.haste_linear_fwd(x, W, act=act)
        assert torch.isnan(y[3]).all() and torch.isfinite(y[row][:, col]).all()
        for c, up in ((5, x[:, K - 1] > 0), (7, x[:, 0] < 0)):
            got, up = y[row, c], up[row]
            assert (got[up] == inf).all()
            assert (torch.isnan(got[~up]) if neg != neg else got[~up] == neg).all()
    # backward: a NaN of dy in its row of dx and its column of dW, an infinity of x in its column of dW
    dy = normal(g, (M, N), dt)
    dy[2, N - 1] = float("nan")
    x = normal(g, (M, K), dt)
    x[M - 1, 4] = inf
    W = normal(g, (N, K), dt)
    dx, dW, db = torch.empty_like(x), torch.empty_like(W), torch.empty(N, device=DEV)
    H.haste_linear_bwd(x, W, dy, dx=dx, dW=dW, dbias=db)
    assert torch.isnan(dx[2]).all() and torch.isfinite(dx[torch.arange(M, device=DEV) != 2]).all()
    assert torch.isnan(dW[N - 1]).all() and torch.isnan(db[N - 1]) and torch.isfinite(db[:-1]).all()
    assert torch.isinf(dW[:-1, 4]).all() and (dW[:-1, 4] * dy[M - 1, :-1] > 0).all()
    assert torch.isfinite(dW[:-1][:, torch.arange(K, device=DEV) != 4]).all()
