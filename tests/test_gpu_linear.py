"""GPU parity of the feature projections (product with bias, activation and
residual, and the gradients) against the fp64 oracle, through the C ABI.

Bounds: u = 2^-24 a rounding of fp32; a sum of k terms in any order is within
k u of the sum of their sizes; the hardware exponential of an argument t is
taken as within (2 |t| + 4) 2 u of it and the reciprocal as within 2 u, and
t itself has four roundings, so that a sigmoid s(t) is within
((1 - s) (12 |t| + 8) + 4) u of itself.  The activations' slopes are below
1.13.  dz is rounded to the operands' type before it is multiplied; every
result is rounded once more to its type."""
import numpy as np
import pytest
import torch

from oracle import features as ft
from tests._gpu import DEV, to_f64
from tests.test_gpu_ops import TINY, TT, gen, rand, rounded, strided, u, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H():
    from sparse_output_layer_amd import haste
    haste.lib()
    return haste


def act_code(H, name):
    return {"none": H.HASTE_ACT_NONE, "relu": H.HASTE_ACT_RELU, "gelu": H.HASTE_ACT_GELU, "silu": H.HASTE_ACT_SILU}[name]


def sigmoid_bounds(name, z):
    """Of the activation and of its slope, at z known exactly."""
    if name in ("none", "relu"):
        return np.zeros_like(z), np.zeros_like(z)
    c = 2.0 * np.sqrt(2.0 / np.pi)
    t, dt = (z, np.ones_like(z)) if name == "silu" else (c * (z + 0.044715 * z ** 3), c * (1.0 + 3 * 0.044715 * z ** 2))
    t = np.minimum(np.abs(t), 200.0) * np.sign(t)
    s = 0.5 * (1.0 + np.tanh(0.5 * t))
    s = np.where(t < -30, np.exp(t), s)
    es = s * ((1 - s) * (12 * np.abs(t) + 8) + 4) * u
    d = np.where(np.abs(t) > 30, np.exp(-np.abs(t)), s * (1 - s))
    ed = d * (12 * np.abs(t) + 20) * u
    return np.abs(z) * (es + 4 * u * s), es + np.abs(z * dt) * (ed + 8 * u * d) + 4 * u


CASES = [  # M, K, N, x, y, activation, bias type, residual, z, row stride beyond K
    (1, 1, 1, "f32", "f32", "none", None, 0, 0, 0), (1, 1024, 1024, "bf16", "bf16", "silu", "f32", 1, 1, 0),
    (16, 77, 35, "bf16", "f32", "gelu", "bf16", 1, 1, 3), (5, 1001, 130, "f32", "f32", "relu", "f32", 1, 0, 0),
    (17, 64, 64, "bf16", "bf16", "gelu", "f32", 0, 1, 0), (33, 40, 24, "f32", "f32", "silu", "bf16", 1, 1, 4),
    (100, 72, 200, "bf16", "f32", "none", "f32", 1, 0, 8), (130, 768, 136, "bf16", "bf16", "relu", None, 0, 1, 0),
    (200, 33, 77, "bf16", "bf16", "gelu", "f32", 1, 1, 0), (65, 129, 66, "f32", "f32", "gelu", "f32", 0, 1, 0),
    (512, 768, 1024, "bf16", "bf16", "gelu", "f32", 1, 1, 768), (1025, 104, 1999, "bf16", "bf16", "silu", "bf16", 1, 1, 0),
    (1500, 100, 2052, "f32", "f32", "silu", "f32", 1, 1, 0), (4100, 72, 4040, "bf16", "bf16", "gelu", "f32", 1, 1, 0),
    (4001, 57, 4099, "bf16", "f32", "relu", "f32", 0, 1, 7), (777, 1001, 513, "f32", "f32", "gelu", "f32", 0, 1, 0),
    (2, 5000, 33, "bf16", "bf16", "none", "bf16", 1, 0, 0), (3000, 8, 16, "bf16", "bf16", "silu", "f32", 0, 1, 0),
    (70, 2050, 5, "bf16", "bf16", "gelu", "f32", 1, 1, 0)]


class Case:
    def __init__(self, case):
        print(f"linear {case}", flush=True)
        (self.M, self.K, self.N, self.xt, self.yt, self.act, bt, res, self.keep, gap) = case
        M, K, N = self.M, self.K, self.N
        g = self.g = gen(M + K + N)
        self.x = rand(g, (M, K), self.xt)
        if gap:
            self.x = strided(self.x, K + gap)
        self.W = rand(g, (N, K), self.xt, 1.5 * K ** -0.5)
        self.b = None if bt is None else rand(g, (N,), bt, 0.5)
        self.res = rand(g, (M, N), self.yt) if res else None
        self.x64, self.W64 = to_f64(self.x), to_f64(self.W)


@pytest.mark.parametrize("case", CASES)
def test_linear_fwd(H, case):
    c = Case(case)
    b, res = (None if t is None else to_f64(t) for t in (c.b, c.res))
    y = torch.full((c.M, c.N), 9.0, dtype=TT[c.yt], device=DEV)
    z = torch.full_like(y, 9.0) if c.keep and c.act != "none" else None
    kw = dict(bias=c.b, act=act_code(H, c.act), residual=c.res)
    H.haste_linear_fwd(c.x, c.W, y, z=z, **kw)
    ry, rz = ft.linear_fwd(c.x64, c.W64, b, c.act, res)
    ez = (c.K + 4) * u * (np.abs(c.x64) @ np.abs(c.W64).T + (0 if b is None else np.abs(b)))
    if z is not None:
        within("z", to_f64(z), rz, ez + rounded(c.yt, np.abs(rz) + ez))
    e = 1.13 * ez + sigmoid_bounds(c.act, rz)[0] + (0 if res is None else u * (np.abs(res) + np.abs(ry))) + TINY
    within("y", to_f64(y), ry, e + rounded(c.yt, np.abs(ry) + e))
    again = H.haste_linear_fwd(c.x, c.W, torch.empty_like(y), **kw)
    assert torch.equal(again, y)
    if res is not None:      # into the residual
        r = c.res.clone()
        H.haste_linear_fwd(c.x, c.W, r, bias=c.b, act=kw["act"], residual=r)
        assert torch.equal(r, y)


@pytest.mark.parametrize("case", CASES)
def test_linear_bwd(H, case):
    c = Case(case)
    M, K, N = c.M, c.K, c.N
    dy = rand(c.g, (M, N), c.yt)
    z = rand(c.g, (M, N), c.yt, 2.0) if c.act != "none" else None
    add = rand(c.g, (M, K), c.xt) if c.res is not None else None
    dx = torch.full((M, K), 7.0, dtype=TT[c.xt], device=DEV)
    if c.x.stride(0) != K and M > 1:
        dx = strided(dx, K + 5)
    dW, db = torch.full_like(c.W, 7.0), torch.full((N,), 7.0, device=DEV)
    kw = dict(act=act_code(H, c.act), z=z)
    H.haste_linear_bwd(c.x, c.W, dy, dx=dx, dW=dW, dbias=db, dx_add=add, **kw)
    z64 = np.zeros((M, N)) if z is None else to_f64(z)
    a64 = None if add is None else to_f64(add)
    rdx, rdw, rdb, rdz = ft.linear_bwd(c.x64, c.W64, to_f64(dy), z64, c.act, a64)
    e0 = np.abs(to_f64(dy)) * sigmoid_bounds(c.act, z64)[1] + 2 * u * np.abs(rdz)
    direct = z is None and c.xt == c.yt
    ez = e0 if direct else e0 + rounded(c.xt, np.abs(rdz) + e0)
    bx = ez @ np.abs(c.W64) + (N + 4) * u * (np.abs(rdz) @ np.abs(c.W64)) + (0 if add is None else u * (np.abs(a64) + np.abs(rdx)))
    within("dx", to_f64(dx), rdx, bx + rounded(c.xt, np.abs(rdx) + bx))
    bw = ez.T @ np.abs(c.x64) + (M + 8) * u * (np.abs(rdz).T @ np.abs(c.x64))
    within("dW", to_f64(dW), rdw, bw + rounded(c.xt, np.abs(rdw) + bw))
    bb = e0.sum(0) + (M + 8) * u * np.abs(rdz).sum(0)
    within("db", to_f64(db), rdb, bb + u * np.abs(rdb) + TINY)
    if dx.stride(0) != K and M > 1:
        assert torch.isnan(dx.as_strided((M - 1, 5), (K + 5, 1), dx.storage_offset() + K)).all()
    # each alone, the same bits; dx over its addend; added to
    one = torch.empty(M, K, dtype=TT[c.xt], device=DEV) if add is None else add.clone()
    H.haste_linear_bwd(c.x, c.W, dy, dx=one, dx_add=None if add is None else one, **kw)
    assert torch.equal(one, dx)
    one = torch.empty_like(dW)
    H.haste_linear_bwd(c.x, c.W, dy, dW=one, **kw)
    assert torch.equal(one, dW)
    one = torch.full_like(db, 3.0)
    H.haste_linear_bwd(c.x, c.W, dy, dbias=one, accumulate_dw=True, **kw)
    assert torch.equal(one, db + 3.0)
    base = rand(c.g, (N, K), c.xt, float(M) ** 0.5)
    got = base.clone()
    H.haste_linear_bwd(c.x, c.W, dy, dW=got, accumulate_dw=True, **kw)
    want = rdw + to_f64(base)
    ba = bw + 2 * u * (np.abs(rdw) + np.abs(to_f64(base)))
    within("dW added", to_f64(got), want, ba + rounded(c.xt, np.abs(want) + ba))


def ints(g, shape, dt, most):
    return torch.randint(-most, most + 1, shape, generator=g).to(TT[dt]).to(DEV)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,K,N", [(16, 31, 17), (64, 32, 64), (65, 33, 63), (128, 96, 128), (129, 128, 257), (640, 160, 2304),
                                   (1000, 136, 3001), (2048, 40, 8192), (5000, 264, 4352), (40000, 48, 24), (30, 20, 40000),
                                   (9000, 520, 100), (255, 8, 255)])
def test_linear_integers(H, M, K, N, dt):
    """Small integers: every product and sum is exact, whatever the tile, the
    sizes and the split, so that each element is equal."""
    print(f"integers {M} {K} {N} {dt}", flush=True)
    g = gen(M + N)
    x, W = ints(g, (M, K), dt, 3), ints(g, (N, K), dt, 3)
    y = torch.empty(M, N, device=DEV)
    H.haste_linear_fwd(x, W, y)
    assert torch.equal(y.double(), x.double() @ W.double().T)
    dy = ints(g, (M, N), dt, 1)
    dx, dW, db = torch.empty_like(x), torch.empty_like(W), torch.empty(N, device=DEV)
    H.haste_linear_bwd(x, W, dy, dx=dx, dW=dW, dbias=db)
    assert torch.equal(dx, (dy.double() @ W.double()).to(TT[dt]))
    assert torch.equal(dW, (dy.double().T.contiguous() @ x.double()).to(TT[dt]))
    assert torch.equal(db.double(), dy.double().sum(0))


@pytest.mark.parametrize("K", [1, 2, 4, 7, 8, 9, 12, 31, 32, 33, 63, 64, 65, 100, 127, 130, 255, 257])
def test_linear_contraction_ends(H, K):
    """Contractions that end at every place of a step, for every tile, with NaN
    behind the rows: what is past the end is not multiplied."""
    for dt in ("bf16", "f32"):
        for M, N in ((9, 70), (70, 130), (1500, 2050), (4100, 4100)):
            g = gen(K)
            x, W = strided(ints(g, (M, K), dt, 3), K + 4 + -K % 4), ints(g, (N, K), dt, 3)
            y = torch.empty(M, N, device=DEV)
            H.haste_linear_fwd(x, W, y)
            assert torch.equal(y.double(), x.double() @ W.double().T), (dt, M, N)
            dx, dW = torch.empty(N, K, dtype=TT[dt], device=DEV), torch.empty(M, K, dtype=TT[dt], device=DEV)
            dy = ints(g, (N, M), dt, 1)      # here W's rows are the batch: the contraction M ends anywhere
            H.haste_linear_bwd(W, x.contiguous(), dy, dx=dx, dW=dW)
            assert torch.equal(dx, (dy.double() @ x.double()).to(TT[dt])) and torch.equal(
                dW, (dy.double().T.contiguous() @ W.double()).to(TT[dt]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("w", [1, 2, 3, 4, 5])
def test_linear_narrow_results(H, w, dt):
    """Results of fewer columns than a lane's run, with what is added to them:
    small integers, every result exact; rows of a residual follow each other."""
    print(f"narrow {w} {dt}", flush=True)
    g = gen(w)
    for M, K in ((33, 40), (700, 24)):
        x, W = ints(g, (M, K), dt, 3), ints(g, (w, K), dt, 3)
        r = ints(g, (M, w), dt, 9)
        want = (x.double() @ W.double().T + r.double()).to(TT[dt])
        assert torch.equal(H.haste_linear_fwd(x, W, torch.empty_like(r), residual=r), want)
        if w > 1:
            with pytest.raises(ValueError, match="residual must be contiguous"):
                H.haste_linear_fwd(x, W, torch.empty_like(r), residual=strided(r, w + 3))
        # the batch of w columns: dx with its addend, dW onto what is there
        v, U = ints(g, (M, w), dt, 3), ints(g, (K, w), dt, 3)
        dy, add, base = ints(g, (M, K), dt, 1), ints(g, (M, w), dt, 9), ints(g, (K, w), dt, 9)
        dx, dW = torch.empty_like(v), base.clone()
        H.haste_linear_bwd(v, U, dy, dx=dx, dW=dW, dx_add=add, accumulate_dw=True)
        assert torch.equal(dx, (dy.double() @ U.double() + add.double()).to(TT[dt]))
        assert torch.equal(dW, (dy.double().T.contiguous() @ v.double() + base.double()).to(TT[dt]))


@pytest.mark.parametrize("n", [200, 1500])
def test_linear_long_sums(H, n):
    """fp32: 2^25 and, from the 257th on, ones: added to it one or two at a time
    they are lost (the spacing there is 4), the sums of runs of 256 are not."""
    K = 4096
    v = torch.ones(n, K, device=DEV)
    v[:, 0], v[:, 1:256] = 2.0 ** 25, 0.0
    one, want = torch.ones(n, K, device=DEV), 2.0 ** 25 + K - 256
    assert (H.haste_linear_fwd(v, one) == want).all()
    dx = torch.empty(n, n, device=DEV)
    H.haste_linear_bwd(torch.zeros(n, n, device=DEV), torch.ones(K, n, device=DEV), v, dx=dx)
    assert (dx == want).all()
    dW = torch.empty(n, n, device=DEV)
    H.haste_linear_bwd(torch.ones(K, n, device=DEV), torch.zeros(n, n, device=DEV), v.T.contiguous(), dW=dW)
    assert (dW == want).all()


@pytest.mark.parametrize("M", [15, 16, 17, 31, 32, 33])
def test_linear_rows_without_tiles(H, M):
    """Both sides of the numbers of rows where the way changes, against 64 bits,
    with everything the epilogue has."""
    for K, N, xt, yt, act in ((1001, 130, "bf16", "f32", "gelu"), (257, 65, "f32", "f32", "silu"), (64, 19, "bf16", "bf16", "relu")):
        test_linear_fwd(H, (M, K, N, xt, yt, act, "f32", 1, 1, 5))


def test_linear_unaligned(H):
    """Bases of every tensor off the vector alignment, few rows and many."""
    def shift(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
        return b.copy_(t.reshape(-1)).view(t.shape)
    for M in (3, 150):
        for dt in ("bf16", "f32"):
            g = gen(M)
            x, W, b, r, dy, z = (rand(g, s, dt) for s in ((M, 64), (96, 64), (96,), (M, 96), (M, 96), (M, 96)))
            a, az = torch.empty_like(r), torch.empty_like(r)
            H.haste_linear_fwd(x, W, a, b, H.HASTE_ACT_GELU, r, az)
            c, cz = shift(a), shift(az)
            H.haste_linear_fwd(shift(x), shift(W), c.zero_(), shift(b), H.HASTE_ACT_GELU, shift(r), cz.zero_())
            assert torch.equal(a, c) and torch.equal(az, cz)
            o = [torch.empty_like(x), torch.empty_like(W), torch.empty(96, device=DEV)]
            H.haste_linear_bwd(x, W, dy, H.HASTE_ACT_SILU, z, *o, dx_add=x)
            p = [shift(t) for t in o]
            H.haste_linear_bwd(shift(x), shift(W), shift(dy), H.HASTE_ACT_SILU, shift(z), *p, dx_add=shift(x))
            assert all(torch.equal(i, j) for i, j in zip(o, p))


def test_linear_nan_and_infinity(H):
    """A NaN in a row of x stays in the row, one in a row of W in its column;
    large arguments reach the activations' limits."""
    for M in (12, 300):
        x, W = rand(gen(1), (M, 72), "bf16"), rand(gen(2), (40, 72), "bf16")
        x[3, 71], W[5, 70] = float("nan"), float("inf")
        y = to_f64(H.haste_linear_fwd(x, W, act=H.HASTE_ACT_GELU))
        bad = np.zeros((M, 40), bool)
        bad[3] = True
        assert np.isnan(y[3]).all() and np.isfinite(np.delete(np.delete(y, 3, 0), 5, 1)).all()
    z = torch.tensor([[-1e30, -1e4, -100.0, -20.0, 0.0, 20.0, 100.0, 1e4, 1e30]], device=DEV)
    one = torch.eye(9, device=DEV)
    for name in ("gelu", "silu", "relu"):
        y = H.haste_linear_fwd(z, one, act=act_code(H, name))
        assert torch.equal(y[0, 4:], z[0, 4:]) or torch.allclose(y[0, 4:], z[0, 4:], rtol=1e-6)
        assert (y[0, :3].abs() <= 1e-30).all()
        db = torch.empty(9, device=DEV)
        H.haste_linear_bwd(z, one, torch.ones_like(z), act_code(H, name), z, dbias=db)
        want = ft.act(name, to_f64(z))[1][0]
        want[[0, 8]] = 0.0, 1.0
        assert np.allclose(to_f64(db), want, atol=1e-6)


def test_linear_gradient_by_differences(H):
    r = np.random.default_rng(5)
    M, K, N = 7, 19, 23
    t = lambda *s: torch.from_numpy(r.standard_normal(s).astype(np.float32)).to(DEV)  # noqa: E731
    x, W, b, dy, res = t(M, K), t(N, K), t(N), t(M, N), t(M, N)
    for name in ft.ACTS:
        z = torch.empty(M, N, device=DEV) if name != "none" else None
        H.haste_linear_fwd(x, W, torch.empty(M, N, device=DEV), b, act_code(H, name), res, z)
        dx, dW, db = torch.empty_like(x), torch.empty_like(W), torch.empty(N, device=DEV)
        H.haste_linear_bwd(x, W, dy, act_code(H, name), z, dx, dW, db)
        at, got = [to_f64(v) for v in (x, W, b)], [to_f64(v) for v in (dx, dW, db)]
        f = lambda a: float((ft.linear_fwd(*a, name)[0] * to_f64(dy)).sum())  # noqa: E731
        for _ in range(3):
            v = [r.standard_normal(a.shape) for a in at]
            h = 1e-7 if name == "relu" else 1e-5
            want = (f([a + h * d for a, d in zip(at, v)]) - f([a - h * d for a, d in zip(at, v)])) / (2 * h)
            have, size = (sum(float(k((a * d)).sum()) for a, d in zip(got, v)) for k in (lambda q: q, np.abs))
            assert abs(have - want) <= 400 * u * size + 1e-6 * size, name


def test_linear_past_32_bits(H):
    """Results of more than 2^31 elements, and x of more."""
    M, K, N = 270_000, 16, 8200
    x, W = ints(gen(1), (M, K), "bf16", 3), ints(gen(2), (N, K), "bf16", 3)
    y = H.haste_linear_fwd(x, W)
    for rows in (slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)):
        assert torch.equal(y[rows], (x[rows].double() @ W.double().T).bfloat16())
    dx = H.haste_linear_fwd(y[:, :16], W)        # strided rows far apart
    assert torch.equal(dx[-300:], H.haste_linear_fwd(y[-300:, :16].contiguous(), W))
    del dx
    y.clamp_(-1, 1)
    dW, db, dx = torch.empty_like(W), torch.empty(N, device=DEV), torch.empty_like(x)
    H.haste_linear_bwd(x, W, y, dW=dW, dbias=db, dx=dx)
    assert torch.equal(dx[-300:], (y[-300:].double() @ W.double()).bfloat16())
    want = sum(y[i:i + 30_000].double().T.contiguous() @ x[i:i + 30_000].double() for i in range(0, M, 30_000))
    assert torch.equal(dW, want.bfloat16())
    assert torch.equal(db.double(), sum(y[i:i + 30_000].double().sum(0) for i in range(0, M, 30_000)))


def test_linear_most_rows(H):
    """2^31 - 1 rows: the last tile ends where 32 bits do."""
    M, K, N = 2 ** 31 - 1, 8, 8
    g = gen(3)
    x, W, b = torch.zeros(M, K, dtype=torch.bfloat16, device=DEV), ints(g, (N, K), "bf16", 3), ints(g, (N,), "f32", 9)
    ends = [slice(0, 300), slice(M // 2, M // 2 + 300), slice(M - 300, M)]
    for e in ends:
        x[e] = ints(g, (300, K), "bf16", 3)
    y = H.haste_linear_fwd(x, W, bias=b)
    for e in ends:
        assert torch.equal(y[e], (x[e].double() @ W.double().T + b.double()).bfloat16())
    assert (y[M // 3:M // 3 + 100_000] == b).all() and (y[-100_000:-300] == b).all()
    y.zero_()
    for e in ends:
        y[e] = ints(g, (300, N), "bf16", 1)
    dx, dW, db = torch.ones_like(x), torch.empty_like(W), torch.empty(N, device=DEV)
    H.haste_linear_bwd(x, W, y, dx=dx, dW=dW, dbias=db)
    for e in ends:
        assert torch.equal(dx[e], (y[e].double() @ W.double()).bfloat16())
    assert not dx[M // 3:M // 3 + 100_000].any() and not dx[-100_000:-300].any()
    assert torch.equal(dW, sum(y[e].double().T.contiguous() @ x[e].double() for e in ends).bfloat16())
    assert torch.equal(db.double(), sum(y[e].double().sum(0) for e in ends))


def test_linear_captured(H):
    M, K, N = 700, 136, 264
    g = gen(1)
    x, W, b, r, dy = (rand(g, s, "bf16") for s in ((M, K), (N, K), (N,), (M, N), (M, N)))
    out = [torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2)] + [torch.empty_like(x), torch.empty_like(W), torch.empty(N, device=DEV)]
    ws = torch.empty(H.haste_linear_bwd_workspace_bytes(x, W, dy, H.HASTE_ACT_GELU), dtype=torch.uint8, device=DEV)

    def go(y, z, dx, dW, db, ws):
        H.haste_linear_fwd(x, W, y, b, H.HASTE_ACT_GELU, r, z)
        H.haste_linear_bwd(x, W, dy, H.HASTE_ACT_GELU, z, dx, dW, db, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(*out, ws)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(*out, ws)
    for i in range(4):
        x.copy_(rand(gen(i), (M, K), "bf16"))
        graph.replay()
        want = [torch.empty_like(t) for t in out]
        go(*want, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want)), i
