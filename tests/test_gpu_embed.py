"""GPU parity of the embedding (bags, lookup, gradients by sorted tokens)
against the fp64 oracle, through the C ABI.

Bounds: u = 2^-24 a rounding; a sum of k terms in any order is within k u of
the sum of their sizes, a term has two roundings (scale times weight, and the
product is fused), and the result is rounded once more to its type."""
import numpy as np
import pytest
import torch

from oracle import features as ft
from tests._gpu import DEV, to_f64
from tests.test_gpu_ops import TT, gen, rand, rounded, u, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H():
    from sparse_output_layer_amd import haste
    haste.lib()
    return haste


def make(B, n, V, bags, seed=0, skew=False, outside=0.05):
    """tokens (some outside the table), row_ptr (rows of all lengths, empty ones among them)."""
    r = np.random.default_rng(seed + n + V)
    tok = np.minimum((V + 1) ** r.random(n) - 1, V - 1).astype(np.int64) if skew else r.integers(0, V, n)
    out = r.random(n) < outside
    tok[out] = r.choice([-1, -2 ** 31, V, V + 5 if V < 2 ** 31 - 9 else V, 2 ** 31 - 1], out.sum())
    rp = None
    if bags:
        cut = np.sort(r.choice(np.concatenate([[0, n], r.integers(0, n + 1, 8)]), B - 1)) if skew else np.sort(r.integers(0, n + 1, B - 1))
        rp = np.concatenate([[0], cut, [n]]).astype(np.int32)
    return tok.astype(np.int32), rp, r.normal(0.5, 1.0, n).astype(np.float32)


def dev(a):
    return None if a is None else torch.from_numpy(a).to(DEV)


CASES = [  # B, n, V, D, bags, weighted, table, y, gradient, skewed
    (1, 1, 1, 1, 0, 0, "f32", "f32", "f32", 0), (1, 24, 500, 768, 1, 1, "bf16", "bf16", "f32", 0),
    (4, 0, 5, 9, 1, 0, "bf16", "f32", "bf16", 0), (1, 3000, 40, 33, 1, 1, "f32", "bf16", "bf16", 0),
    (600, 512, 700, 96, 1, 0, "bf16", "f32", "f32", 0), (600, 513, 700, 96, 1, 1, "bf16", "f32", "f32", 0),
    (77, 5000, 1000, 768, 1, 1, "f32", "f32", "f32", 1), (300, 4999, 65, 1001, 1, 1, "bf16", "bf16", "f32", 1),
    (2000, 1500, 3000, 40, 1, 0, "f32", "bf16", "f32", 1), (777, 777, 100, 1024, 0, 1, "bf16", "bf16", "f32", 1),
    (4097, 4097, 4, 64, 0, 0, "bf16", "bf16", "bf16", 0), (5000, 5000, 1, 130, 0, 0, "f32", "f32", "f32", 0),
    (33, 2049, 1 << 20, 7, 1, 1, "f32", "f32", "f32", 0), (64, 8200, 1500, 2500, 1, 0, "bf16", "f32", "bf16", 1),
    (512, 512, 2000, 520, 0, 1, "f32", "bf16", "f32", 1), (3, 1025, 1023, 4, 1, 1, "bf16", "bf16", "bf16", 0),
    (9, 1100, 1024, 250, 1, 1, "f32", "f32", "bf16", 0)]


@pytest.mark.parametrize("case", CASES)
def test_embed_fwd(H, case):
    B, n, V, D, bags, weighted, et, yt, gt, skew = case
    print(f"embed fwd {case}", flush=True)
    tok, rp, w = make(B, n, V, bags, skew=skew)
    w = w if weighted else None
    E = rand(gen(D), (V, D), et)
    y = torch.full((B, D), 9.0, dtype=TT[yt], device=DEV)
    H.haste_embed_fwd(dev(tok), E, y, dev(rp), dev(w), 1.5)
    ref, size = ft.embed_fwd(tok, to_f64(E), B, rp, w, 1.5)
    most = 1 if rp is None else int(np.diff(rp).max())
    bound = (most + 4) * u * size
    within("y", to_f64(y), ref, bound + rounded(yt, np.abs(ref) + bound))
    again = H.haste_embed_fwd(dev(tok), E, torch.empty_like(y), dev(rp), dev(w), 1.5)
    assert torch.equal(again, y)


@pytest.mark.parametrize("case", CASES)
def test_embed_bwd(H, case):
    B, n, V, D, bags, weighted, et, yt, gt, skew = case
    print(f"embed bwd {case}", flush=True)
    tok, rp, w = make(B, n, V, bags, skew=skew)
    w = w if weighted else None
    E, dy = rand(gen(D), (V, D), et), rand(gen(D + 1), (B, D), yt)
    dE, dw = torch.full((V, D), 9.0, dtype=TT[gt], device=DEV), torch.full((n,), 9.0, device=DEV)
    args = dict(row_ptr=dev(rp), weights=dev(w), scale=0.75)
    H.haste_embed_bwd(dev(tok), dy, dE, table=E, dweights=dw, **args)
    ref, size, rdw, dsize = ft.embed_bwd(tok, to_f64(dy), V, to_f64(E), rp, w, 0.75)
    inside = tok[(tok >= 0) & (tok < V)]
    cnt = np.bincount(inside, minlength=V)[:, None]
    bound = (cnt + 4) * u * size
    within("dE", to_f64(dE), ref, bound + rounded(gt, np.abs(ref) + bound))
    assert (to_f64(dE)[cnt[:, 0] == 0] == 0).all()
    within("dw", to_f64(dw), rdw, (D + 4) * u * dsize + rounded("f32", np.abs(rdw)))
    # equal bits, each alone; added to, where tokens occur and only there
    alone = H.haste_embed_bwd(dev(tok), dy, torch.empty_like(dE), **args)
    assert torch.equal(alone, dE)
    dw2 = torch.empty_like(dw)
    H.haste_embed_bwd(dev(tok), dy, None, table=E, dweights=dw2, **args)
    assert torch.equal(dw2, dw)
    base = rand(gen(3), (V, D), gt)
    absent = torch.from_numpy(cnt[:, 0] == 0).to(DEV)
    base[absent] = float("nan")
    got = H.haste_embed_bwd(dev(tok), dy, base.clone(), accumulate=True, **args)
    assert torch.isnan(got[absent]).all()
    b0, here = to_f64(base), cnt[:, 0] > 0
    b2 = bound + u * (np.abs(b0) + size) + rounded(gt, np.abs(ref) + np.abs(b0) + bound)
    within("dE added", to_f64(got)[here], (ref + b0)[here], b2[here])


def test_embed_update_in_place(H):
    """With the table as its own gradient and scale -lr the call is the SGD
    update of the rows that occur."""
    tok, rp, w = make(50, 900, 64, True)
    E, dy = rand(gen(1), (64, 96), "f32"), rand(gen(2), (50, 96), "f32")
    E[50:] = float("inf")
    tok[tok >= 50] = 3
    want = to_f64(E) - 0.1 * ft.embed_bwd(tok, to_f64(dy), 64, None, rp, w, 1.0)[0]
    H.haste_embed_bwd(dev(tok), dy, E, dev(rp), dev(w), scale=-0.1, accumulate=True)
    assert np.allclose(to_f64(E)[:50], want[:50], rtol=1e-5, atol=1e-5) and torch.isinf(E[50:]).all()


def test_embed_outside_and_nan(H):
    """A row of the table that no token names is not read into a result, a
    token outside takes nothing, and a NaN stays in the rows it belongs to."""
    for n in (40, 4000):
        E = rand(gen(5), (10, 37), "bf16")
        E[0], E[9] = float("nan"), float("inf")
        tok = np.tile(np.array([-1, 10, 3, 4, 5], np.int32), n // 5)
        rp = np.arange(0, n + 1, 5).astype(np.int32)
        tok[12] = 0
        y = to_f64(H.haste_embed_fwd(dev(tok), E, row_ptr=dev(rp), y=torch.empty(n // 5, 37, device=DEV)))
        bad = np.zeros(n // 5, bool)
        bad[2] = True
        assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()
        z = to_f64(H.haste_embed_fwd(dev(tok), E))
        assert np.isnan(z[12]).all() and np.isfinite(np.delete(z, 12, 0)).all() and (z[tok == -1] == 0).all()
        dy = torch.ones(n, 37, device=DEV)
        dy[12] = float("nan")
        dy[0] = float("nan")          # a token outside
        dE = to_f64(H.haste_embed_bwd(dev(tok), dy, torch.empty(10, 37, device=DEV)))
        assert np.isnan(dE[0]).all() and np.isfinite(dE[1:]).all() and (dE[9] == 0).all()


@pytest.mark.parametrize("D", [2, 5, 8, 15, 127, 128, 129, 256, 257, 513, 1025, 2049, 4100])
def test_embed_row_ends(H, D):
    for et, yt in (("bf16", "f32"), ("f32", "bf16")):
        for n in (200, 1200):
            case = (17, n, 50, D, 1, 1, et, yt, et, 0)
            test_embed_fwd(H, case)
            test_embed_bwd(H, case)
        test_embed_fwd(H, (70, 70, 50, D, 0, 1, et, yt, et, 0))


def test_embed_unaligned(H):
    """Bases of every tensor off the vector alignment."""
    tok, rp, w = make(20, 700, 30, True)
    E, dy = rand(gen(1), (30, 25), "bf16"), rand(gen(2), (20, 25), "bf16")

    def shift(t):
        b = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
        return b.copy_(t.reshape(-1)).view(t.shape)
    a = H.haste_embed_fwd(dev(tok), E, None, dev(rp), dev(w))
    b = H.haste_embed_fwd(shift(dev(tok)), shift(E), shift(a), shift(dev(rp)), shift(dev(w)))
    assert torch.equal(a, b)
    g = H.haste_embed_bwd(dev(tok), dy, torch.empty_like(E), dev(rp), dev(w))
    h = H.haste_embed_bwd(dev(tok), shift(dy), shift(torch.full_like(E, 7.0)), dev(rp), dev(w))
    assert torch.equal(g, h)


def test_embed_many_entries(H):
    """A list of more than 2^18 entries with tokens that fill thousands of
    chunks, on integers, where every sum is exact: equal bit for bit."""
    n, V, D, B = 400_003, 70_001, 12, 1000
    tok, rp, _ = make(B, n, V, True, skew=True)
    tok[1000:150_000] = 7
    t = torch.from_numpy(tok.astype(np.int64)).to(DEV)
    row = torch.repeat_interleave(torch.arange(B, device=DEV), torch.from_numpy(np.diff(rp)).long().to(DEV))
    live = (t >= 0) & (t < V)
    E = torch.randint(-3, 4, (V, D), generator=gen(1)).float().to(DEV)
    dy = torch.randint(-3, 4, (B, D), generator=gen(2)).float().to(DEV)
    y = H.haste_embed_fwd(dev(tok), E, None, dev(rp))
    want = torch.zeros(B, D, device=DEV, dtype=torch.float64).index_add_(0, row[live], E[t[live]].double())
    assert torch.equal(y.double(), want)
    dE = H.haste_embed_bwd(dev(tok), dy, torch.empty_like(E), dev(rp))
    want = torch.zeros(V, D, device=DEV, dtype=torch.float64).index_add_(0, t[live], dy[row[live]].double())
    assert torch.equal(dE.double(), want)


def test_embed_past_32_bits(H):
    """A table of more than 2^31 elements."""
    V, D = 2_200_000, 1024
    E = torch.zeros(V, D, dtype=torch.bfloat16, device=DEV)
    tok = torch.tensor([V - 1, 5, 2_097_153, V - 2], dtype=torch.int32, device=DEV)
    E[tok.long()] = rand(gen(1), (4, D), "bf16")
    assert torch.equal(H.haste_embed_fwd(tok, E), E[tok.long()])
    rp = torch.tensor([0, 1, 4], dtype=torch.int32, device=DEV)
    y = H.haste_embed_fwd(tok, E, None, rp)
    assert torch.equal(y[0], E[V - 1])
    dy = rand(gen(2), (4, D), "bf16")
    H.haste_embed_bwd(tok, dy, E, scale=1.0)
    assert torch.equal(E[tok.long()], dy) and int((E != 0).any(1).sum()) == 4


def test_embed_gradient_by_differences(H):
    """dE and dweights against central differences of the oracle's forward."""
    r = np.random.default_rng(3)
    tok, rp, w = make(9, 700, 30, True)
    E, dy = rand(gen(1), (30, 17), "f32"), rand(gen(2), (9, 17), "f32")
    dE, dw = torch.empty_like(E), torch.empty(700, device=DEV)
    H.haste_embed_bwd(dev(tok), dy, dE, dev(rp), dev(w), 0.5, E, dw)
    f = lambda a, b: float((ft.embed_fwd(tok, a, 9, rp, b, 0.5)[0] * to_f64(dy)).sum())  # noqa: E731
    for _ in range(3):
        vE, vw, h = r.standard_normal((30, 17)), r.standard_normal(700), 1e-5
        want = (f(to_f64(E) + h * vE, w + h * vw) - f(to_f64(E) - h * vE, w - h * vw)) / (2 * h)
        got = float((to_f64(dE) * vE).sum() + (to_f64(dw) * vw).sum())
        size = float(np.abs(to_f64(dE) * vE).sum() + np.abs(to_f64(dw) * vw).sum())
        assert abs(got - want) <= 800 * u * size + 1e-8 * size


def test_embed_captured(H):
    """Captured and replayed with changed tokens, eager work between; each
    replay against the eager call."""
    tok, rp, w = make(64, 3000, 500, True)
    T, R, W = dev(tok), dev(rp), dev(w)
    E, dy = rand(gen(1), (500, 136), "bf16"), rand(gen(2), (64, 136), "f32")
    y, dE, dw = torch.empty(64, 136, device=DEV), torch.empty(500, 136, device=DEV), torch.empty(3000, device=DEV)
    ws = torch.empty(H.haste_embed_bwd_workspace_bytes(T, dy, dE, R), dtype=torch.uint8, device=DEV)
    wf = torch.empty(1 << 22, dtype=torch.uint8, device=DEV)

    def go(y, dE, dw, ws, wf):
        H.haste_embed_fwd(T, E, y, R, W, workspace=wf)
        H.haste_embed_bwd(T, dy, dE, R, W, table=E, dweights=dw, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        go(y, dE, dw, ws, wf)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go(y, dE, dw, ws, wf)
    for i in range(4):
        T.copy_(torch.randint(-3, 510, (3000,), generator=gen(i), dtype=torch.int32))
        g.replay()
        want = [torch.empty_like(t) for t in (y, dE, dw)]
        go(*want, torch.empty_like(ws), torch.empty_like(wf))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dE, dw), want)), i


@pytest.mark.parametrize("n", [0, 1, 300])
def test_embed_many_rows(H, n):
    """More rows than a launch has workgroups for, nearly all of them empty."""
    B, V, D = (1 << 24) + 5, 50, 8
    print(f"many rows {n}", flush=True)
    tok, _, _ = make(2, n, V, 0, outside=0.0)
    rows = np.sort(np.random.default_rng(n).integers(0, B, n))
    if n:
        rows[-1] = B - 1
    rp = np.searchsorted(rows, np.arange(B + 1), "left").astype(np.int32)
    E = rand(gen(1), (V, D), "f32")
    y = H.haste_embed_fwd(dev(tok), E, torch.full((B, D), 9.0, device=DEV), row_ptr=dev(rp))
    want = torch.zeros(B, D, dtype=torch.float64, device=DEV)
    want.index_add_(0, dev(rows), E.double()[dev(tok).long()])
    assert (y.double() - want).abs().max() <= 16 * u * 4 * E.abs().max()
    assert not y[want.abs().sum(1) == 0].any()


@pytest.mark.parametrize("B", [1, 2, 256, 257, 1000])
@pytest.mark.parametrize("n", [768, 769])
def test_embed_one_launch_or_chunks(H, B, n):
    """Both sides of the number of entries and of bags where the way changes,
    bags of very unequal lengths."""
    for D, et, yt in ((768, "bf16", "f32"), (513, "f32", "bf16")):
        test_embed_fwd(H, (B, n, 400, D, 1, 1, et, yt, et, 1))
