"""The feature stage at the sizes its entry points allow at most, on small
integers, whose sums are exact, against tensor operations on the device."""
import pytest
import torch

from tests._gpu import DEV
from tests.test_gpu_ops import TT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def H():
    from sparse_output_layer_amd import haste
    haste.lib()
    return haste


@pytest.fixture(autouse=True)
def give_back():
    yield
    torch.cuda.empty_cache()


def ints(seed, shape, dt, most):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV).to(TT[dt])


def test_embed_most_rows_of_a_table(H):
    """2^31 - 1 table rows: keys of 31 bits, the padding's among them."""
    V, n = 2 ** 31 - 1, 5000
    E = torch.zeros(V, 1, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    tok = torch.randint(-100, V, (n,), generator=g, device=DEV).to(torch.int32)
    tok[:8] = torch.tensor([0, V - 1, 2 ** 30, V, -1, -2 ** 31, V - 1, 2 ** 30 - 1], device=DEV)
    tok[4000:4500] = V - 1
    live = (tok >= 0) & (tok < V)
    at = tok.long()[live]
    E[at] = ints(2, (len(at), 1), "bf16", 9)
    want = torch.zeros(n, 1, device=DEV)
    want[live] = E[at].float()
    assert torch.equal(H.haste_embed_fwd(tok, E, torch.empty(n, 1, device=DEV)), want)
    dy = ints(3, (n, 1), "f32", 3)
    met, which = torch.unique(at, return_inverse=True)
    sums = torch.zeros(len(met), 1, device=DEV, dtype=torch.float64).index_add_(0, which, dy[live].double())
    E.fill_(5.0)
    H.haste_embed_bwd(tok, dy, E)
    assert torch.equal(E[met].double(), sums.bfloat16().double())
    assert int((E != 0).sum()) == int((sums != 0).sum())


@pytest.mark.parametrize("n", [5, 800])
def test_embed_widest_rows(H, n):
    """Rows of 2^20, in bags of one launch and in chunks, and one token a row."""
    V, D, B = 3, 1 << 20, 5
    E, dy = ints(1, (V, D), "f32", 3), ints(2, (B, D), "bf16", 3)
    tok = ints(3, (n,), "f32", 3).to(torch.int32)      # some outside
    rp = torch.tensor([0, 1, 1, n // 2, n, n], dtype=torch.int32, device=DEV)
    row = torch.repeat_interleave(torch.arange(B, device=DEV), (rp[1:] - rp[:-1]).long())
    live = (tok >= 0) & (tok < V)
    t, r = tok.long()[live], row[live]
    y = H.haste_embed_fwd(tok, E, None, rp)
    assert torch.equal(y, torch.zeros(B, D, device=DEV).index_add_(0, r, E[t]))
    dE, dw = torch.full_like(E, 7.0), torch.empty(n, device=DEV)
    H.haste_embed_bwd(tok, dy, dE, rp, table=E, dweights=dw)
    assert torch.equal(dE, torch.zeros_like(E).index_add_(0, t, dy[r].float()))
    want = torch.zeros(n, device=DEV, dtype=torch.float64)
    pairs = E.double() @ dy.double().T
    want[live] = pairs[t, r]
    assert torch.equal(dw.double(), want)
    if n == B:
        assert torch.equal(H.haste_embed_fwd(tok, E), E[tok.long().clamp(0, V - 1)] * live[:, None])


def test_embed_most_entries(H):
    """2^28 entries of bags and of a gradient, seven tokens."""
    n, V, B = 1 << 28, 7, 1000
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    tok = torch.randint(0, V + 1, (n,), generator=g, device=DEV, dtype=torch.int32)      # V: outside
    cut = torch.sort(torch.randint(0, n + 1, (B - 1,), generator=g, device=DEV))[0]
    ends = torch.cat([torch.zeros(1, device=DEV), cut, torch.full((1,), n, device=DEV)]).long()
    rp = ends.to(torch.int32)
    E, dy = torch.tensor([[0.], [1.], [-1.], [2.], [-2.], [1.], [-1.]], device=DEV), ints(5, (B, 1), "f32", 1)
    table = torch.cat([E[:, 0], torch.zeros(1, device=DEV)])
    count = torch.zeros(B, V + 1, dtype=torch.float64, device=DEV)
    for b, (lo, hi) in enumerate(zip(ends[:-1].tolist(), ends[1:].tolist())):
        count[b] = torch.bincount(tok[lo:hi].long(), minlength=V + 1)
    y = H.haste_embed_fwd(tok, E, None, rp)
    assert torch.equal(y[:, 0].double(), count @ table.double())
    dE = H.haste_embed_bwd(tok, dy, torch.empty_like(E), rp)
    assert torch.equal(dE.double(), count.T[:V].contiguous() @ dy.double())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M", [5, 40])
@pytest.mark.parametrize("K,N", [(8, 1 << 22), (1 << 22, 9)])
def test_linear_widest(H, M, K, N, dt):
    """2^22 output features and 2^22 input features, with and without tiles."""
    x, W, dy = ints(1, (M, K), dt, 1), ints(2, (N, K), dt, 1), ints(3, (M, N), dt, 1)
    b = ints(4, (N,), "f32", 9)
    y = H.haste_linear_fwd(x, W, torch.empty(M, N, device=DEV), bias=b)
    assert torch.equal(y.double(), x.double() @ W.double().T + b.double())
    dx, dW, db = torch.empty_like(x), torch.empty_like(W), torch.empty(N, device=DEV)
    H.haste_linear_bwd(x, W, dy, dx=dx, dW=dW, dbias=db)
    assert torch.equal(dx, (dy.double() @ W.double()).to(TT[dt]))
    assert torch.equal(dW, (dy.double().T.contiguous() @ x.double()).to(TT[dt]))
    assert torch.equal(db.double(), dy.double().sum(0))


@pytest.mark.parametrize("dt,M", [("bf16", 3584), ("bf16", 700), ("f32", 1792), ("f32", 300)])
def test_linear_farthest_rows(H, dt, M):
    """Rows of x 2^22 elements apart (a tile of them reaches over 2^31 bytes less
    one row), dx's as far."""
    K, N, ld = 40, M, 1 << 22
    x = torch.empty(M, ld, dtype=TT[dt], device=DEV)[:, 24:24 + K]
    x.copy_(ints(1, (M, K), dt, 3))
    W, dy = ints(2, (N, K), dt, 3), ints(3, (M, N), dt, 1)
    X = x.double()
    assert torch.equal(H.haste_linear_fwd(x, W, torch.empty(M, N, device=DEV)).double(), X @ W.double().T)
    dW = torch.empty_like(W)
    H.haste_linear_bwd(x, W, dy, dW=dW)
    assert torch.equal(dW, (dy.double().T.contiguous() @ X).to(TT[dt]))
    H.haste_linear_bwd(torch.empty_like(x), W, dy, dx=x)      # x is only a shape here
    assert torch.equal(x, (dy.double() @ W.double()).to(TT[dt]))


def test_addnorm_many_rows_and_long_ones(H):
    """2^25 + 3 rows of 8, and rows of 2^24 + 5: means, sums and ends."""
    B, D = 2 ** 25 + 3, 8
    o, r = ints(1, (B, D), "bf16", 4), ints(2, (B, D), "bf16", 4)
    st = torch.zeros(4, B, device=DEV)
    norm, grad = H.NormWeights(), H.NormWeights(torch.empty(D, device=DEV), torch.empty(D, device=DEV))
    r_out, y = H.haste_addnorm_fwd(o, r, torch.empty(B, D, device=DEV, dtype=torch.bfloat16), norm=norm, stats=st)
    s = o.float() + r.float()
    assert torch.equal(r_out.float(), s) and torch.equal(st[2], s.mean(1))
    v = (s - s.mean(1, keepdim=True)).double()
    rstd = 1 / torch.sqrt((v * v).mean(1) + 1e-5)
    assert ((st[3].double() - rstd).abs() <= 1e-6 * rstd).all()
    assert ((y.double() - v * rstd[:, None]).abs() <= 2.0 ** -8 * (v * rstd[:, None]).abs() + 1e-5).all()
    del v, rstd, y
    dy = ints(3, (B, D), "bf16", 1)
    dr, do = H.haste_addnorm_bwd(o, r_out, st, dy, norm=norm, dnorm=grad)
    assert torch.equal(grad.beta.double(), dy.double().sum(0)) and torch.equal(dr, do)
    assert (dr[-1000:].float().sum(1).abs() <= 0.05).all() and torch.isfinite(dr).all()
    del o, r, st, r_out, s, dy, dr, do
    D = 2 ** 24 + 5
    o, r = ints(4, (2, D), "bf16", 1), ints(5, (2, D), "f32", 1)
    st = torch.zeros(4, 2, device=DEV)
    r_out, y = H.haste_addnorm_fwd(o, r, y=torch.empty(2, D, device=DEV), norm=norm, stats=st)
    s = o.float() + r
    assert torch.equal(r_out, s)
    m = s.double().mean(1, keepdim=True)
    q = 1 / torch.sqrt(((s.double() - m) ** 2).mean(1, keepdim=True) + 1e-5)
    assert ((st[2].double() - m[:, 0]).abs() <= 1e-6).all() and ((st[3].double() - q[:, 0]).abs() <= 1e-3 * q[:, 0]).all()
    assert ((y.double() - (s - m) * q).abs() <= 5e-3).all()
