"""Sums of the feature projections whose terms differ in size, so that an order
of summation that rounds them at every step is seen: integers in fp32, where a
sum that is rounded only once has the exact value."""
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


# rows and columns of results: no tiles, tiles of 64, 128 and 256 (bf16), ragged ones among them
SIZES = [(1, 70), (32, 33), (33, 70), (512, 768), (1500, 2052), (4100, 4040)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", SIZES)
def test_linear_bias_large_against_the_sum(H, M, N, dt):
    """Sixteen ones 256 k apart and a bias of 2^25, where the spacing of fp32 is
    4: added to the bias one at a time they are lost, their sum is not."""
    print(f"large bias {M} {N} {dt}", flush=True)
    K = 4096
    x, W = torch.ones(M, K, dtype=TT[dt], device=DEV), torch.zeros(N, K, dtype=TT[dt], device=DEV)
    W[:, ::256] = 1.0
    for bt in ("bf16", "f32"):
        b = torch.full((N,), 2.0 ** 25, dtype=TT[bt], device=DEV)
        b[::3] = 0.0
        want = b.float() + 16.0
        y, z = torch.empty(M, N, device=DEV), torch.empty(M, N, device=DEV)
        H.haste_linear_fwd(x, W, y, bias=b)
        assert torch.equal(y, want.expand(M, N))
        H.haste_linear_fwd(x, W, y, bias=b, act=H.HASTE_ACT_RELU, z=z)
        assert torch.equal(z, want.expand(M, N)) and torch.equal(y, z)
        y.fill_(8.0)      # the residual is added to the finished sum
        H.haste_linear_fwd(x, W, y, bias=b, residual=y)
        assert torch.equal(y, (want + 8.0).expand(M, N))


@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33])
def test_linear_long_sums_of_few_rows(H, n):
    """fp32, with and without tiles: 2^25, where the spacing is 4, and from the
    513th on ones 64 k apart, which one chain loses and runs of up to 256 do not
    (a wave without tiles takes 16 k of every 64)."""
    K, N = 4096, 70
    x, W = torch.ones(n, K, device=DEV), torch.zeros(N, K, device=DEV)
    W[:, 0], W[:, 512::64] = 2.0 ** 25, 1.0
    assert (H.haste_linear_fwd(x, W) == 2.0 ** 25 + (K - 512) // 64).all()
    assert (H.haste_linear_fwd(x[:, :-3], W[:, :-3].contiguous()) == 2.0 ** 25 + (K - 512) // 64).all()
