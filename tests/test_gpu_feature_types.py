"""Every pairing of types through every width's kernel of the embedding and of
the norms around a block, against the fp64 oracle with the bounds of their own
tests."""
import pytest

from tests import test_gpu_addnorm as an
from tests import test_gpu_embed as em

pytestmark = pytest.mark.gpu
TYPES = [(a, b, c) for a in ("bf16", "f32") for b in ("bf16", "f32") for c in ("bf16", "f32")]


@pytest.fixture(scope="module")
def H():
    from sparse_output_layer_amd import haste
    haste.lib()
    return haste


@pytest.mark.parametrize("o,r,y", TYPES)
@pytest.mark.parametrize("D", [128, 127, 256, 250, 512, 511, 768, 765, 1024, 1001, 2048, 2045, 4096, 4093, 8192, 8190, 9000, 9001])
def test_addnorm_types_and_widths(H, D, o, r, y):
    """Widths of whole vectors and others; gate, post norm, weights' type and
    dropout change with the width."""
    k = D % 5
    case = (19 if D < 2000 else 3, D, o, r, y, ("f32", "bf16")[D & 1], int(k != 3), 1, ("vector", "rows", "none")[k % 3], 1, 0.2 * (k & 1))
    an.test_addnorm_fwd(H, case)
    an.test_addnorm_bwd(H, case, True)


@pytest.mark.parametrize("e,y,g", TYPES)
@pytest.mark.parametrize("D", [100, 104, 200, 251, 400, 509, 800, 1001, 1504, 2047])
def test_embed_types_and_widths(H, D, e, y, g):
    """Bags as a list and by a workgroup each (of 16 and of four waves), lookups,
    the table's gradient with the weights' and alone."""
    for case in ((40, 900, 60, D, 1, 1, e, y, g, D & 1), (9, 300, 60, D, 1, 0, e, y, g, 0), (300, 500, 60, D, 1, 1, e, y, g, 0),
                 (90, 90, 60, D, 0, D & 1, e, y, g, 0)):
        em.test_embed_fwd(H, case)
        em.test_embed_bwd(H, case)
