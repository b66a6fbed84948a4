"""Attention over a paged cache where keys or values are infinite or NaN: in
any of a head's dimensions, at scores far below the largest, and where only
other queries see them."""
import math

import pytest

from lossless_bf16_weight_afx_amd import afx
from test_gpu_attend import Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


@pytest.mark.parametrize("dim", [8, 24, 64, 72, 88, 120, 128, 136, 152, 168, 184, 192, 200, 216, 232, 248, 256])
@pytest.mark.parametrize("new", [1, 40])
def test_scores_of_minus_infinity_from_any_dimension(dim, new):
    """Keys whose score is minus infinity weigh nothing, whichever of their values is infinite."""
    b = Batch(dim + new, [70, 60, 45], [(0, new), (1, new), (2, 1)], kv_heads=1, group=2, dim=dim)
    first, last = torch.arange(2) * dim, torch.arange(2) * dim + dim - 1
    for at in (first, last):
        b.q[:, at] = 1.0
    for s, place in ((0, dim - 1), (1, dim - 1), (2, 0)):
        seen = 0 if s == 1 else 5  # sequence 1: nothing else
        b.keys[s][seen:, 0] = 0.0
        b.keys[s][seen:, 0, place] = -math.inf
    b.upload()
    b.run(scale=dim ** -0.5)
    b.check()
