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


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("new, length, max_len", [(1, 300, 300), (1, 5000, 5000), (6, 5000, 5000), (1, 30000, 30000),
                                                  (60, 300, 300), (60, 5000, 5000)])
def test_what_a_query_sees_shows_however_the_work_is_cut(new, length, max_len, value):
    """A value that is infinite or NaN at a score of 256 below the largest: its weight is above 0, so that the output is
    no number that is finite, wherever its token stands beside the largest one."""
    top = 37
    for far in (38, 45, 70, 100, 200, length - new - 20):
        b = Batch(far, [length], [(0, new)], kv_heads=1, group=2, dim=64)
        b.q[:] = 0.0
        b.q[:, [0, 64]] = 16.0
        b.keys[0][:] = 0.0
        b.keys[0][top, 0, 0] = 8.0
        b.keys[0][far, 0, 0] = -8.0
        b.values[0][far, 0, 3] = value
        b.upload()
        b.run(scale=1.0, max_len=max_len)
        out = b.out[:new].reshape(new, 2, 64).cpu()
        bad = out[:, :, 3]
        assert bool((~torch.isfinite(bad)).all()), f"token {far}: {bad[0, 0]} where the value is {value}"
        assert not math.isnan(value) or bool(torch.isnan(bad).all())
        rest = [d for d in range(64) if d != 3]
        # the others are the top token's (all other weights together: 30000 e^-128)
        assert torch.equal(out[:, :, rest], b.values[0][top, 0, rest].expand(new, 2, 63))


@pytest.mark.parametrize("dim", [64, 128, 136, 256])
@pytest.mark.parametrize("length, new", [(200, 6), (4000, 6), (150, 70), (2000, 70)])
@pytest.mark.parametrize("value", [1.0, math.nan, math.inf])
@pytest.mark.parametrize("window", [0, 50])
def test_what_a_query_does_not_see_changes_none_of_its_bits(dim, length, new, value, window):
    """The last two new tokens' keys and values, and what only the first new token's window reaches, are replaced."""
    b = Batch(dim + length + new, [length], [(0, new)], kv_heads=1, group=3, dim=dim)
    b.upload()
    how = dict(scale=dim ** -0.5, window=window)
    b.run(**how)
    b.check()
    out, lse = b.out.clone(), b.lse.clone()
    places = [length - 1, length - 2]
    if window:
        places.append(length - new - window + 1)  # (the first new token's first)
    for at in places:
        b.keys[0][at] = b.q[new - 1, :dim] * 4  # larger scores than any
        b.values[0][at, 0, ::3] = value
    b.upload()
    b.run(**how)
    first, end = 1 if window else 0, new - 2
    assert torch.equal(b.lse[first:end], lse[first:end])
    assert torch.equal(b.out[first:end].view(torch.int16), out[first:end].view(torch.int16))
    changed = b.out[end:new].reshape(2, 3, dim)[:, :, ::3].float()
    assert math.isfinite(value) == bool(torch.isfinite(changed).all())


@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("new, length", [(1, 700), (5, 700), (80, 700), (80, 3000)])
def test_beside_pages_outside_the_cache(page, new, length):
    """Tiles that every query sees but for a page that is not there."""
    b = Batch(page + new, [length, 40], [(0, new), (1, 1)], kv_heads=2, group=3, dim=72, page=page)
    for i in (1, 3):
        b.table[0, i] = -1
        b.there[0][page * i:page * (i + 1)] = False
    for at, value in ((page - 1, math.inf), (2 * page, math.nan), (2 * page + 3, -math.inf), (4 * page, math.inf),
                      (length - 1, math.nan), (length - new, math.inf)):
        b.values[0][at, at % 2, at % 72] = value
    b.upload()
    b.run(scale=0.125)
    b.check()
