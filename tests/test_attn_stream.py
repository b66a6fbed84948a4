"""Which rows of r' attn.Attention takes as its next stream, with the library's
calls recorded (CPU): a stream is refused before anything is enqueued, above
all before keys and values are written to the cache."""
import pytest

from lossless_bf16_weight_afx_amd import afx
from test_attn import calls, half, ints, paged, refused  # noqa: F401

torch = pytest.importorskip("torch")


def test_rows_of_the_last_pass(calls):  # noqa: F811
    c = paged()
    t = half(c)
    for m, first in ((7, 0), (1, 0), (3, 3), (1, 1), (20, 20)):
        step = c.extend(ints(3), ints(0, m), m)
        t.forward(t.r_out[first:first + m], step)
        n = len(calls)
        assert n and calls[-1][1][4] == t.r_out[first].data_ptr()


def test_rows_that_others_are_written_to_first(calls):  # noqa: F811
    c = paged()
    t = half(c)
    flat = t.r_out.view(-1)
    for m, r in ((7, t.r_out[1:8]), (7, t.r_out[6:13]), (2, t.r_out[:4:2]), (2, flat[128:128 + 512].view(2, 256)),
                 (1, flat[8:264].view(1, 256)), (1, flat[255:511].view(1, 256))):
        step = c.extend(ints(3), ints(0, m), m)
        refused(calls, t.forward, r, step)


@pytest.mark.parametrize("kw", [dict(scale=float("nan")), dict(scale=float("inf")), dict(eps=0.0), dict(eps=-1e-6),
                                dict(eps=float("nan")), dict(eps=float("inf")), dict(d=afx.MAX_NORM_WIDTH + 256)])
def test_norms_that_a_pass_would_refuse(calls, kw):  # noqa: F811
    """When the object is made, not by the last call of each pass."""
    refused(calls, half, paged(), **kw)
