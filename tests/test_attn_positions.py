"""The positions that attn.Attention passes on, with the library's calls
recorded (CPU): every axis has a row of its own in memory, as the kernel reads
rows pos_stride apart."""
import pytest

from test_attn import calls, half, ints, paged, refused  # noqa: F401

torch = pytest.importorskip("torch")


def several(c):
    return half(c, freq=torch.ones(16), axis=torch.arange(16).remainder(3).to(torch.uint8), n_axes=3)


def given(calls):
    """The positions' address and stride of the last pass."""
    return next(a[2:4] for n, a in reversed(calls) if n == "afx_heads_async")


def test_rows_that_share_memory_are_refused(calls):  # noqa: F811
    c = paged()
    t, m = several(c), 7
    r, step = torch.ones(m, 256, dtype=torch.bfloat16), c.extend(ints(3, 1), ints(0, 2, m), m)
    line = torch.arange(m, dtype=torch.int32)
    for bad in (line[None].expand(3, m),  # the same positions along every axis
                torch.arange(9, dtype=torch.int32).as_strided((3, m), (1, 1)),
                torch.arange(m + 12, dtype=torch.int32).as_strided((3, m), (m - 1, 1))):
        refused(calls, t.forward, r, step, bad)


def test_rows_with_memory_of_their_own(calls):  # noqa: F811
    c = paged()
    t, m = several(c), 7
    r, step = torch.ones(m, 256, dtype=torch.bfloat16), c.extend(ints(3, 1), ints(0, 2, m), m)
    whole = torch.arange(60, dtype=torch.int32).view(3, 20)
    for pos in (whole[:, :m], whole[:, 5:5 + m], whole[:, :m].contiguous(),
                torch.arange(m, dtype=torch.int32)[None].repeat(3, 1)):
        t.forward(r, step, pos)
        assert given(calls) == (pos.data_ptr(), pos.stride(0))
        last = pos.data_ptr() + 4 * (2 * given(calls)[1] + m)  # behind the last value that is read
        assert last <= pos.untyped_storage().data_ptr() + pos.untyped_storage().nbytes()


def test_one_axis_has_one_row(calls):  # noqa: F811
    c = paged()
    t, m = half(c, freq=torch.ones(16)), 7
    r, step = torch.ones(m, 256, dtype=torch.bfloat16), c.extend(ints(3, 1), ints(0, 2, m), m)
    line = torch.arange(m, dtype=torch.int32)
    for pos in (line[None], line[None].expand(1, m), torch.arange(40, dtype=torch.int32).view(2, 20)[1:, :m]):
        t.forward(r, step, pos)
        assert given(calls) == (pos.data_ptr(), m)
    t.forward(r, step)
    assert given(calls) == (step.pos.data_ptr(), m)


def test_one_token(calls):  # noqa: F811
    c = paged()
    t = several(c)
    r, step = torch.ones(1, 256, dtype=torch.bfloat16), c.extend(ints(3), ints(0, 1), 1)
    pos = ints(5, 1, 2)[:, None]
    t.forward(r, step, pos)
    assert given(calls) == (pos.data_ptr(), 1)
    refused(calls, t.forward, r, step, ints(5)[None].expand(3, 1))
