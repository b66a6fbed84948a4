"""The lengths by which attn.Attention divides its attention's work: those that
the step was told, with the library's calls recorded (CPU)."""
import pytest

from lossless_bf16_weight_afx_amd import afx
from test_attn import calls, half, ints, paged, refused  # noqa: F401

torch = pytest.importorskip("torch")


def planned(calls):
    """The attention's parameters and workspace in the last pass."""
    a = next(a for n, a in reversed(calls) if n == "afx_attend_async")
    return a[0], a[13]


def test_a_step_is_planned_by_the_length_it_was_told(calls):  # noqa: F811
    """As a call of the attention itself with that length, not with what the cache could hold."""
    c = paged(max_pages=8192, max_tokens=300)  # 131072 tokens a sequence
    t = half(c)
    for m, new, lengths in ((1, 1, (1, 500, 4096, 16000, 131072)), (4, 1, (700, 131072)), (4, 4, (3000,)),
                            (300, 300, (300, 2048, 100000))):
        rows = m // new
        starts = torch.arange(rows + 1, dtype=torch.int32) * new
        for length in lengths:
            step = c.extend(torch.arange(rows, dtype=torch.int32), starts, m, new, length)
            assert step.max_len == length
            t.forward(torch.ones(m, 256, dtype=torch.bfloat16), step)
            p, ws = planned(calls)
            assert (p.max_new, p.max_len) == (new, length)
            told = afx.attend(4, 0.125, True, 0, new, length)
            assert afx.afx_attend_workspace(told, t.kv, rows, m) <= ws


def test_without_a_length_it_is_the_caches(calls):  # noqa: F811
    c = paged()
    t = half(c)
    step = c.extend(ints(0), ints(0, 7), 7)
    assert step.max_len == 128
    t.forward(torch.ones(7, 256, dtype=torch.bfloat16), step)
    assert planned(calls)[0].max_len == 128


def test_lengths_that_are_refused(calls):  # noqa: F811
    c = paged()
    for length in (0, -1, 129):
        refused(calls, c.extend, ints(0), ints(0, 7), 7, 7, length)


def test_steps_of_unusual_sizes_are_cut_into_what_there_is_room_for(calls, monkeypatch):  # noqa: F811
    """Not into one part as soon as the workspace is smaller than the plan's."""
    c = paged(max_pages=8192, max_tokens=384, max_seqs=40, max_rows=40)
    t = half(c)
    for rows, new in ((1, 1), (38, 7), (3, 1)):
        m = rows * new
        starts = torch.arange(rows + 1, dtype=torch.int32) * new
        need = afx.afx_attend_workspace(t._attend(new, 131072), t.kv, rows, m)
        for part in (1, 2, 3, 8):
            if need // part < 4 * m * 4 * 66 * 2:
                continue  # (less than two parts of its queries)
            monkeypatch.setattr(t, "ws", torch.empty(need // part, dtype=torch.uint8))
            step = c.extend(torch.arange(rows, dtype=torch.int32), starts, m, new)
            t.forward(torch.ones(m, 256, dtype=torch.bfloat16), step)
            p, ws = planned(calls)
            assert ws == need // part
            assert ws / 2.5 < afx.afx_attend_workspace(p, t.kv, rows, m) <= ws, (rows, new, part)
