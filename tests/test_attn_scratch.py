"""The memory that the layers' halves over one cache share, with the library's
calls recorded (CPU)."""
import pytest

from test_attn import calls, half, ints, paged  # noqa: F401

torch = pytest.importorskip("torch")


def held(t):
    """Where an object's shared buffers begin, and how many bytes they have."""
    return [(x.data_ptr(), x.numel() * x.element_size()) for x in (t.y, t.ws)]


def test_layers_share_what_a_pass_uses_up(calls):  # noqa: F811
    c = paged(layers=3)
    first, second, third = (half(c, layer=i) for i in range(3))
    assert held(first) == held(second) == held(third)
    other = half(paged())
    assert not {p for p, _ in held(other)} & {p for p, _ in held(first)}
    # what a layer keeps or hands on is its own
    kept = [x.data_ptr() for t in (first, second) for x in (t.xn, t.qn, t.a, t.r_out)]
    assert len(set(kept)) == len(kept)


def test_sizes_differ(calls):  # noqa: F811
    """Objects for fewer tokens use a part, those for more get more; nobody's buffer is taken away."""
    c = paged(max_tokens=100, n_pages=100, max_pages=80)
    small, large = half(c, max_tokens=7), half(c)
    assert held(large)[0][1] == 4 * 100 * (256 + 256 + 256) and held(small)[0][1] == 4 * 7 * (256 + 256 + 256)
    again = half(c, max_tokens=9)
    assert held(again)[0][0] == held(large)[0][0] and held(again)[0][1] == 4 * 9 * 768
    for t, m in ((small, 7), (large, 100), (again, 9), (small, 1)):
        t.forward(torch.ones(m, 256, dtype=torch.bfloat16), c.extend(ints(0), ints(0, m), m))
        a = next(a for n, a in reversed(calls) if n == "afx_attend_async")
        assert a[12:14] == held(t)[1] and a[12] % 16 == 0
        heads = next(a for n, a in reversed(calls) if n == "afx_heads_async")
        assert heads[4] == held(t)[0][0]
