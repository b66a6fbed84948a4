"""Steps of a fixed number of tokens, of which the last belong to no row or to
refused rows, as a captured step has them; and graphs of several layers over
one cache that share its scratch memory. Tolerances as in
tests/test_gpu_attn_run.py."""
import pytest

from lossless_bf16_weight_afx_amd import afx
from test_gpu_attn_run import Model, ints

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


@pytest.mark.parametrize("m", [8, 33, 150])
def test_tokens_of_no_row_reach_nobody(m):
    """Whatever they hold, and whatever the buffers held before."""
    g = Model(m)
    g.take([(0, 20), (3, 41), (6, 1)])
    for t in g.layers:
        for x in (t.attn.xn, t.attn.qn, t.attn.a, t.attn.r_out, t.attn.xn_next):
            x.fill_(float("nan"))
    for rows in ([(0, 1), (3, 2), (6, 1)], [(6, 3), (0, 1)], [(3, 0), (0, 4)]):
        n = sum(k for _, k in rows)
        r = g.values(m)
        r[n:] = float("nan")
        r[n::2] = float("inf")
        starts = [0]
        for _, k in rows:
            starts.append(starts[-1] + k)
        before = g.c.data.view(torch.int16).clone()
        step, got = g.step(r, ints(*(s for s, _ in rows)), ints(*starts), max(k for _, k in rows))
        assert step.granted.tolist() == [k for _, k in rows] and step.slots[n:].tolist() == [-1] * (m - n)
        g.compare(r[:n], rows, [(a[:n], b[:n]) for a, b in got])
        # the cache has changed in as many places as tokens were written
        changed = (g.c.data.view(torch.int16) != before).sum()
        assert int(changed) <= n * 2 * len(g.layers) * 2 * 64
    g.lengths()


def test_refused_rows_beside_others_with_strange_tokens():
    g = Model(5, n_pages=4)
    g.take([(0, 30), (1, 16)])
    r = g.values(37)
    r[4:] = float("nan")
    step, got = g.step(r, ints(0, 1, 9, 2), ints(0, 2, 4, 6, 37), 31)  # an id outside the table, too few pages
    assert step.granted.tolist() == [2, 2, 0, 0]
    g.compare(r[:4], [(0, 2), (1, 2)], [(a[:4], b[:4]) for a, b in got])


def test_graphs_of_steps_of_two_sizes_share_the_scratch():
    """Replayed in turn, with eager steps between them: what one leaves in the shared memory is not read by another."""
    g = Model(9)
    g.take([(0, 20), (3, 9), (6, 47)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sizes = {"one": ([(0, 1), (3, 1), (6, 1)], 1), "drafts": ([(6, 4), (0, 3)], 4)}
    graphs = {}
    with torch.cuda.stream(side):
        for name, (rows, most) in sizes.items():
            n = sum(k for _, k in rows)
            starts = [0]
            for _, k in rows:
                starts.append(starts[-1] + k)
            r, seqs, at = g.values(n), ints(*(s for s, _ in rows)), ints(*starts)
            _, got = g.step(r, seqs, at, most)
            side.synchronize()
            g.compare(r, rows, got)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                step, got = g.step(r, seqs, at, most)
            graphs[name] = graph, r, step, got, rows, (seqs, at)
    for i, name in enumerate(["one", "drafts", "drafts", "one", "one", "drafts", "one"]):
        graph, r, step, got, rows, _ = graphs[name]
        r.copy_(g.values(r.shape[0]))
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert step.granted[:len(rows)].tolist() == [k for _, k in rows]
        g.compare(r, rows, got)
        if i % 3 == 1:
            g.take([(1, 60 - 20 * (i // 3)), (3, 2)])
            torch.cuda.synchronize()
    g.lengths()
