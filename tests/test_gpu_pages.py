"""The cache's pages forked, trimmed, grown, compacted and copied, against the
rules on lists of whole numbers (tests/paged_reference.py): tables, lengths,
counts, slots and every byte of the pages have to be equal."""
import random

import pytest

import paged_reference as ref
from lossless_bf16_weight_afx_amd import afx

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Cache:
    def __init__(self, seed, n_seqs, max_pages, n_pages, size=16, *, planes=3, page_bytes=4096, gap=32):
        self.model = ref.Pages(n_seqs, max_pages, n_pages, size)
        self.n_pages, self.planes, self.page_bytes = n_pages, planes, page_bytes
        self.stride = n_pages * page_bytes + gap
        gen = torch.Generator().manual_seed(seed)
        self.data = torch.randint(0, 256, (planes, self.stride), generator=gen, dtype=torch.uint8).cuda()
        self.bytes = self.data.clone()
        self.table = torch.full((n_seqs, max_pages + 3), -1, dtype=torch.int32, device="cuda")
        self.table[:, max_pages:] = 99
        self.len, self.refs = ints([0] * n_seqs), ints([0] * n_pages)
        self.t = afx.page_table(self.table.data_ptr(), max_pages + 3, self.len.data_ptr(), self.refs.data_ptr(), n_seqs,
                                max_pages, n_pages, size)
        self.d = afx.page_data(self.data.data_ptr(), page_bytes, self.stride, planes)
        self.stream = torch.cuda.current_stream().cuda_stream

    def page(self, i):
        return self.bytes[:, i * self.page_bytes:(i + 1) * self.page_bytes]

    def check(self):
        torch.cuda.synchronize()
        m = self.model
        for a, b in m.copies:
            self.page(b).copy_(self.page(a))
        m.copies.clear()
        assert self.table[:, :len(m.table[0])].tolist() == m.table
        assert bool((self.table[:, len(m.table[0]):] == 99).all())
        assert self.len.tolist() == m.len and self.refs.tolist() == m.refs
        held = [0] * self.n_pages
        for row in m.table:
            for e in row:
                if e >= 0:
                    held[e] += 1
        assert held == m.refs
        assert torch.equal(self.data, self.bytes)

    def fork(self, src, dst):
        granted, a, b = ints([7] * len(src)), ints(src), ints(dst)
        afx.afx_pages_fork_async(self.t, len(src), a.data_ptr(), b.data_ptr(), granted.data_ptr(), self.stream)
        want = self.model.fork(src, dst)
        self.check()
        assert granted.tolist() == want

    def trim(self, seqs, lens=None):
        a, b = ints(seqs), None if lens is None else ints(lens)
        afx.afx_pages_trim_async(self.t, len(seqs), a.data_ptr(), 0 if b is None else b.data_ptr(), self.stream)
        self.model.trim(seqs, lens)
        self.check()

    def extend(self, seqs, new, before=0, behind=0):
        starts = [before]
        for n in new:
            starts.append(starts[-1] + n)
        m = starts[-1] + behind
        a, b = ints(seqs), ints(starts)
        slots, pos, granted = ints([7] * max(m, 1)), ints([7] * max(m, 1)), ints([7] * len(seqs))
        ws = torch.empty(afx.afx_pages_extend_workspace(self.t, len(seqs)), dtype=torch.uint8, device="cuda")
        afx.afx_pages_extend_async(self.t, self.d, len(seqs), a.data_ptr(), b.data_ptr(), m, slots.data_ptr(),
                                   pos.data_ptr(), granted.data_ptr(), ws.data_ptr(), ws.numel(), self.stream)
        ws_slots, ws_pos, ws_granted = self.model.extend(seqs, starts, m)
        self.check()
        assert granted.tolist() == ws_granted
        assert slots.tolist()[:m] == ws_slots and pos.tolist()[:m] == ws_pos

    def compact(self):
        moved, live = ints([7] * self.n_pages), ints([7])
        ws = torch.empty(afx.afx_pages_compact_workspace(self.t), dtype=torch.uint8, device="cuda")
        afx.afx_pages_compact_async(self.t, self.d, moved.data_ptr(), live.data_ptr(), ws.data_ptr(), ws.numel(),
                                    self.stream)
        want = self.model.compact()
        self.check()
        assert (moved.tolist(), live.item()) == want


def test_a_sequence_grows_branches_and_goes():
    c = Cache(1, 5, 6, 14)
    c.extend([2], [20])
    c.extend([2], [1])
    c.fork([2], [0])
    c.extend([2], [3])  # the shared last page is copied
    c.extend([0], [3])  # its last holder keeps it
    c.fork([0], [4])
    c.trim([0], [17])   # a partly used page that 4 holds too
    c.extend([0, 4], [2, 2])
    c.trim([2])
    c.compact()
    c.trim([0, 4])
    c.compact()


@pytest.mark.parametrize("size", [16, 32, 64, 128, 256])
def test_lengths_around_pages(size):
    c = Cache(size, 4, 5, 24, size, planes=1, page_bytes=16)
    for n in (1, size - 2, 1, 1, size, size - 1, 0, 1, 2 * size, size, 1):
        c.extend([1, 3], [n, 1])
        if n == size:
            c.fork([1], [0])
            c.trim([1], [size])
            c.fork([0], [2])
    c.trim([0, 1, 2, 3], [size, 0, size + 1, -5])


def test_several_holders_of_one_page():
    """Of rows that share a partly filled page all but its last holder copy
    it, and all do if others hold it too."""
    for rows in ([1, 2, 3], [0, 1, 2, 3], [3, 0]):
        c = Cache(2, 4, 4, 12)
        c.extend([0], [20])
        c.fork([0, 0, 0], [1, 2, 3])
        c.extend(rows, [1] * len(rows))


def test_too_few_pages():
    c = Cache(3, 6, 8, 7)
    c.extend([0, 1, 2, 3], [33, 40, 30, 1])  # 3 + 3 pages, then not 2, nor any
    c.extend([3, 4], [0, 5])
    c.fork([0, 1], [2, 3])
    c.extend([2, 3], [1, 1])  # copies wanted, none left
    c.trim([3])
    c.extend([0, 2], [15, 1])
    c.extend([1], [200])  # more pages than there are, and than a row holds
    c.extend([1], [88])


def test_rows_that_are_refused():
    c = Cache(4, 6, 4, 40)
    c.extend([-1, 6, 2 ** 31 - 1, -2 ** 31, 1, 1, 2], [3, 3, 3, 3, 20, 5, 7], before=2, behind=5)
    c.extend([1, 2], [45, 100])  # more than max_pages pages
    c.fork([1, 1, 1, 0, -1, 1, 6, 3], [3, 3, 2, 4, 5, 6, 5, 5])
    c.fork([3, 4, 1], [4, 5, 1])  # a source that is a destination; a sequence onto itself
    c.fork([4], [5])  # of an empty sequence
    c.trim([1, -1, 6, 1, 3, 5], [17, 0, 0, 0, 10 ** 6, 0])
    c.trim([3, 3, 2], [5, 0, 7])


def test_no_tokens():
    c = Cache(5, 3, 4, 8)
    c.extend([0, 1], [0, 0])
    c.extend([0, 1], [0, 18], behind=3)
    c.trim([0, 2])


def test_full_lists():
    """1024 rows, over more counts than one block of the scan."""
    rng = random.Random(6)
    c = Cache(6, 1100, 3, 9000, planes=1, page_bytes=32)
    order = list(range(1100))
    rng.shuffle(order)
    c.extend(order[:1024], [rng.randrange(0, 48) for _ in range(1024)])
    c.trim(order[:500])
    c.extend(order[100:1100], [rng.randrange(0, 20) for _ in range(1000)])
    held = [s for s in range(1100) if c.model.len[s]]
    empty = [s for s in range(1100) if not c.model.len[s]]
    if empty:
        c.fork([rng.choice(held) for _ in empty], empty)
    c.compact()


@pytest.mark.parametrize("seed", range(6))
def test_steps_at_random(seed):
    rng = random.Random(seed)
    n_seqs, max_pages, n_pages = rng.randrange(3, 40), rng.randrange(1, 12), rng.randrange(5, 200)
    size = rng.choice((16, 32))
    c = Cache(seed, n_seqs, max_pages, n_pages, size, planes=rng.choice((1, 4)),
              page_bytes=rng.choice((16, 4096, 40000, 16400)))
    for _ in range(40):
        n = rng.randrange(1, n_seqs + 3)
        rows = [rng.randrange(-1, n_seqs + 1) for _ in range(n)]
        what = rng.choice(("extend", "extend", "extend", "fork", "trim", "free", "compact"))
        if what == "extend":
            c.extend(rows, [rng.choice((0, 1, 1, 2, 15, 16, 17, 40)) for _ in rows], rng.randrange(2), rng.randrange(3))
        elif what == "fork":
            c.fork(rows, [rng.randrange(-1, n_seqs + 1) for _ in rows])
        elif what == "trim":
            c.trim(rows, [rng.randrange(-2, max_pages * size) for _ in rows])
        elif what == "free":
            c.trim(rows[:2])
        else:
            c.compact()


def test_copies():
    c = Cache(7, 2, 4, 50, planes=5, page_bytes=20000 // 16 * 16)
    src, dst = [0, 7, 49, -1, 3, 50, 2 ** 31 - 1, 9, 7], [1, 8, 48, 2, 50, 4, 5, 9, 11]
    a, b = ints(src), ints(dst)
    afx.afx_pages_copy_async(c.d, 50, len(src), a.data_ptr(), b.data_ptr(), c.stream)
    c.model.copies += [(s, d) for s, d in zip(src, dst) if 0 <= s < 50 and 0 <= d < 50 and s != d]
    c.check()


def test_far_pages():
    """Pages above 2^32 bytes of a plane, planes above that too."""
    page_bytes, n_pages = 1 << 20, 4100
    data = torch.empty(2, n_pages, page_bytes, dtype=torch.uint8, device="cuda")
    data[:, 4099] = 3
    data[1, 4099] = 5
    d = afx.page_data(data.data_ptr(), page_bytes, n_pages * page_bytes, 2)
    src, dst = ints([4099]), ints([4098])
    afx.afx_pages_copy_async(d, n_pages, 1, src.data_ptr(), dst.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert bool((data[0, 4098] == 3).all()) and bool((data[1, 4098] == 5).all())


def test_many_free_pages():
    """Counts over many blocks: free pages at the far end, then all of them moved to the front."""
    n = 300000
    c = Cache(8, 3, 9, n, planes=1, page_bytes=16, gap=0)
    c.refs[:n - 5] = 1
    c.model.refs[:n - 5] = [1] * (n - 5)
    slots, pos = ints([7] * 70), ints([7] * 70)
    a, b, granted = ints([1, 0]), ints([0, 60, 70]), ints([7, 7])
    ws = torch.empty(afx.afx_pages_extend_workspace(c.t, 2), dtype=torch.uint8, device="cuda")
    afx.afx_pages_extend_async(c.t, c.d, 2, a.data_ptr(), b.data_ptr(), 70, slots.data_ptr(), pos.data_ptr(),
                               granted.data_ptr(), ws.data_ptr(), ws.numel(), c.stream)
    want = c.model.extend([1, 0], [0, 60, 70], 70)
    torch.cuda.synchronize()
    assert (slots.tolist(), pos.tolist(), granted.tolist()) == want
    assert c.refs.tolist() == c.model.refs
    # every other page goes
    c.refs[:n - 5:2] = 0
    c.model.refs[:n - 5:2] = [0] * len(c.model.refs[:n - 5:2])
    moved, live = ints([7] * n), ints([7])
    ws = torch.empty(afx.afx_pages_compact_workspace(c.t), dtype=torch.uint8, device="cuda")
    afx.afx_pages_compact_async(c.t, c.d, moved.data_ptr(), live.data_ptr(), ws.data_ptr(), ws.numel(), c.stream)
    want = c.model.compact()
    torch.cuda.synchronize()
    assert (moved.tolist(), live.item()) == want
    assert c.refs.tolist() == c.model.refs and c.table[:, :9].tolist() == c.model.table
    src, dst = (torch.tensor(v, device="cuda") for v in zip(*c.model.copies))
    bytes_ = c.bytes.view(n, 16)
    bytes_[dst] = bytes_[src]
    assert torch.equal(c.data, c.bytes)


def test_captured_steps():
    """A captured step of generation: branches dropped, forked and grown at every replay."""
    c = Cache(9, 6, 8, 40)
    c.extend([0, 1], [20, 35])
    s = ints([0, 1, 1]), ints([2, 3, 4]), ints([0, 1, 2, 3])
    slots, pos, granted = ints([0] * 3), ints([0] * 3), ints([0] * 3)
    ws = torch.empty(afx.afx_pages_extend_workspace(c.t, 3), dtype=torch.uint8, device="cuda")

    def step(stream):
        afx.afx_pages_trim_async(c.t, 3, s[1].data_ptr(), 0, stream)
        afx.afx_pages_fork_async(c.t, 3, s[0].data_ptr(), s[1].data_ptr(), 0, stream)
        afx.afx_pages_extend_async(c.t, c.d, 3, s[1].data_ptr(), s[2].data_ptr(), 3, slots.data_ptr(), pos.data_ptr(),
                                   granted.data_ptr(), ws.data_ptr(), ws.numel(), stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream().cuda_stream)
    c.check()  # (capturing runs nothing)
    for src in ([0, 1, 1], [1, 1, 1], [0, 0, 1], [1, 0, 0]):
        s[0].copy_(ints(src))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        c.model.trim([2, 3, 4])
        c.model.fork(src, [2, 3, 4])
        want = c.model.extend([2, 3, 4], [0, 1, 2, 3], 3)
        c.check()
        assert (slots.tolist(), pos.tolist(), granted.tolist()) == want
