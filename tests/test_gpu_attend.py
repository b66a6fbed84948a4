"""Attention of new tokens over a paged cache against the definition in 64
bits, within bounds that tests/paged_reference.py derives."""
import math

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


class Batch:
    """Sequences of given lengths in a cache whose other places hold NaN, and
    new tokens of batch rows: (sequence, new tokens) each."""

    def __init__(self, seed, lens, rows, *, kv_heads=2, group=2, dim=64, page=16, spread=1.0, behind=3, gap=0):
        self.gen = torch.Generator().manual_seed(seed)
        self.lens, self.rows = lens, rows
        self.kv_heads, self.group, self.dim, self.page, self.gap = kv_heads, group, dim, page, gap
        need = [-(-n // page) for n in lens]
        self.n_pages, wide = sum(need) + 2, max(max(need), 1) + 1
        order = torch.randperm(self.n_pages, generator=self.gen).tolist()
        self.table = torch.full((len(lens), wide), -1, dtype=torch.int32)
        self.k = torch.full((self.n_pages, kv_heads, dim // 8, page, 8), math.nan, dtype=torch.bfloat16)
        self.v = torch.full((self.n_pages, kv_heads, page // 8, dim, 8), math.nan, dtype=torch.bfloat16)
        self.keys, self.values = [], []
        for s, n in enumerate(lens):
            ids, order = order[:need[s]], order[need[s]:]
            self.table[s, :need[s]] = torch.tensor(ids, dtype=torch.int32)
            self.keys.append(self.normal(n, kv_heads, dim, std=spread))
            self.values.append(self.normal(n, kv_heads, dim))
        self.m = sum(n for _, n in rows)
        starts = [0]
        for _, n in rows:
            starts.append(starts[-1] + n)
        self.starts = torch.tensor(starts, dtype=torch.int32)
        self.m_all = self.m + behind  # rows behind the last new token
        self.q = self.normal(self.m_all, kv_heads * group * dim + gap, std=spread)
        self.there = [torch.ones(n, dtype=torch.bool) for n in lens]

    def normal(self, *shape, std=1.0):
        return (torch.randn(*shape, generator=self.gen) * std).bfloat16()

    def upload(self):
        for s, n in enumerate(self.lens):
            j = torch.arange(n)
            ids, off = self.table[s, j // self.page].long(), j % self.page
            ok = (ids >= 0) & (ids < self.n_pages)
            ref.k_to_pages(self.keys[s][ok], ids[ok], off[ok], self.k)
            ref.v_to_pages(self.values[s][ok], ids[ok], off[ok], self.v)
        self.dev = {n: getattr(self, n).cuda() for n in ("k", "v", "table", "q", "starts")}
        self.dev["len"] = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.dev["seqs"] = torch.tensor([s for s, _ in self.rows], dtype=torch.int32, device="cuda")
        width = self.kv_heads * self.group * self.dim
        self.out = torch.full((self.m_all, width + self.gap), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.m_all, self.kv_heads * self.group), 7.0, device="cuda")

    def args(self, *, scale, causal=True, window=0, max_new=None, max_len=None, seqs=True):
        d = self.dev
        kv = afx.kv_pages(d["k"].data_ptr(), d["v"].data_ptr(), self.n_pages, self.page, self.kv_heads, self.dim)
        t = afx.page_table(d["table"].data_ptr(), d["table"].stride(0), d["len"].data_ptr(), 0, len(self.lens),
                           d["table"].shape[1], self.n_pages, self.page)
        p = afx.attend(self.kv_heads * self.group, scale, causal, window,
                       max(n for _, n in self.rows) if max_new is None else max_new,
                       max(self.lens) if max_len is None else max_len)
        ws = torch.empty(max(16, afx.afx_attend_workspace(p, kv, len(self.rows), self.m_all)), dtype=torch.uint8,
                         device="cuda")
        return (p, kv, t, len(self.rows), d["seqs"].data_ptr() if seqs else 0, d["starts"].data_ptr(), self.m_all,
                d["q"].data_ptr(), d["q"].stride(0), self.out.data_ptr(), self.out.stride(0), self.lse.data_ptr(),
                ws.data_ptr(), ws.numel()), (p, kv, t, ws)

    def run(self, **how):
        self.how = how
        args, keep = self.args(**how)
        afx.afx_attend_async(*args, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        del keep

    def want(self):
        """Output, log-sum-exp and their bounds, [m, heads, ..]."""
        scale, causal, window = self.how["scale"], self.how.get("causal", True), self.how.get("window", 0)
        heads = self.kv_heads * self.group
        out, lse = torch.zeros(self.m, heads, self.dim).double(), torch.full((self.m, heads), -math.inf).double()
        bound, lbound = torch.full_like(out, 1e-30), torch.full_like(lse, 1e-30)
        for r, (s, n) in enumerate(self.rows):
            if n == 0 or not 0 <= s < len(self.lens) or self.lens[s] == 0:
                continue
            at = torch.arange(n) + self.lens[s] - n
            lo = (at - window + 1).clamp(min=0) if window else torch.zeros_like(at)
            hi = at + 1 if causal else torch.full_like(at, self.lens[s])
            rows = slice(int(self.starts[r]), int(self.starts[r]) + n)
            for h in range(heads):
                g = h // self.group
                q = self.q[rows, h * self.dim:(h + 1) * self.dim]
                out[rows, h], lse[rows, h], bound[rows, h], lbound[rows, h] = ref.attend(
                    q, self.keys[s][:, g], self.values[s][:, g], self.there[s], lo, hi, scale)
        return out, lse, bound, lbound

    def check(self):
        out, lse, bound, lbound = self.want()
        width = self.kv_heads * self.group * self.dim
        got, gl = self.out.cpu().double(), self.lse.cpu().double()
        o = got[:self.m, :width].reshape(out.shape)
        odd = ~torch.isfinite(out)
        assert torch.equal(torch.isnan(o), torch.isnan(out)), "NaN where none belongs, or none where one does"
        sure = odd & ~torch.isnan(out)
        assert torch.equal(o[sure], out[sure])
        err = ((o - out).abs() / bound)[~odd]
        assert err.numel() == 0 or float(err.max()) <= 1, f"output off by {float(err.max())} of its bound"
        none = lse == -math.inf
        assert torch.equal(gl[:self.m][none], lse[none])
        err = ((gl[:self.m] - lse).abs() / lbound)[torch.isfinite(lse)]
        assert err.numel() == 0 or float(err.max()) <= 1, f"lse off by {float(err.max())} of its bound"
        assert bool((got[self.m:] == 7).all()) and bool((gl[self.m:] == 7).all()), "rows behind the last were written"
        assert bool((got[:, width:] == 7).all()), "values between the rows were written"


@pytest.mark.parametrize("dim", [8, 16, 40, 64, 72, 80, 96, 104, 128, 136, 192, 248, 256])
@pytest.mark.parametrize("new", [1, 3, 70])
def test_head_sizes(dim, new):
    lens = [200, 71, 97]
    b = Batch(dim + new, lens, [(0, new), (2, 1), (1, min(new, 71))], dim=dim, kv_heads=2, group=3, gap=8)
    b.upload()
    b.run(scale=dim ** -0.5)
    b.check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("kv_heads, group", [(1, 1), (1, 5), (8, 5), (3, 16), (1, 17), (2, 40), (1, 256)])
def test_pages_and_groups(page, kv_heads, group):
    n = 1 if group > 40 else 2
    b = Batch(page + group, [333, 1, 64], [(0, n), (1, 1), (2, n)], kv_heads=kv_heads, group=group, page=page)
    b.upload()
    b.run(scale=0.125)
    b.check()


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513, 1000])
@pytest.mark.parametrize("new", [1, 40])
def test_lengths(length, new):
    b = Batch(length, [length, 5], [(0, min(new, length)), (1, 1)], kv_heads=1, group=4)
    b.upload()
    b.run(scale=0.125)
    b.check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 2, 33, 64, 100, 10 ** 6, 2 ** 32 - 1])
@pytest.mark.parametrize("new", [1, 6, 90])
def test_masks(causal, window, new):
    b = Batch(window % 1000 + new, [300, 90, 500], [(2, new), (0, new), (1, new), (2, 0)], group=2)
    b.upload()
    b.run(scale=0.125, causal=causal, window=window)
    b.check()


@pytest.mark.parametrize("new", [5, 80])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(new, causal):
    """More new tokens than the sequence holds (the first stand before its
    start), empty sequences, sequences outside the table, rows without new tokens."""
    b = Batch(5, [3, 0, 40], [(0, new), (1, new), (-1, 2), (3, new), (2, 0), (2 ** 30, 1), (2, new)])
    b.upload()
    b.run(scale=0.125, causal=causal)
    b.check()


@pytest.mark.parametrize("max_new, max_len", [(1, 1), (1, 100000), (3000, 1), (100, 3000), (2 ** 32 - 1, 2 ** 32 - 1)])
def test_sizes_given_wrong(max_new, max_len):
    b = Batch(6, [700, 1300, 64], [(0, 50), (1, 1), (2, 9)], kv_heads=1, group=3)
    b.upload()
    b.run(scale=0.125, max_new=max_new, max_len=max_len)
    b.check()


@pytest.mark.parametrize("length, new", [(9000, 1), (9000, 4), (5000, 64)])
def test_long_sequences_in_parts(length, new):
    b = Batch(length + new, [length, 300], [(0, new), (1, 1)], kv_heads=1, group=4, page=64, spread=1.5)
    b.upload()
    b.run(scale=0.125)
    b.check()


@pytest.mark.parametrize("length", [900, 1000, 1500, 2000, 3000, 4000])
@pytest.mark.parametrize("new, window", [(50, 0), (140, 0), (140, 700)])
def test_any_number_of_parts(length, new, window):
    """Numbers of parts that do not divide the tiles, rows that see nothing of some of them."""
    b = Batch(length + new + window, [length, 260], [(0, new), (1, 40)], kv_heads=2, group=3, dim=64, page=32, spread=1.5)
    b.upload()
    b.run(scale=0.125, window=window)
    b.check()


@pytest.mark.parametrize("new", [1, 60])
def test_scores_that_rise_and_fall(new):
    """Keys that grow along the sequence move the running maximum at every
    tile; others that shrink, never after the first."""
    b = Batch(8, [600, 600], [(0, new), (1, new)], kv_heads=1, group=2)
    ramp = torch.linspace(0.01, 1.0, 600)[:, None, None]
    for s, r in ((0, ramp), (1, ramp.flip(0))):
        b.keys[s] = (b.q[0, :64].float() * r * 1.2).reshape(600, 1, 64).bfloat16()
    b.upload()
    b.run(scale=0.125)
    b.check()


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-30, 3.0])
@pytest.mark.parametrize("new", [2, 50])
def test_scales(scale, new):
    b = Batch(9, [120, 77], [(0, new), (1, 3)], kv_heads=1, group=2)
    b.upload()
    b.run(scale=scale)
    b.check()


@pytest.mark.parametrize("new", [1, 2, 6, 100])
@pytest.mark.parametrize("causal, window", [(True, 0), (True, 20), (False, 20)])
def test_infinities_and_nan_reach_only_those_who_see_them(new, causal, window):
    b = Batch(10 + new, [150, 260], [(0, new), (1, min(new, 100))], kv_heads=2, group=2, dim=40)
    for s, length in enumerate(b.lens):
        for back, value in ((1, math.nan), (new // 2 + 1, math.inf), (new, -math.inf), (new + 10, math.nan), (60, math.inf)):
            b.values[s][length - back, s % 2, back % 40] = value
        b.keys[s][length - 1 - new // 3, 1, 3] = math.nan
    b.upload()
    b.run(scale=0.125, causal=causal, window=window)
    b.check()


def test_scores_of_minus_infinity():
    """Keys whose scores are minus infinity weigh nothing; a query with no
    other gets zeros."""
    b = Batch(11, [70, 40], [(0, 1), (1, 30)], kv_heads=1, group=1)
    b.q[:, 0] = 1.0
    for s in range(2):
        b.keys[s][5:, 0, 0] = -math.inf
        b.keys[s][5:, 0, 1:] = 0.0
    b.keys[1][:, 0, 0] = -math.inf
    b.keys[1][:, 0, 1:] = 0.0
    b.upload()
    b.run(scale=0.125)
    b.check()


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("page", [16, 128])
def test_pages_outside_the_cache_are_seen_by_none(new, page):
    b = Batch(12, [3 * page + 5, 2 * page, 50], [(0, new), (1, new), (2, 1)], page=page)
    b.table[0, 1] = -1
    b.table[0, 3] = b.n_pages
    b.there[0][page:2 * page] = False
    b.there[0][3 * page:] = False
    b.table[1, :2] = torch.tensor([2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    b.there[1][:] = False
    b.upload()
    b.run(scale=0.125)
    b.check()


@pytest.mark.parametrize("new", [1, 60])
def test_lengths_and_starts_out_of_range(new):
    """Lengths are capped at max_pages pages, starts at m; negative ones are 0."""
    b = Batch(13, [100, 20], [(0, new), (1, 3)])
    b.upload()
    wide = b.table.shape[1]
    b.dev["len"][:] = torch.tensor([2 ** 31 - 1, -5])
    b.dev["starts"][2] = 2 ** 31 - 1
    b.run(scale=0.125)
    # row 0: its sequence as if it filled the table; row 1: nothing, for all rows from its start on
    full = wide * 16
    for name in ("keys", "values"):
        t = getattr(b, name)
        t[0] = torch.cat((t[0], torch.full((full - 100, 2, 64), math.nan, dtype=torch.bfloat16)))
    seen = torch.zeros(full, dtype=torch.bool)
    b.lens = [full, 0]
    b.there = [seen, torch.ones(0, dtype=torch.bool)]
    pages = b.table[0]
    for i, page in enumerate(pages.tolist()):
        if page >= 0:
            seen[16 * i:16 * i + 16] = True
    seen &= torch.arange(full) < 112  # (behind 100 tokens the last page holds NaN)
    got = b.out.cpu().double()
    want, _, bound, _ = b.want()
    # (queries that stand behind the sequence's 100 tokens see the NaN of the last page's tail)
    o = got[:new].reshape(want[:new].shape)
    nan = torch.isnan(want[:new])
    assert bool(nan[-1].all()) and torch.equal(torch.isnan(o), nan)
    assert bool(((o - want[:new]).abs() <= bound[:new])[~nan].all())
    assert bool((got[new:] == 0).all())


def test_far_pages():
    """Offsets above 2^32 elements."""
    page, heads, dim = 256, 8, 256
    n_pages = 2 ** 32 // (page * heads * dim) + 3
    b = Batch(14, [700, 90], [(0, 1), (1, 50)], kv_heads=heads, group=1, dim=dim, page=page)
    far = torch.arange(b.n_pages) + n_pages - b.n_pages
    b.upload()
    small, want_table = {n: b.dev[n] for n in "kv"}, b.dev["table"]
    for n in "kv":
        b.dev[n] = torch.empty((n_pages, *small[n].shape[1:]), dtype=torch.bfloat16, device="cuda")
        b.dev[n][far.cuda()] = small[n]
    b.dev["table"] = torch.where(want_table >= 0, want_table + int(far[0]), want_table)
    b.n_pages = n_pages
    b.run(scale=0.0625)
    b.check()


def test_same_bits_on_every_run_and_beside_another_call():
    """Two calls at once on two streams, each with its workspace."""
    a = Batch(15, [3000, 40, 700], [(0, 70), (1, 1), (2, 5)], kv_heads=2, group=3)
    c = Batch(16, [5000], [(0, 1)], kv_heads=2, group=4)
    for b in (a, c):
        b.upload()
        b.run(scale=0.125)
        b.check()
    first = [(b.out.clone(), b.lse.clone()) for b in (a, c)]
    held = [b.args(scale=0.125) for b in (a, c)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for b, s, (args, _) in zip((a, c), streams, held):
            with torch.cuda.stream(s):
                b.out.fill_(7)
                afx.afx_attend_async(*args, s.cuda_stream)
        torch.cuda.synchronize()
        for b, (o, l) in zip((a, c), first):
            assert torch.equal(b.out, o) and torch.equal(b.lse, l)


@pytest.mark.parametrize("new", [1, 33])
def test_captured_and_replayed(new):
    """A graph reads lengths, tables and starts when it is replayed."""
    b = Batch(17, [900, 300], [(0, new), (1, 1)], kv_heads=1, group=4)
    b.upload()
    args, keep = b.args(scale=0.125)
    b.how = dict(scale=0.125)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        afx.afx_attend_async(*args, s.cuda_stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        afx.afx_attend_async(*args, torch.cuda.current_stream().cuda_stream)
    keys, values, there = b.keys[0], b.values[0], b.there[0]
    for length in (900, 500, 41, 899):
        b.dev["len"][0] = length
        b.lens[0] = length
        b.keys[0], b.values[0], b.there[0] = keys[:length], values[:length], there[:length]
        b.dev["q"].copy_(b.q)
        b.out.fill_(7)
        b.lse.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        b.check()
    del keep


def test_sequences_in_order_without_a_list():
    b = Batch(18, [50, 60, 70], [(0, 2), (1, 1), (2, 3)])
    b.upload()
    b.run(scale=0.125, seqs=False)
    b.check()
