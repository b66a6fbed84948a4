"""The attention operators run together as attn.Attention and cache.PagedCache
call them: prompts, drafts, single tokens (captured and replayed), sequences
forked, trimmed, freed and compacted between them, against the formulas in 64
bits over the tokens that each sequence should hold.

Tolerance, of a result's norm. On the way from r to b, values are rounded to
BF16: xn; q and k; v; the weights; a. One rounding changes an array by at most
2^-8 of its norm, and random matrices and norms pass on that part of what they
are given. A score is a sum of products q_i k_i, each changed by two roundings
and by those of xn before them, independent of each other: with heads of norm
sqrt(dim) and the scale 1 / sqrt(dim), that is sqrt(4) 2^-8 / sqrt(3) times
sqrt(sum (q_i k_i)^2) / sqrt(dim), about 1.2 2^-8, so a weight, and with it the
outputs, by no more than two further roundings. b is thus within 8 roundings,
and r' = r + b within one more of its own, xn' again within one."""
import sys

import numpy as np
import pytest

import oracle
from lossless_bf16_weight_afx_amd import afx, attn, cache, synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D, HEADS, KV, DIM, EPS = 256, 4, 2, 64, 1e-6
STEP = 2.0 ** -8


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def norm(x, w=None):
    n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return n if w is None else n * w


class Layer:
    """One attention half and its formula."""

    def __init__(self, rng, c, layer, window=0):
        self.window, self.layer, mats = window, layer, []
        self.w = []
        for rows, cols in ((HEADS * DIM, D), (KV * DIM, D), (KV * DIM, D), (D, HEADS * DIM)):
            bits = synth.f32_to_bf16_bits((rng.standard_normal(rows * cols) * cols ** -0.5).astype(np.float32))
            blob = oracle.encode(bits, (rows, cols))
            mats.append((afx.afx_query(blob), afx.to_device(blob)))
            self.w.append(torch.from_numpy(synth.bf16_bits_to_f32(bits).reshape(rows, cols).astype(np.float64)))
        vec = lambda n: torch.from_numpy(1 + 0.1 * rng.standard_normal(n)).bfloat16().cuda()  # noqa: E731
        self.pre, self.wq, self.wk, self.nxt = vec(D), vec(DIM), vec(DIM), vec(D)
        self.freq = torch.tensor([100.0 ** (-i / 16) for i in range(16)], device="cuda")
        self.attn = attn.Attention(*mats, D, c, layer, HEADS, self.pre, w_q=self.wq, w_k=self.wk, freq=self.freq,
                                   w_next=self.nxt, eps=EPS, window=window)
        self.held = {}  # sequence: its keys and values, [tokens, KV, DIM] each

    def turn(self, x, pos):
        t = pos.double()[:, None, None] * self.freq.cpu().double()
        a, b, rest = x[..., :16], x[..., 16:32], x[..., 32:]
        return torch.cat([a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin(), rest], -1)

    def formula(self, r, rows):
        """r' and xn' of the new tokens of rows (sequence, tokens), which `held` gets."""
        vec = lambda t: t.cpu().double()  # noqa: E731
        xn = norm(r, vec(self.pre))
        q, k, v = (xn @ w.t() for w in self.w[:3])
        out, at = torch.zeros(r.shape[0], HEADS * DIM).double(), 0
        for s, n in rows:
            hk, hv = self.held.get(s, (torch.zeros(0, KV, DIM).double(),) * 2)
            pos = torch.arange(n) + hk.shape[0]
            rows_ = slice(at, at + n)
            qs = self.turn(norm(q[rows_].view(n, HEADS, DIM), vec(self.wq)), pos)
            hk = torch.cat([hk, self.turn(norm(k[rows_].view(n, KV, DIM), vec(self.wk)), pos)])
            hv = torch.cat([hv, v[rows_].view(n, KV, DIM)])
            self.held[s] = hk, hv
            there = torch.arange(hk.shape[0])
            seen = there[None] <= pos[:, None]
            if self.window:
                seen &= there[None] > pos[:, None] - self.window
            for h in range(HEADS):
                sc = (qs[:, h] @ hk[:, h // (HEADS // KV)].t() * DIM ** -0.5).masked_fill(~seen, -torch.inf)
                out[rows_, h * DIM:(h + 1) * DIM] = torch.softmax(sc, -1) @ hv[:, h // (HEADS // KV)]
            at += n
        r1 = r + out @ self.w[3].t()
        return r1, norm(r1, vec(self.nxt))


class Model:
    def __init__(self, seed, n_pages=64, page_tokens=16, **kw):
        self.rng = np.random.default_rng(seed)
        self.c = cache.PagedCache(2, KV, DIM, n_pages=n_pages, page_tokens=page_tokens, max_seqs=8, max_pages=16,
                                  max_tokens=160, **kw)
        self.c.data.fill_(float("nan"))  # what no token wrote is never used
        self.layers = [Layer(self.rng, self.c, 0), Layer(self.rng, self.c, 1, window=24)]

    def values(self, m):
        return torch.from_numpy(self.rng.standard_normal((m, D))).bfloat16().cuda()

    def step(self, r, seqs, starts, max_new=None):
        step = self.c.extend(seqs, starts, r.shape[0], max_new)
        got = []
        for t in self.layers:
            r, xn = t.attn.forward(r, step)
            got.append((r, xn))
        return step, got

    def compare(self, r, rows, got):
        r = r.cpu().double()
        for t, (r1, xn) in zip(self.layers, got):
            want, wxn = t.formula(r, rows)
            r1, xn = r1.cpu().double(), xn.cpu().double()
            err, b = (r1 - want).norm(), (want - r).norm()
            assert err <= 8 * STEP * b + STEP * want.norm(), f"layer {t.layer}: r' off by {float(err / b / STEP)} roundings"
            err = (xn - wxn).norm()
            assert err <= 10 * STEP * wxn.norm(), f"layer {t.layer}: xn' off by {float(err / wxn.norm() / STEP)} roundings"
            r = r1  # the next layer's own error

    def take(self, rows, max_new=None):
        """A step of rows (sequence, tokens), compared."""
        say("step", rows)
        starts = np.concatenate([[0], np.cumsum([n for _, n in rows])])
        r = self.values(int(starts[-1]))
        step, got = self.step(r, ints(*(s for s, _ in rows)), ints(*starts), max_new)
        assert step.granted.tolist() == [n for _, n in rows]
        self.compare(r, rows, got)

    def lengths(self):
        want = [self.layers[0].held[s][0].shape[0] if s in self.layers[0].held else 0 for s in range(self.c.max_seqs)]
        assert self.c.len.tolist() == want

    def keep(self, s, n):
        for t in self.layers:
            t.held[s] = tuple(x[:n] for x in t.held[s])

    def fork(self, a, b):
        for t in self.layers:
            t.held[b] = t.held[a]

    def drop(self, s):
        for t in self.layers:
            del t.held[s]


@pytest.mark.parametrize("page_tokens", [16, 32])
def test_generation(page_tokens):
    g = Model(page_tokens, page_tokens=page_tokens)
    g.take([(2, 37), (0, 5), (5, 70)])
    g.take([(0, 1), (2, 1), (5, 1)], 1)
    g.take([(5, 4), (2, 1), (0, 3)], 4)  # drafts
    assert g.c.fork(ints(2, 5), ints(1, 7)).tolist() == [1, 1]
    g.fork(2, 1), g.fork(5, 7)
    g.take([(1, 1), (2, 1), (5, 1), (7, 1), (0, 1)], 1)  # the copies part
    g.c.trim(ints(5, 1), ints(40, 33))  # drafts that were not taken
    g.keep(5, 40), g.keep(1, 33)
    g.take([(7, 2), (5, 1), (1, 3)], 3)
    g.c.free(ints(2, 0))
    g.drop(2), g.drop(0)
    where, live = g.c.compact()
    assert int(live) == int((g.c.refs > 0).sum()) and bool((g.c.refs[int(live):] == 0).all())
    g.lengths()
    g.take([(3, 100), (1, 1), (5, 1), (7, 1)])
    for _ in range(3):
        g.take([(1, 1), (3, 1), (5, 1), (7, 1)], 1)
    g.lengths()


def test_a_captured_step_is_replayed():
    """Lengths and pages move on in the graph; what the host does between the replays is seen by them."""
    g = Model(7)
    rows = [(0, 20), (3, 1), (6, 47)]
    g.take(rows)
    seqs, starts, r = ints(0, 3, 6), ints(0, 1, 2, 3), g.values(3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (once before the capture, as a step of its own)
        _, got = g.step(r, seqs, starts, 1)
    side.synchronize()
    ones = [(0, 1), (3, 1), (6, 1)]
    g.compare(r, ones, got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step, got = g.step(r, seqs, starts, 1)
    for i in range(20):
        say("replay", i)
        r.copy_(g.values(3))
        graph.replay()
        torch.cuda.synchronize()
        assert step.granted.tolist() == [1, 1, 1]
        g.compare(r, ones, got)
        if i == 6:
            g.c.trim(ints(6), ints(9))
            g.keep(6, 9)
        if i == 9:
            assert g.c.fork(ints(0), ints(1)).tolist() == [1]
            g.fork(0, 1)
            torch.cuda.synchronize()
        if i == 13:
            g.c.free(ints(3))
            for t in g.layers:
                t.held[3] = tuple(x[:0] for x in t.held[3])
            g.c.compact()
    g.lengths()


def test_a_refused_row_leaves_the_others():
    """Too few pages: the row, and those after it, get no slots; what the sequences hold stays."""
    g = Model(3, n_pages=4)
    g.take([(0, 30), (1, 16)])
    r = g.values(35)
    step, got = g.step(r, ints(0, 1, 2), ints(0, 2, 34, 35), 32)
    assert step.granted.tolist() == [2, 0, 0] and step.slots[2:].tolist() == [-1] * 33
    g.compare(r[:2], [(0, 2)], [(a[:2], b[:2]) for a, b in got])
    assert g.c.len.tolist()[:3] == [32, 16, 0]
    g.take([(1, 1)], 1)


def test_before_the_feed_forward_half():
    """r' of one half is the other's r, in place, as a layer has them."""
    from lossless_bf16_weight_afx_amd import ffn

    g = Model(11)
    mats, wide = [], []
    for rows, cols in ((512, D), (512, D), (D, 512)):
        bits = synth.f32_to_bf16_bits((g.rng.standard_normal(rows * cols) * cols ** -0.5).astype(np.float32))
        blob = oracle.encode(bits, (rows, cols))
        mats.append((afx.afx_query(blob), afx.to_device(blob)))
        wide.append(torch.from_numpy(synth.bf16_bits_to_f32(bits).reshape(rows, cols).astype(np.float64)))
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    block = ffn.FeedForward(*mats, D, 512, w, eps=EPS, max_tokens=160)
    for rows in ([(4, 33), (1, 8)], [(4, 1), (1, 1)]):
        starts = np.concatenate([[0], np.cumsum([n for _, n in rows])])
        r = g.values(int(starts[-1]))
        step = g.c.extend(ints(*(s for s, _ in rows)), ints(*starts), r.shape[0])
        r1, _ = g.layers[0].attn.forward(r, step)
        r2, _ = block.forward(r1)
        want, _ = g.layers[0].formula(r.cpu().double(), rows)
        r1 = r1.cpu().double()
        assert (r1 - want).norm() <= 8 * STEP * (want - r.cpu().double()).norm() + STEP * want.norm()
        xn = norm(r1)
        want = r1 + (torch.nn.functional.silu(xn @ wide[0].t()) * (xn @ wide[1].t())) @ wide[2].t()
        assert (r2.cpu().double() - want).norm() <= 3 * STEP * want.norm()
