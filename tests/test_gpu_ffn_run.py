"""The feed-forward operators run together: a layer's half (norm, gated
block, product, norm) and its gradients, as ffn.FeedForward calls them,
against the formulas and autograd in 64 bits.

Tolerance, of a result's norm. On the way to a result, values are rounded to
BF16 a known number of times; a rounding changes an array by at most 2^-8 of
its norm, and a random matrix, a norm or an activation near the origin passes
on about that part of what it is given, so n roundings come to at most n 2^-8
(FP32 sums add 2^-14 at these sizes). Forward: xn, h, r' (and xn'). Backward:
those of xn, h, r' and of g, u, db, dg, du, dxn, dr."""
import sys

import numpy as np
import pytest

import oracle
from blob_damage import KINDS, damage
from lossless_bf16_weight_afx_amd import afx, ffn, synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D, FF, EPS, SCALE = 256, 512, 1e-6, 0.7
STEP = 2.0 ** -8


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


class Coded:
    def __init__(self, rng, rows, cols, std):
        bits = synth.f32_to_bf16_bits((rng.standard_normal(rows * cols) * std).astype(np.float32))
        self.blob = oracle.encode(bits, (rows, cols))
        self.pair = (afx.afx_query(self.blob), afx.to_device(self.blob))
        self.w = torch.from_numpy(synth.bf16_bits_to_f32(bits).reshape(rows, cols).astype(np.float64))


class Block:
    def __init__(self, seed, max_tokens, post=True, gated=True, nxt=True, training=True):
        rng = self.rng = np.random.default_rng([seed, max_tokens])
        self.mats = [Coded(rng, FF, D, D ** -0.5), Coded(rng, FF, D, D ** -0.5), Coded(rng, D, FF, FF ** -0.5)]
        vec = lambda on: torch.from_numpy(1 + 0.2 * rng.standard_normal(D)).bfloat16().cuda() if on else None  # noqa: E731
        self.vectors = [vec(True), vec(post), vec(gated), vec(nxt)]
        w_pre, w_post, gate, w_next = self.vectors
        self.ffn = ffn.FeedForward(*(c.pair for c in self.mats), D, FF, w_pre, w_post=w_post, block_gate=gate,
                                   w_next=w_next, eps=EPS, scale=SCALE, max_tokens=max_tokens, training=training)

    def values(self, m, std=1.0):
        return torch.from_numpy(self.rng.standard_normal((m, D)) * std).bfloat16().cuda()

    def formula(self, r, dro=None, dxo=None):
        """r', xn' and the gradients of (r, w_pre, w_post, gate, w_next), all FP64."""
        r = r.cpu().double().requires_grad_()
        vec = [None if v is None else v.cpu().double().requires_grad_() for v in self.vectors]
        rms = lambda t: t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)  # noqa: E731
        wg, wu, wd = (c.w for c in self.mats)
        xn = rms(r) * vec[0]
        g, u = xn @ wg.t(), xn @ wu.t()
        b = (g / (1 + torch.exp(-g)) * u) @ wd.t()
        bh = b if vec[1] is None else rms(b) * vec[1]
        ro = r + SCALE * (bh if vec[2] is None else vec[2] * bh)
        xo = None if vec[3] is None else rms(ro) * vec[3]
        if dro is None:
            return ro.detach(), None if xo is None else xo.detach(), None
        loss = (ro * dro.cpu().double()).sum()
        if dxo is not None:
            loss = loss + (xo * dxo.cpu().double()).sum()
        loss.backward()
        grads = [None if v is None else v.grad for v in [r] + vec]
        return ro.detach(), None if xo is None else xo.detach(), grads


def near(name, got, want, roundings):
    got = got.detach().cpu().double()
    assert bool(torch.isfinite(got).all()), name
    want = want.detach()
    err = float((got - want).norm() / want.norm())
    say(f"[gpu]   {name}: error {err:.3g} of the norm, bound {roundings * STEP:.3g}")
    assert err <= roundings * STEP, f"{name}: {err}"


@pytest.mark.parametrize("m", [1, 2, 3, 5, 16, 33, 64, 65, 129, 300])
@pytest.mark.parametrize("post,gated,nxt", [(True, True, True), (False, False, False), (True, False, True)])
def test_run_and_gradients(m, post, gated, nxt):
    say(f"[gpu] case feed-forward run m={m} post={post} gate={gated} next={nxt}")
    t = Block(3, m, post, gated, nxt)
    r, dro, dxo = t.values(m, 1.5), t.values(m), t.values(m) if nxt else None
    ro, xo = t.ffn.forward(r)
    dr = t.ffn.backward(r, dro, dxo)
    torch.cuda.synchronize()
    want_ro, want_xo, grads = t.formula(r, dro, dxo)
    near("r'", ro, want_ro, 3)
    if nxt:
        near("xn'", xo, want_xo, 4)
    else:
        assert xo is None
    for name, got, want in zip(("dr", "dw_pre", "dw_post", "dgate", "dw_next"),
                               (dr, t.ffn.dw_pre, t.ffn.dw_post, t.ffn.dgate, t.ffn.dw_next), grads):
        assert (got is None) == (want is None)
        if got is not None:
            near(name, got, want, 10)


def test_fewer_tokens_than_the_buffers_and_a_strided_stream():
    """The rows behind the last token stay as they were; r may be a column
    range of a wider tensor, and one row's stride anything."""
    t = Block(4, 40)
    wide = torch.full((7, 2 * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    r = wide[:, :D]
    r.copy_(t.values(7))
    keep = [t.ffn.xn, t.ffn.h, t.ffn.b, t.ffn.r_out, t.ffn.xn_next, t.ffn.g, t.ffn.u, t.ffn.dr, t.ffn.dh, t.ffn.dxn]
    for k in keep:
        k.fill_(-7.0)
    dro = t.values(7)
    ro, xo = t.ffn.forward(r)
    t.ffn.backward(r, dro)
    torch.cuda.synchronize()
    want, want_x, _ = t.formula(r)
    near("r'", ro, want, 3)
    near("xn'", xo, want_x, 4)
    for k in keep:
        assert bool((k[7:] == -7.0).all())
    one = r[2:3].t().contiguous().t()  # a row whose own stride is 1
    ro, _ = t.ffn.forward(one)
    near("one row", ro, want[2:3], 3)


def test_two_blocks_in_a_graph():
    """Two layers' halves, forward and backward, in one graph; replays on new
    inputs, between eager work, against the formulas. (The down product adds
    its parts in any order, so its sums' last bits may differ from run to run.)"""
    m = 20
    a, b = Block(5, m), Block(6, m)
    r, dro, dxo = a.values(m), a.values(m), a.values(m)

    def step():
        ra, _ = a.ffn.forward(r)
        b.ffn.forward(ra)
        a.ffn.backward(r, b.ffn.backward(ra, dro, dxo))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for x in (r, dro, dxo):
            x.copy_(a.values(m))
        a.values(m).float().sum()  # eager work between the replays
        torch.cuda.synchronize()
        for k in (a.ffn.dr, a.ffn.r_out, b.ffn.r_out, b.ffn.dr, a.ffn.dw_pre):
            k.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        ra, _, _ = a.formula(r)
        rb, _, gb = b.formula(ra, dro, dxo)
        near("r' of the first", a.ffn.r_out, ra, 3)
        near("r' of the second", b.ffn.r_out, rb, 6)
        _, _, ga = a.formula(r, gb[0])
        near("dr of the second", b.ffn.dr, gb[0], 13)
        near("dr of the first", a.ffn.dr, ga[0], 23)
        near("dw_pre of the first", a.ffn.dw_pre, ga[1], 23)


def test_streams_take_turns():
    """One object on two streams, ordered by events."""
    t = Block(8, 24)
    r1, r2 = t.values(24), t.values(24)
    side = torch.cuda.Stream()
    ro, _ = t.ffn.forward(r1)
    first = ro.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ro, _ = t.ffn.forward(r2)
        second = ro.clone()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    near("first", first, t.formula(r1)[0], 3)
    near("second", second, t.formula(r2)[0], 3)


def test_refusals():
    t = Block(9, 8, nxt=False, training=False)
    r = t.values(8)
    for bad in (t.values(9), r[:0], r.float(), r[:, :-1], torch.empty(8, D, dtype=torch.bfloat16), r[0],
                torch.empty(D, 8, dtype=torch.bfloat16, device="cuda").t()):
        with pytest.raises(ValueError):
            t.ffn.forward(bad)
    with pytest.raises(ValueError):
        t.ffn.backward(r, r)
    t = Block(9, 8, nxt=False)
    t.ffn.forward(r)
    for grads in ((r[:7],), (r, r), (r.float(),)):
        with pytest.raises(ValueError):
            t.ffn.backward(r, *grads)
    with pytest.raises(afx.AfxError):
        t.ffn.forward(r[:1].expand(8, D))  # rows that share memory
    mats, w = [c.pair for c in t.mats], t.vectors[0]
    for bad in (dict(d=D + 8), dict(ff=FF - 256), dict(max_tokens=0), dict(w_pre=w.float()), dict(w_pre=w[:-1]),
                dict(w_next=w.cpu()), dict(block_gate=torch.ones(2 * D, dtype=torch.bfloat16, device="cuda")[::2])):
        with pytest.raises(ValueError):
            ffn.FeedForward(*mats, **{**dict(d=D, ff=FF, w_pre=w, max_tokens=8), **bad})


def test_workspace_is_the_largest_of_all_token_counts():
    """A size between the ones the constructor looks at never needs more."""
    t = Block(10, 700)
    need = 0
    for m in range(1, 701):
        need = max(need, afx.afx_restore_gated_workspace(FF, D, m), afx.afx_restore_gated_workspace(FF, D, m, True),
                   afx.afx_restore_gemm_t_workspace(D, FF, m), afx.afx_block_norm_workspace(t.ffn.norm_in, m),
                   afx.afx_block_norm_workspace(t.ffn.norm_out, m))
    assert t.ffn.ws.numel() == need


@pytest.mark.parametrize("cols", [1312, 1320])
@pytest.mark.parametrize("m", [1, 4, 16, 64, 100, 150])
@pytest.mark.parametrize("what", KINDS)
def test_damaged_device_blobs_stay_in_bounds(what, m, cols):
    """Device copies that differ from the validated host blobs give wrong
    results, never an access out of bounds: guards around every output stay."""
    say(f"[gpu] case damaged blob: {what}, m={m}")
    rng = np.random.default_rng([KINDS.index(what), m, 11])
    rows = 144  # ends inside a tile of rows, as the columns do inside a slab
    mats = [Coded(rng, rows, cols, 0.05) for _ in range(2)]
    (gi, _), (ui, _) = (c.pair for c in mats)
    bad = [afx.to_device(damage(c.blob, what, rng)) for c in mats]
    guard, mark = 256, -7.0

    def guarded(n, dtype):
        return torch.full((n + 2 * guard,), mark, dtype=dtype, device="cuda")

    def intact(t):
        return bool((t[:guard] == mark).all() and (t[-guard:] == mark).all())

    at = lambda t: t.data_ptr() + guard * t.element_size()  # noqa: E731
    x = torch.from_numpy(rng.standard_normal((m, cols))).bfloat16().cuda()
    d = torch.from_numpy(rng.standard_normal((m, rows))).bfloat16().cuda()
    dh = torch.from_numpy(rng.standard_normal((m, rows))).float().cuda()
    h, g, u = (guarded(m * rows, torch.bfloat16) for _ in range(3))
    dx, y = guarded(m * cols, torch.bfloat16), guarded(m * cols, torch.float32)
    need = max(afx.afx_restore_gated_workspace(rows, cols, m), afx.afx_restore_gated_workspace(rows, cols, m, True),
               afx.afx_restore_gemm_t_workspace(rows, cols, m))
    ws = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
    ws[need:] = 0x5A
    w = afx.gated_weights(gi, bad[0].data_ptr(), ui, bad[1].data_ptr(), rows, cols)
    s = torch.cuda.current_stream().cuda_stream
    afx.afx_restore_gated_async(w, m, x.data_ptr(), cols, at(h), rows, at(g), at(u), rows, ws.data_ptr(), need, s)
    afx.afx_restore_gated_backward_async(w, m, dh.data_ptr(), rows, at(g), at(u), rows, at(dx), cols, 0, 0,
                                         ws.data_ptr(), need, s)
    afx.afx_restore_gemm_t_async(gi, bad[0].data_ptr(), rows, cols, d.data_ptr(), m, at(y), False, ws.data_ptr(),
                                 need, s)
    torch.cuda.synchronize()
    for t in (h, g, u, dx, y):
        assert intact(t)
    assert bool((ws[need:] == 0x5A).all())
