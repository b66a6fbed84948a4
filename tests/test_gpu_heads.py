"""Norms and rotary positions of heads, their gradients, and the write to the
cache's pages, against the formulas in 64 bits.

Bounds. A head's sum of squares has at most dim roundings, its root, the
products with the weight and the rotation a few more; an angle's fraction of a
turn is off by 2^-25 of it, sine and cosine by 2^-22 at most: e below is
relative to the two values that a rotation adds. Each output is rounded to
BF16 once (2^-8)."""
import math

import pytest

import paged_reference as ref
from lossless_bf16_weight_afx_amd import afx

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
U, EPS = ref.U, 1e-6


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


class Heads:
    def __init__(self, seed, m, dim, rot, *, q_heads=3, kv_heads=2, pairing=afx.ROPE_HALVES, axes=1, w_q=True, w_k=True,
                 page=16, shift=0, gap=0, first=1000):
        self.gen = torch.Generator().manual_seed(seed)
        self.m, self.dim, self.rot, self.q_heads, self.kv_heads = m, dim, rot, q_heads, kv_heads
        self.pairing, self.axes, self.page = pairing, axes, page
        # q, k and v: column ranges of one wider matrix, which may start off 16 bytes
        wide = (q_heads + 2 * kv_heads) * dim + gap
        self.qkv = self.host(m, wide + shift, std=1.5)[:, shift:] if m else torch.zeros(0, wide)
        cuts = [q_heads * dim, (q_heads + kv_heads) * dim, (q_heads + 2 * kv_heads) * dim]
        self.x = {"q": self.qkv[:, :cuts[0]], "k": self.qkv[:, cuts[0]:cuts[1]], "v": self.qkv[:, cuts[1]:cuts[2]]}
        self.dy = {n: self.host(m, self.x[n].shape[1] + gap).bfloat16()[:, :self.x[n].shape[1]] for n in "qk"}
        self.w = {"q": (self.host(dim, std=0.3) + 1).bfloat16() if w_q else None,
                  "k": (self.host(dim, std=0.3) + 1).bfloat16() if w_k else None}
        self.pos = torch.randint(-first, 3 * first, (axes, m + 5), generator=self.gen).int()
        self.freq = (1e6 ** (-torch.arange(rot // 2) / max(rot // 2, 1))).float()
        self.axis = torch.randint(0, axes, (rot // 2,), generator=self.gen).to(torch.uint8) if axes > 1 else None
        self.n_pages = m // page + 3
        self.slots = torch.randperm(self.n_pages * page, generator=self.gen)[:m].int()

    def host(self, *shape, std=1.0):
        return torch.randn(*shape, generator=self.gen) * std

    def params(self):
        self.kept = {n: t.cuda() for n, t in (("w_q", self.w["q"]), ("w_k", self.w["k"]), ("freq", self.freq),
                                              ("axis", self.axis)) if t is not None and t.numel()}
        at = lambda n: self.kept[n].data_ptr() if n in self.kept else 0  # noqa: E731
        return afx.heads(self.q_heads, self.kv_heads, self.dim, self.rot, self.pairing, self.axes, EPS, at("w_q"),
                         at("w_k"), at("freq"), at("axis"))

    def angles(self):
        """Cosines and sines [m, rot / 2] in 64 bits."""
        axis = self.axis.long().clamp(max=self.axes - 1) if self.axis is not None else torch.zeros(self.rot // 2).long()
        t = self.pos[axis, :self.m].double().t() * self.freq.double()
        return torch.cos(t), torch.sin(t)

    def halves(self):
        r = self.rot
        return (slice(0, r // 2), slice(r // 2, r)) if self.pairing == afx.ROPE_HALVES else (slice(0, r, 2), slice(1, r, 2))

    def turn(self, x, sign=1.0):
        """Turned heads, and the size of the values that each is made of."""
        (c, s), (a, b) = self.angles(), self.halves()
        y, size = x.clone(), x.abs()
        y[..., a] = x[..., a] * c[:, None] - sign * x[..., b] * s[:, None]
        y[..., b] = x[..., b] * c[:, None] + sign * x[..., a] * s[:, None]
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
        return y, size

    def want(self, n):
        x = self.x[n].double().reshape(self.m, -1, self.dim)
        if self.w[n] is not None:
            x = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * self.w[n].double()
        y, size = self.turn(x)
        return y, ((self.dim + 8) * U + 2.0 ** -21) * size + 2.0 ** -8 * y.abs() + 1e-30

    def want_grad(self, n):
        """dx, its bound, dw, its bound."""
        x = self.x[n].double().reshape(self.m, -1, self.dim)
        dm, size = self.turn(self.dy[n].double().reshape(self.m, -1, self.dim), -1.0)
        e = 2 * (self.dim + 8) * U + 2.0 ** -20
        if self.w[n] is None:
            return dm, e * size + 2.0 ** -8 * dm.abs() + 1e-30, None, None
        w = self.w[n].double()
        k = 1 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        nh = x * k
        dx = k * (dm * w - nh * (dm * w * nh).mean(-1, keepdim=True))
        near = k * e * (size * w.abs() + nh.abs() * (size * w.abs() * nh.abs()).mean(-1, keepdim=True))
        terms = self.m * x.shape[1]
        return (dx, near + 2.0 ** -8 * dx.abs() + 1e-30, (dm * nh).sum((0, 1)),
                (size * nh.abs()).sum((0, 1)) * (e + 2 * terms * U) + 1e-30)


def near(name, got, want, bound):
    ok = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), ok), name
    err = float(((got.double() - want).abs() / bound)[ok].max()) if bool(ok.any()) else 0.0
    assert err <= 1, f"{name} is off by {err} of its bound"


def forward(t, *, dense=True, parts="qkv", stream=None):
    p, m, d = t.params(), t.m, t.dim
    x = {n: t.qkv.cuda() if n == "q" else None for n in "q"}["q"]
    cut = {"q": 0, "k": t.q_heads * d, "v": (t.q_heads + t.kv_heads) * d}
    at = lambda n: x.data_ptr() + 4 * cut[n] if n in parts else 0  # noqa: E731
    shape = {"q": (m, t.q_heads * d + 8), "k": (m, t.kv_heads * d + 8)}
    out = {n: torch.full(shape[n], 7.0, dtype=torch.bfloat16, device="cuda") for n in "qk"}
    pages = [torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for s in (
        (t.n_pages, t.kv_heads, d // 8, t.page, 8), (t.n_pages, t.kv_heads, t.page // 8, d, 8))]
    kv = afx.kv_pages(pages[0].data_ptr(), pages[1].data_ptr(), t.n_pages, t.page, t.kv_heads, d)
    pos, slots = t.pos.cuda(), t.slots.cuda()
    afx.afx_heads_async(p, m, pos.data_ptr(), pos.stride(0), at("q"), x.stride(0), at("k"), x.stride(0), at("v"),
                        x.stride(0), out["q"].data_ptr() if "q" in parts else 0, out["q"].stride(0),
                        out["k"].data_ptr() if dense and "k" in parts else 0, out["k"].stride(0),
                        kv if set(parts) & {"k", "v"} else None, slots.data_ptr() if set(parts) & {"k", "v"} else 0,
                        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return out, pages


def check(t, out, pages, dense=True, parts="qkv"):
    m, d = t.m, t.dim
    size = {"q": t.q_heads * d, "k": t.kv_heads * d}
    got = {n: o.cpu() for n, o in out.items()}
    want = {n: t.want(n) for n in "qk"}
    for n in "qk":
        if n in parts and (n == "q" or dense):
            near(n, got[n][:, :size[n]].reshape(m, -1, d), *want[n])
            assert bool((got[n][:, size[n]:] == 7).all())
        else:
            assert bool((got[n] == 7).all())
    k, v = (p.cpu() for p in pages)
    ok = (t.slots >= 0) & (t.slots < t.n_pages * t.page)
    page, off = t.slots[ok].long() // t.page, t.slots[ok].long() % t.page
    if "k" in parts:
        near("cached k", k[page, :, :, off].reshape(-1, t.kv_heads, d), want["k"][0][ok], want["k"][1][ok])
    if "v" in parts:
        assert torch.equal(v[page, :, off // 8, :, off % 8], t.x["v"][ok].reshape(-1, t.kv_heads, d).bfloat16())
    for name, cache, put in (("k", k, ref.k_to_pages), ("v", v, ref.v_to_pages)):  # nothing else was written
        if name in parts:
            put(torch.full((len(page), t.kv_heads, d), 7.0, dtype=torch.bfloat16), page, off, cache)
        assert bool((cache == 7).all())


SIZES = [(8, 8), (16, 8), (64, 64), (64, 0), (72, 36), (80, 40), (80, 20), (96, 96), (128, 128), (128, 64), (136, 10),
         (192, 192), (256, 256), (256, 64)]


@pytest.mark.parametrize("dim, rot", SIZES)
@pytest.mark.parametrize("pairing", [afx.ROPE_HALVES, afx.ROPE_NEIGHBOURS])
@pytest.mark.parametrize("m", [1, 37])
def test_sizes(dim, rot, pairing, m):
    t = Heads(dim + rot + m, m, dim, rot, pairing=pairing, axes=1 + m % 2 * 2)
    check(t, *forward(t))


@pytest.mark.parametrize("m", [2, 7, 15, 16, 17, 33, 300])
@pytest.mark.parametrize("q_heads, kv_heads, page", [(40, 8, 16), (1, 1, 256), (9, 17, 64)])
def test_tokens_and_heads(m, q_heads, kv_heads, page):
    t = Heads(m, m, 64, 64, q_heads=q_heads, kv_heads=kv_heads, page=page, axes=2)
    check(t, *forward(t))


@pytest.mark.parametrize("shift, gap", [(1, 0), (0, 3), (2, 6), (0, 8)])
@pytest.mark.parametrize("pairing", [afx.ROPE_HALVES, afx.ROPE_NEIGHBOURS])
def test_alignments(shift, gap, pairing):
    t = Heads(shift + gap, 21, 128, 128, pairing=pairing, shift=shift, gap=gap)
    keep = t.qkv
    whole = torch.zeros(21, keep.shape[1] + shift)
    whole[:, shift:] = keep
    device = whole.cuda()
    t.qkv = type("Rows", (), {"cuda": lambda self: device[:, shift:]})()
    check(t, *forward(t))


@pytest.mark.parametrize("w_q, w_k", [(False, False), (True, False), (False, True)])
def test_without_norms(w_q, w_k):
    t = Heads(3, 19, 96, 96, w_q=w_q, w_k=w_k)
    check(t, *forward(t))


@pytest.mark.parametrize("parts", ["q", "k", "v", "qk", "kv", "qv"])
@pytest.mark.parametrize("dense", [True, False])
def test_parts(parts, dense):
    t = Heads(4, 18, 64, 32)
    check(t, *forward(t, dense=dense, parts=parts), dense=dense, parts=parts)


def test_far_positions():
    """Angles of millions of turns, and back."""
    t = Heads(5, 64, 128, 128)
    t.pos[0, :8] = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 16777217, -16777217, 131071, 0, 1], dtype=torch.int32)
    check(t, *forward(t))


def test_axes_out_of_range_are_the_last():
    t = Heads(6, 20, 64, 64, axes=3)
    t.axis[::3] = 3
    t.axis[1::7] = 255
    check(t, *forward(t))


def test_slots_outside_the_cache_write_nothing():
    t = Heads(7, 40, 64, 64)
    t.slots[::3] = -1
    t.slots[1::9] = t.n_pages * t.page
    t.slots[2::9] = 2 ** 31 - 1
    t.slots[5::9] = -2 ** 31
    check(t, *forward(t))


def test_infinities_stay_in_their_heads():
    t = Heads(8, 20, 64, 32)
    for n in "qkv":
        t.x[n][3, 5] = math.inf
        t.x[n][9, 60] = math.nan
    out, pages = forward(t)
    for n in "qk":
        y = out[n].cpu()[:, :t.x[n].shape[1]].reshape(20, -1, 64)
        want = torch.isfinite(t.want(n)[0])
        assert torch.equal(torch.isfinite(y), want) and bool(want[:3].all()) and not bool(want[3, 0].all())


def test_far_slots():
    """Offsets above 2^32 elements."""
    t = Heads(9, 18, 256, 256, kv_heads=8, page=256)
    page_elems = 256 * 8 * 256
    n_pages = 2 ** 32 // page_elems + 3
    t.slots = (torch.randperm(3 * 256, generator=t.gen)[:18] + (n_pages - 3) * 256).int()
    p, x, pos, slots = t.params(), t.qkv.cuda(), t.pos.cuda(), t.slots.cuda()
    k = torch.empty(n_pages, 8, 32, 256, 8, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(n_pages, 8, 32, 256, 8, dtype=torch.bfloat16, device="cuda")
    kv = afx.kv_pages(k.data_ptr(), v.data_ptr(), n_pages, 256, 8, 256)
    cut = 4 * 256 * t.q_heads
    afx.afx_heads_async(p, 18, pos.data_ptr(), pos.stride(0), 0, 0, x.data_ptr() + cut, x.stride(0),
                        x.data_ptr() + cut + 4 * 256 * 8, x.stride(0), 0, 0, 0, 0, kv, slots.data_ptr(),
                        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    page, off = slots.long() // 256, slots.long() % 256
    near("k", k[page, :, :, off].cpu().reshape(18, 8, 256), *t.want("k"))
    assert torch.equal(v[page, :, off // 8, :, off % 8].cpu(), t.x["v"].reshape(18, 8, 256).bfloat16())


def backward(t, *, in_place=False, parts="qk", dw=True):
    p, m, d = t.params(), t.m, t.dim
    x = t.qkv.cuda()
    at = {"q": x.data_ptr(), "k": x.data_ptr() + 4 * t.q_heads * d}
    dy = {n: t.dy[n].contiguous().cuda() for n in "qk"}
    out = {n: dy[n] if in_place else torch.full((m, dy[n].shape[1] + 8), 7.0, dtype=torch.bfloat16, device="cuda")
           for n in "qk"}
    grads = {n: torch.full((d,), 7.0, device="cuda") for n in "qk"}
    pos = t.pos.cuda()
    ws = torch.empty(max(16, afx.afx_heads_workspace(p, m)), dtype=torch.uint8, device="cuda")
    do = lambda n, v: v if n in parts else 0  # noqa: E731
    w = lambda n: grads[n].data_ptr() if dw and t.w[n] is not None else 0  # noqa: E731
    afx.afx_heads_backward_async(
        p, m, pos.data_ptr(), pos.stride(0), do("q", at["q"]), x.stride(0), do("k", at["k"]), x.stride(0),
        do("q", dy["q"].data_ptr()), dy["q"].stride(0), do("k", dy["k"].data_ptr()), dy["k"].stride(0),
        do("q", out["q"].data_ptr()), out["q"].stride(0), do("k", out["k"].data_ptr()), out["k"].stride(0),
        do("q", w("q")), do("k", w("k")), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return out, grads


def check_grad(t, out, grads, parts="qk", dw=True, in_place=False):
    for n in "qk":
        if n not in parts:
            assert in_place or bool((out[n] == 7).all())
            assert bool((grads[n] == 7).all())
            continue
        dx, bound, want, wbound = t.want_grad(n)
        size = t.dy[n].shape[1]
        near("d" + n, out[n].cpu()[:, :size].reshape(dx.shape), dx, bound)
        if not in_place:
            assert bool((out[n][:, size:] == 7).all())
        if want is not None and dw:
            near("dw_" + n, grads[n].cpu(), want, wbound)
        else:
            assert bool((grads[n] == 7).all())


@pytest.mark.parametrize("dim, rot", SIZES)
@pytest.mark.parametrize("pairing", [afx.ROPE_HALVES, afx.ROPE_NEIGHBOURS])
@pytest.mark.parametrize("m", [1, 50])
def test_gradients(dim, rot, pairing, m):
    t = Heads(dim + rot + m, m, dim, rot, pairing=pairing, axes=1 + m % 3)
    check_grad(t, *backward(t))


@pytest.mark.parametrize("m", [15, 16, 17, 130, 2500])
@pytest.mark.parametrize("q_heads, kv_heads", [(40, 8), (1, 1), (9, 17)])
def test_gradients_of_many_tokens_and_heads(m, q_heads, kv_heads):
    t = Heads(m, m, 64, 64, q_heads=q_heads, kv_heads=kv_heads)
    check_grad(t, *backward(t))


@pytest.mark.parametrize("w_q, w_k", [(False, False), (True, False), (False, True)])
def test_gradients_without_norms(w_q, w_k):
    t = Heads(13, 31, 96, 48, w_q=w_q, w_k=w_k)
    check_grad(t, *backward(t))


@pytest.mark.parametrize("parts, dw, in_place", [("q", True, False), ("k", True, False), ("qk", False, False),
                                                 ("qk", True, True), ("k", True, True)])
def test_gradients_in_part_and_in_place(parts, dw, in_place):
    t = Heads(14, 45, 128, 128, gap=4)
    check_grad(t, *backward(t, parts=parts, dw=dw, in_place=in_place), parts=parts, dw=dw, in_place=in_place)


def test_gradients_of_no_tokens_are_zeros():
    t = Heads(15, 0, 64, 64)
    p, g = t.params(), torch.full((2, 64), 7.0, device="cuda")
    afx.afx_heads_backward_async(p, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, g[0].data_ptr(), g[1].data_ptr(), 0, 0,
                                 torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert bool((g == 0).all())


def test_gradients_against_differences():
    """The sum of dy times the forward formula, moved along a direction."""
    t = Heads(16, 6, 40, 24, pairing=afx.ROPE_NEIGHBOURS, axes=2)
    out, grads = backward(t)
    step = 1e-5
    for n in "qk":
        x0, w0 = t.x[n].double().clone(), t.w[n].double().clone()
        dx, dw = torch.randn(x0.shape, generator=t.gen).double(), torch.randn(40, generator=t.gen).double()

        def value(sx, sw):
            x = (x0 + sx * dx).reshape(6, -1, 40)
            y = t.turn(x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * (w0 + sw * dw))[0]
            return float((y.reshape(6, -1) * t.dy[n].double()).sum())

        _, bound, _, wbound = t.want_grad(n)
        got = float((out[n].cpu()[:, :x0.shape[1]].double() * dx).sum())
        diff = (value(step, 0) - value(-step, 0)) / (2 * step)
        assert abs(got - diff) <= float((bound.reshape(6, -1) * dx.abs()).sum()) + 1e-6 * abs(diff) + 1e-6
        got = float((grads[n].cpu().double() * dw).sum())
        diff = (value(0, step) - value(0, -step)) / (2 * step)
        assert abs(got - diff) <= float((wbound * dw.abs()).sum()) + 1e-6 * abs(diff) + 1e-6


def test_captured_replayed_and_on_two_streams():
    t = Heads(17, 70, 128, 128, q_heads=8, kv_heads=2)
    a = backward(t)
    check_grad(t, *a)
    b = backward(t)
    assert all(torch.equal(x[n], y[n]) for x, y in zip(a, b) for n in "qk"), "other bits on another run"
    p, d = t.params(), 128
    x, pos, slots = t.qkv.cuda(), t.pos.cuda(), t.slots.cuda()
    q = [torch.zeros(70, 8 * d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    dq = t.dy["q"].contiguous().cuda()
    dx = torch.zeros(70, 8 * d, dtype=torch.bfloat16, device="cuda")
    dw = torch.zeros(d, device="cuda")
    ws = torch.empty(afx.afx_heads_workspace(p, 70), dtype=torch.uint8, device="cuda")

    def calls(out, stream):
        afx.afx_heads_async(p, 70, pos.data_ptr(), pos.stride(0), x.data_ptr(), x.stride(0), 0, 0, 0, 0, out.data_ptr(),
                            8 * d, 0, 0, None, 0, stream)

    def grad(stream):
        afx.afx_heads_backward_async(p, 70, pos.data_ptr(), pos.stride(0), x.data_ptr(), x.stride(0), 0, 0,
                                     dq.data_ptr(), 8 * d, 0, 0, dx.data_ptr(), 8 * d, 0, 0, dw.data_ptr(), 0,
                                     ws.data_ptr(), ws.numel(), stream)

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s, out in zip(streams, q):
        calls(out, s.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(q[0], q[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = torch.cuda.current_stream().cuda_stream
        calls(q[0], s)
        grad(s)
    for i in range(3):
        t.pos = t.pos + 11
        pos.copy_(t.pos)
        q[0].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        near("q", q[0].cpu().reshape(70, 8, d), *t.want("q"))
        want, bound, ww, wb = t.want_grad("q")
        near("dq", dx.cpu().reshape(70, 8, d), want, bound)
        near("dw", dw.cpu(), ww, wb)
    del slots
