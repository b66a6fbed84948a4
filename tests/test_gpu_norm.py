"""GPU parity of the block norms and their gradients, against the formulas in
64 bits (gradients by autograd of the forward formula).

Tolerances. A mean over a row is a sum of at most 32 values per lane, 6 steps
across a wave and 16 across waves: its relative error is at most gamma_60 of
the sum of absolute terms, u = 2^-24; rsqrt, products and the final additions
add a few u. E = 72 u of the magnitudes below covers them. A BF16 output adds
half a step, 2^-8 of its value. Sums over m rows add gamma_(m + 64)."""
import sys

import numpy as np
import pytest

from lossless_bf16_weight_afx_amd import afx

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -24
E = 72 * U
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EPS, SCALE = 1e-5, 0.625
TYPES = {"bf16": (torch.bfloat16, afx.TYPE_BF16), "fp32": (torch.float32, afx.TYPE_FP32)}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


def make(rng, m, d, dtype, stride, std=1.0, mean=0.0):
    """[m, d] values in rows `stride` apart, NaN between and behind."""
    t = torch.full((m + 2, stride), float("nan"), dtype=dtype, device="cuda")
    t[:m, :d] = torch.from_numpy(rng.standard_normal((m, d)) * std + mean).to(dtype)
    return t


def blank(m, d, dtype):
    return torch.full((m + 2, d), -7.0, dtype=dtype, device="cuda")


def untouched(t, m, d):
    t = t.clone()
    t[:m, :d] = -7.0
    return bool((t == -7.0).all())


def ptr(t):
    return 0 if t is None else t.data_ptr()


def row(t):
    return 0 if t is None else t.shape[1]


def cpu(t, m, d):
    return None if t is None else t[:m, :d].cpu().double()


def check(name, got, want, tol):
    err = (got - want).abs()
    worst = float((err / tol.clamp_min(1e-300)).max()) if err.numel() else 0.0
    say(f"[gpu]   {name}: worst error / bound = {worst:.3g}")
    assert bool((err <= tol).all()), f"{name}: worst error / bound = {worst}"


def mean(t):
    return t.mean(-1, keepdim=True)


class Case:
    """Inputs of one shape and set of options, and the parameters struct."""

    def __init__(self, m, d, r_type, post, gate, pre=True, block=True, pad=0, seed=0):
        rng = np.random.default_rng([m, d, seed])
        self.m, self.d = m, d
        self.dtype, code = TYPES[r_type]
        s = d + pad
        self.b = make(rng, m, d, torch.float32, s, 1.5) if block else None
        self.r = make(rng, m, d, self.dtype, s, 2.0)
        vec = lambda: make(rng, 1, d, torch.bfloat16, d, 0.3, 1.0)  # noqa: E731
        self.w_post = vec() if post else None
        self.w_pre = vec() if pre else None
        self.gate = None if gate == "none" else vec() if gate == "channel" else \
            make(rng, m, d, torch.bfloat16, s, 0.5)
        self.per_row = gate == "row"
        self.dxn = make(rng, m, d, torch.bfloat16, s)
        self.dr_out = make(rng, m, d, self.dtype, s)
        self.p = afx.block_norm(d, EPS, SCALE, code, ptr(self.w_post), ptr(self.gate), s if self.per_row else 0,
                                ptr(self.w_pre))

    def wide(self, name):
        """An input in 64 bits ([m, d], or [1, d] for a shared vector)."""
        t = getattr(self, name)
        return cpu(t, self.m if name not in ("w_post", "w_pre") and (name != "gate" or self.per_row) else 1, self.d)


def forward(c, pad=0, in_place=False):
    ro = c.r if in_place else blank(c.m, c.d + pad, c.dtype)
    xn = blank(c.m, c.d + pad, torch.bfloat16) if c.w_pre is not None else None
    afx.afx_block_norm_async(c.p, c.m, ptr(c.b), row(c.b), ptr(c.r), row(c.r), ptr(ro), row(ro), ptr(xn), row(xn),
                             torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert in_place or untouched(ro, c.m, c.d)
    assert xn is None or untouched(xn, c.m, c.d)
    return cpu(ro, c.m, c.d), cpu(xn, c.m, c.d)


def forward64(c):
    """r', xn and the error magnitudes of each."""
    r = c.wide("r")
    add = torch.zeros_like(r)
    if c.b is not None:
        add = c.wide("b")
        if c.w_post is not None:
            add = add / torch.sqrt(mean(add ** 2) + EPS) * c.wide("w_post")
        if c.gate is not None:
            add = add * c.wide("gate")
        add = add * SCALE
    out = r + add
    er = E * (add.abs() + out.abs())
    if c.w_pre is None:
        return out, None, er, None
    k = 1 / torch.sqrt(mean(out ** 2) + EPS)
    w = c.wide("w_pre")
    ek = k ** 3 * mean(out.abs() * er) + E * k  # of k, from r' and from its own sums
    return out, out * k * w, er, (er * k + out.abs() * ek) * w.abs() + E * (out * k * w).abs()


# widths around every team: 16 lanes, a wave, a workgroup, 8 and 32 values a lane
WIDTHS = [1, 7, 8, 64, 127, 128, 129, 136, 511, 512, 513, 520, 1000, 1023, 4096, 5120, 8191, 8192, 8193, 8200, 16384,
          20003, 32768]


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("r_type,post,gate,pad", [("bf16", True, "none", 0), ("fp32", True, "channel", 8),
                                                  ("bf16", False, "row", 3), ("fp32", False, "none", 0)])
def test_forward(d, r_type, post, gate, pad):
    for m in (1, 2, 33):
        say(f"[gpu] case norm {m}x{d} {r_type} post={post} gate={gate} pad={pad}")
        c = Case(m, d, r_type, post, gate, pad=pad)
        ro, xn = forward(c, pad)
        want_r, want_x, er, ex = forward64(c)
        check("r'", ro, want_r, er + HALF[c.dtype] * (want_r.abs() + er))
        check("xn", xn, want_x, ex + HALF[torch.bfloat16] * (want_x.abs() + ex))
        ro2, xn2 = forward(c, in_place=True)
        assert torch.equal(ro2, ro) and torch.equal(xn2, xn)


@pytest.mark.parametrize("d", [96, 5120, 333])
def test_forward_parts(d):
    """Only the norm before a block; only the residual add; with no r' kept."""
    c = Case(9, d, "bf16", False, "none", block=False)
    ro, xn = forward(c)
    assert torch.equal(ro, cpu(c.r, 9, d))
    _, want, _, ex = forward64(c)
    check("xn", xn, want, ex + HALF[torch.bfloat16] * (want.abs() + ex))
    alone = blank(9, d, torch.bfloat16)
    afx.afx_block_norm_async(c.p, 9, 0, 0, ptr(c.r), d, 0, 0, ptr(alone), d, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(cpu(alone, 9, d), xn)
    c = Case(9, d, "fp32", True, "channel", pre=False)
    ro, xn = forward(c)
    want, _, er, _ = forward64(c)
    assert xn is None
    check("r'", ro, want, er + HALF[c.dtype] * (want.abs() + er))


@pytest.mark.parametrize("d", [64, 300, 5120])
def test_rows_of_zeros_infinities_and_nan(d):
    """A row of zeros gives zeros (eps keeps its norm finite); infinities and
    NaN stay in their rows."""
    c = Case(40, d, "fp32", True, "none")
    c.b[3, :d] = 0
    c.r[3, :d] = 0
    c.b[5, 1] = float("inf")
    c.r[7, d - 1] = float("nan")
    ro, xn = forward(c)
    assert not ro[3].any() and not xn[3].any()
    assert bool(torch.isnan(xn[5]).any()) and bool(torch.isnan(xn[7]).all())
    keep = [t for t in range(40) if t not in (5, 7)]
    want_r, want_x, er, ex = forward64(c)
    check("r'", ro[keep], want_r[keep], (er + HALF[c.dtype] * (want_r.abs() + er))[keep])
    check("xn", xn[keep], want_x[keep], (ex + HALF[torch.bfloat16] * (want_x.abs() + ex))[keep])


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
def backward(c, in_place=False, sums=True, use_dxn=True, use_dro=True, pad=0):
    m, d = c.m, c.d
    dro = c.dr_out if use_dro else None
    dxn = c.dxn if use_dxn and c.w_pre is not None else None
    dr = dro if in_place else blank(m, d + pad, c.dtype)
    db = blank(m, d + pad, torch.bfloat16) if c.b is not None else None
    new = lambda ok: torch.full((d + 2,), -7.0, device="cuda") if ok else None  # noqa: E731
    dw_pre, dw_post = new(sums and c.w_pre is not None), new(sums and c.w_post is not None and c.b is not None)
    dgate = None
    if c.gate is not None and c.b is not None:
        dgate = torch.full((m * d + 2,), -7.0, device="cuda") if c.per_row else new(sums)
    n = afx.afx_block_norm_workspace(c.p, m)
    ws = torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    afx.afx_block_norm_backward_async(c.p, m, ptr(c.b), row(c.b), ptr(c.r), row(c.r), ptr(dxn), row(dxn), ptr(dro),
                                      row(dro), ptr(dr), row(dr), ptr(db), row(db), ptr(dw_pre), ptr(dw_post),
                                      ptr(dgate), ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert in_place or untouched(dr, m, d)
    assert db is None or untouched(db, m, d)
    for t in (dw_pre, dw_post, dgate):
        assert t is None or bool((t[-2:] == -7.0).all())
    flat = lambda t: None if t is None else t[:-2].cpu().double()  # noqa: E731
    dg = flat(dgate)
    return dict(dr=cpu(dr, m, d), db=cpu(db, m, d), dw_pre=flat(dw_pre), dw_post=flat(dw_post),
                dgate=dg.view(m, d) if dg is not None and c.per_row else dg)


def backward64(c, use_dxn=True, use_dro=True):
    """The gradients by autograd in 64 bits, and the magnitudes that their
    FP32 errors scale with."""
    m, d = c.m, c.d
    r = c.wide("r").requires_grad_()
    dro = c.wide("dr_out") if use_dro else torch.zeros(m, d, dtype=torch.float64)
    dr, mag_r = dro.clone(), dro.abs()
    want, mag = {}, {}
    if c.w_pre is not None:
        dxn = c.wide("dxn") if use_dxn else torch.zeros(m, d, dtype=torch.float64)
        w = c.wide("w_pre").requires_grad_()
        k = 1 / torch.sqrt(mean(r ** 2) + EPS)
        g, want["dw_pre"] = torch.autograd.grad((dxn * (r * k * w)).sum(), (r, w))
        dr = dr + g
        k, v, dn = k.detach(), r.detach().abs(), (dxn * w.detach()).abs()
        mag_r = mag_r + k * dn + k ** 3 * v * mean(dn * v)
        mag["dw_pre"] = dxn.abs() * v * k
    want["dr"], mag["dr"] = dr, mag_r
    if c.b is not None:
        b = c.wide("b").requires_grad_()
        n, leaves = b, {"db": b}
        k = torch.ones(m, 1, dtype=torch.float64)
        if c.w_post is not None:
            leaves["dw_post"] = w = c.wide("w_post").requires_grad_()
            k = (1 / torch.sqrt(mean(b ** 2) + EPS))
            n = b * k * w
            k = k.detach()
        bh = n
        if c.gate is not None:
            leaves["dgate"] = gate = c.wide("gate").requires_grad_()
            n = n * gate
        got = torch.autograd.grad((SCALE * n * dr).sum(), list(leaves.values()))
        want.update(zip(leaves, got))
        a = SCALE * mag_r
        if c.gate is not None:
            mag["dgate"] = a * bh.detach().abs()
            a = a * gate.detach().abs()
        if c.w_post is not None:
            v = b.detach().abs()
            mag["dw_post"] = a * v * k
            a = a * w.detach().abs()
            a = k * a + k ** 3 * v * mean(a * v)
        mag["db"] = a
    return want, mag


def check_backward(c, got, want, mag):
    m = c.m
    for name, v in got.items():
        if v is None:
            continue
        w = want[name]
        if name in ("dr", "db") or (name == "dgate" and c.per_row):
            half = HALF[c.dtype if name == "dr" else torch.bfloat16 if name == "db" else torch.float32]
            e = 3 * E * mag[name]  # dr's error, then its own sums'
            check(name, v, w, e + half * (w.abs() + e))
        else:
            e = (3 * E + (m + 64) * U) * mag[name].sum(0, keepdim=True)
            check(name, v.view(1, -1), w, e)


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("r_type,post,gate,pad", [("bf16", True, "none", 0), ("fp32", True, "channel", 8),
                                                  ("bf16", False, "row", 3), ("fp32", True, "row", 0),
                                                  ("fp32", False, "channel", 1)])
def test_backward(d, r_type, post, gate, pad):
    for m in (1, 3, 70):
        say(f"[gpu] case norm backward {m}x{d} {r_type} post={post} gate={gate} pad={pad}")
        c = Case(m, d, r_type, post, gate, pad=pad, seed=1)
        want, mag = backward64(c)
        got = backward(c, pad=pad)
        check_backward(c, got, want, mag)
        no_sums = backward(c, sums=False)
        assert torch.equal(no_sums["dr"], got["dr"]) and torch.equal(no_sums["db"], got["db"])
        again = backward(c, in_place=True)  # the same bits, dr over dr_out
        for k, v in got.items():
            assert v is None or torch.equal(again[k], v), k


@pytest.mark.parametrize("m,d", [(513, 136), (5000, 128), (1025, 5120), (2100, 72)])
def test_backward_many_rows(m, d):
    """More rows than workgroups: the sums over rows run through both stages."""
    say(f"[gpu] case norm backward {m}x{d}")
    c = Case(m, d, "fp32", True, "channel", seed=2)
    want, mag = backward64(c)
    check_backward(c, backward(c), want, mag)


@pytest.mark.parametrize("d", [96, 5120])
@pytest.mark.parametrize("parts", ["no dxn", "no dr_out", "no block", "no w_pre"])
def test_backward_parts(d, parts):
    c = Case(20, d, "bf16", parts != "no block", "none", pre=parts != "no w_pre", block=parts != "no block", seed=3)
    kw = dict(use_dxn=parts != "no dxn", use_dro=parts != "no dr_out")
    want, mag = backward64(c, **kw)
    check_backward(c, backward(c, **kw), want, mag)


def test_no_rows_give_zero_sums():
    d = 100
    c = Case(1, d, "bf16", True, "channel")
    out = [torch.full((d + 1,), -7.0, device="cuda") for _ in range(3)]
    afx.afx_block_norm_backward_async(c.p, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, *[ptr(o) for o in out], 0, 0,
                                      torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for o in out:
        assert not o[:d].any() and float(o[d]) == -7.0


def test_graph_replays_and_two_streams():
    m, d = 600, 5120
    cases = [Case(m, d, "fp32", True, "channel", seed=s) for s in (5, 6)]
    eager = []
    for c in cases:
        eager.append((forward(c), backward(c)))
    # each stream has its own buffers and workspace
    streams, got = [torch.cuda.Stream() for _ in cases], []
    torch.cuda.synchronize()
    bufs = []
    for c, s in zip(cases, streams):
        ro, xn, dr, db = (blank(m, d, t) for t in (c.dtype, torch.bfloat16, c.dtype, torch.bfloat16))
        dw = [torch.zeros(d, device="cuda") for _ in range(3)]
        ws = torch.empty(afx.afx_block_norm_workspace(c.p, m), dtype=torch.uint8, device="cuda")
        bufs.append((ro, xn, dr, db, dw, ws))
    torch.cuda.synchronize()

    def step(c, buf, handle):
        ro, xn, dr, db, dw, ws = buf
        afx.afx_block_norm_async(c.p, m, ptr(c.b), d, ptr(c.r), d, ptr(ro), d, ptr(xn), d, handle)
        afx.afx_block_norm_backward_async(c.p, m, ptr(c.b), d, ptr(c.r), d, ptr(c.dxn), d, ptr(c.dr_out), d, ptr(dr),
                                          d, ptr(db), d, *[ptr(t) for t in dw], ptr(ws), ws.numel(), handle)

    def same():
        torch.cuda.synchronize()
        for (fw, bw), (ro, xn, dr, db, dw, _) in zip(eager, bufs):
            for a, b in zip((fw[0], fw[1], bw["dr"], bw["db"]), (ro, xn, dr, db)):
                assert torch.equal(a, cpu(b, m, d))
            for a, b in zip((bw["dw_pre"], bw["dw_post"], bw["dgate"]), dw):
                assert torch.equal(a, b.cpu().double())

    for c, s, b in zip(cases, streams, bufs):
        step(c, b, s.cuda_stream)
    same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c, b in zip(cases, bufs):
            step(c, b, torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        for b in bufs:
            for t in (*b[:4], *b[4]):
                t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        same()
