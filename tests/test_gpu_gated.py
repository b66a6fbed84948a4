"""GPU parity of the gated feed-forward block over coded weights, its
gradients and the transposed product, against the formulas in 64 bits.

Tolerances. A sum of k products of BF16 values (exact in FP32) errs by at
most gamma_k sum |terms|, gamma_k = k u / (1 - k u), u = 2^-24, whatever its
order. An output rounded to BF16 adds half a step, 2^-8 of its value. The
activations and their derivatives are FP32: with |g| <= 2^6 here, e^-g is
off by at most (|g| + 2) 2^-23 relatively (its argument times log2(e) is
rounded, then v_exp_f32's ulp), and the divisions, products and erfc that
follow by a few u more: 2^-18 (1 + |g|) of the largest term covers them.
|act'| is at most 1.13 for all three."""
import math
import sys

import numpy as np
import pytest

import oracle
from lossless_bf16_weight_afx_amd import afx, synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ACTS = {"silu": afx.ACT_SILU, "gelu_tanh": afx.ACT_GELU_TANH, "gelu": afx.ACT_GELU}
U = 2.0 ** -24
HALF_BF16 = 2.0 ** -8


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


def gamma(k):
    return k * U / (1 - k * U)


def act64(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "gelu_tanh":
        return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return 0.5 * g * torch.special.erfc(-g / math.sqrt(2))


def dact64(g, act):
    """Central differences of act64 (step 2^-14: off by about 2^-30 + 2^-38)."""
    s = 2.0 ** -14
    return (act64(g + s, act) - act64(g - s, act)) / (2 * s)


class Coded:
    """A matrix, coded on the device, and its values."""

    def __init__(self, w):  # float32 [rows, cols]
        bits = synth.f32_to_bf16_bits(np.ascontiguousarray(w, np.float32).ravel())
        self.rows, self.cols = w.shape
        blob = oracle.encode(bits, w.shape)
        self.info, self.dev = afx.afx_query(blob), afx.to_device(blob)
        self.w = torch.from_numpy(synth.bf16_bits_to_f32(bits).reshape(w.shape).astype(np.float64))


def rng_of(*k):
    return np.random.default_rng([int(v) for v in k])


def normal(rng, shape, std=1.0):
    return (rng.standard_normal(shape) * std).astype(np.float32)


def strided(values, stride, dtype, extra_rows=2, fill=float("nan"), shift=0):
    """values [m, n] in rows `stride` apart, `fill` between and behind them,
    the first row `shift` elements into the allocation."""
    m, n = values.shape
    flat = torch.full((shift + (m + extra_rows) * stride,), fill, dtype=dtype, device="cuda")
    t = flat[shift:].view(m + extra_rows, stride)
    t[:m, :n] = torch.as_tensor(values).to(dtype)
    return t


def untouched(t, m, n, fill=-7.0):
    """Nothing was written beside the n values of the first m rows."""
    t = t.clone()
    t[:m, :n] = fill
    return bool((t == fill).all())


def workspace(n):
    return torch.full((max(n, 16),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns


def stream():
    return torch.cuda.current_stream().cuda_stream


def run_forward(gate, up, act, x, save, h_stride=None, gu_stride=None):
    """x: device BF16 [>= m rows, stride] made by strided(); returns h, g, u."""
    t, m = x
    rows, cols = gate.rows, gate.cols
    hs, gs = h_stride or rows, gu_stride or rows
    out = [torch.full((m + 2, s), -7.0, dtype=torch.bfloat16, device="cuda") for s in (hs, gs, gs)]
    n = afx.afx_restore_gated_workspace(rows, cols, m)
    ws = workspace(n)
    w = afx.gated_weights(gate.info, gate.dev.data_ptr(), up.info, up.dev.data_ptr(), rows, cols, ACTS[act])
    g, u = (out[1].data_ptr(), out[2].data_ptr()) if save else (0, 0)
    afx.afx_restore_gated_async(w, m, t.data_ptr(), t.shape[1], out[0].data_ptr(), hs, g, u, gs, ws.data_ptr(), n,
                                stream())
    torch.cuda.synchronize()
    assert untouched(out[0], m, rows)
    for o in out[1:]:
        assert untouched(o, m if save else 0, rows)
    return [o[:m, :rows].cpu().double() for o in out]


def check(name, got, want, tol):
    err = (got - want).abs()
    worst = float((err / tol.clamp_min(1e-300)).max()) if err.numel() else 0.0
    say(f"[gpu]   {name}: worst error / bound = {worst:.3g}")
    assert bool((err <= tol).all()), f"{name}: worst error / bound = {worst}"


# sizes where something changes: one row, one chunk of columns, rows and
# columns that end inside a tile, tokens around every tile height, rows past
# one tile of 128, columns past one of 64 and odd numbers of column tiles
SIZES = [(1, 8, 1), (5, 8, 2), (3, 72, 3), (130, 136, 4), (128, 64, 5), (257, 200, 7), (64, 264, 31), (131, 5120, 1),
         (96, 4104, 2), (33, 4096, 4), (640, 1024, 33), (129, 328, 64), (100, 1032, 65), (383, 192, 128),
         (127, 256, 129), (300, 72, 255), (128, 520, 256), (385, 320, 257), (70, 128, 513),
         # the fused matrix-core kernel (rows of whole groups): one group a row, rows that end inside a slab, a tile
         # over many ranges, token counts around every operand count, more slabs than ranges
         (17, 32, 5), (33, 5120, 6), (100, 2080, 16), (31, 8192, 17), (1000, 288, 32), (2100, 2336, 48),
         (50, 480, 63), (4000, 2624, 80), (129, 1056, 100), (16, 96, 127), (48, 16384, 128)]


@pytest.mark.parametrize("rows,cols,m", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_forward(rows, cols, m, act):
    say(f"[gpu] case gated {act} {rows}x{cols} m={m}")
    rng = rng_of(rows, cols, m)
    gate, up = Coded(normal(rng, (rows, cols), cols ** -0.5)), Coded(normal(rng, (rows, cols), cols ** -0.5))
    x = strided(normal(rng, (m, cols), 1.5), cols + 8, torch.bfloat16)
    x64 = x[:m, :cols].cpu().double()
    h, g, u = run_forward(gate, up, act, (x, m), True, rows + 3, rows + 5)
    gr, ur = x64 @ gate.w.T, x64 @ up.w.T
    eg, eu = gamma(cols) * (x64.abs() @ gate.w.abs().T), gamma(cols) * (x64.abs() @ up.w.abs().T)
    check("g", g, gr, eg + HALF_BF16 * (gr.abs() + eg))
    check("u", u, ur, eu + HALF_BF16 * (ur.abs() + eu))
    a = act64(gr, act)
    ea = 1.13 * eg + 2.0 ** -18 * (1 + gr.abs()) * a.abs()
    eh = ea * ur.abs() + (a.abs() + ea) * eu
    check("h", h, a * ur, eh + HALF_BF16 * ((a * ur).abs() + eh) + 1e-37)
    only_h = run_forward(gate, up, act, (x, m), False)
    assert torch.equal(only_h[0], h)  # the same bits without g and u, and in another run


@pytest.mark.parametrize("rows,cols,m", [(70, 320, 1), (70, 320, 3), (70, 320, 6), (200, 5120, 40), (90, 4128, 90),
                                         (200, 520, 300)])
def test_forward_integers_exact(rows, cols, m):
    """Small integers: g and u are exact in FP32 whatever the order of the
    sums, so the kept g and u are exactly their BF16 roundings."""
    say(f"[gpu] case gated integers {rows}x{cols} m={m}")
    rng = rng_of(7, rows, cols, m)
    gate = Coded(rng.integers(-2, 3, (rows, cols)).astype(np.float32))
    up = Coded(rng.integers(-3, 4, (rows, cols)).astype(np.float32))
    x = strided(rng.integers(-2, 3, (m, cols)).astype(np.float32), cols, torch.bfloat16)
    x64 = x[:m].cpu().double()
    _, g, u = run_forward(gate, up, "silu", (x, m), True)
    for got, w in ((g, gate.w), (u, up.w)):
        assert torch.equal(got, (x64 @ w.T).float().bfloat16().double())


@pytest.mark.parametrize("m,cols", [(1, 200), (4, 200), (20, 200), (20, 224), (100, 288), (200, 200)])
def test_special_values_stay_where_they_are(m, cols):
    """An infinity in one token and NaN in another reach those tokens only,
    an infinite weight only its own output; large pre-activations saturate."""
    rows = 40
    rng = rng_of(3, m)
    wg, wu = normal(rng, (rows, cols)), normal(rng, (rows, cols))
    wg[5, 3] = np.inf
    gate, up = Coded(wg), Coded(wu)
    xv = normal(rng, (m, cols), 30.0)
    xv[:, 3] = np.abs(xv[:, 3]) + 1  # times inf: +inf, never NaN
    if m > 2:
        xv[1, 7], xv[2, 9] = np.inf, np.nan
    x = strided(xv, cols, torch.bfloat16)
    h, g, u = run_forward(gate, up, "silu", (x, m), True)
    tokens = [t for t in range(m) if t not in (1, 2)] if m > 2 else list(range(m))
    keep = [f for f in range(rows) if f != 5]
    assert bool(torch.isfinite(h[tokens][:, keep]).all())
    assert bool(torch.isinf(g[tokens, 5]).all()) and bool(torch.isinf(h[tokens, 5]).all())
    x64 = x[:m].cpu().double()
    gr, ur = x64[tokens] @ gate.w[keep].T, x64[tokens] @ up.w[keep].T
    want = act64(gr, "silu") * ur
    eg = gamma(cols) * (x64[tokens].abs() @ gate.w[keep].abs().T)
    eu = gamma(cols) * (x64[tokens].abs() @ up.w[keep].abs().T)
    # far below zero silu(g) = g e^g: relative to it, an error e of g is e itself, e^-g is off by
    # 2^-23 |g|, and beyond |g| = 88 it is 0 or subnormal
    a = act64(gr, "silu").abs()
    ea = 1.13 * eg * torch.maximum(a, torch.ones_like(a) * 1e-30).clamp_max(1) + 1.13 * eg * (gr > -20) + \
        2.0 ** -18 * (1 + gr.abs()) * a
    eh = ea * ur.abs() + (a + ea) * eu
    check("h", h[tokens][:, keep], want, eh + HALF_BF16 * (want.abs() + eh) + 1e-36 * (1 + ur.abs()))
    if m > 2:
        assert bool(torch.isnan(g[2]).all())


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------
def run_backward(gate, up, act, dh, gu, m, keep_grads=True, in_place=False, dx_stride=None):
    rows, cols = gate.rows, gate.cols
    g, u = gu
    gs = g.shape[1]
    dxs = dx_stride or cols
    dx = torch.full((m + 2, dxs), -7.0, dtype=torch.bfloat16, device="cuda")
    if in_place:
        dg, du = g, u
    else:
        dg, du = (torch.full((m + 2, gs), -7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = afx.afx_restore_gated_workspace(rows, cols, m, backward=True)
    ws = workspace(n)
    w = afx.gated_weights(gate.info, gate.dev.data_ptr(), up.info, up.dev.data_ptr(), rows, cols, ACTS[act])
    afx.afx_restore_gated_backward_async(w, m, dh.data_ptr(), dh.shape[1], g.data_ptr(), u.data_ptr(), gs,
                                         dx.data_ptr(), dxs, dg.data_ptr() if keep_grads else 0,
                                         du.data_ptr() if keep_grads else 0, ws.data_ptr(), n, stream())
    torch.cuda.synchronize()
    assert untouched(dx, m, cols)
    if not in_place:
        assert untouched(dg, m if keep_grads else 0, rows) and untouched(du, m if keep_grads else 0, rows)
    return [v[:m, :k].cpu().double() for v, k in ((dx, cols), (dg, rows), (du, rows))]


@pytest.mark.parametrize("rows,cols,m", [(1, 8, 1), (5, 8, 2), (63, 72, 3), (64, 136, 17), (65, 264, 64),
                                         (200, 256, 65), (333, 520, 129), (128, 264, 257), (1500, 64, 40),
                                         (4100, 40, 300)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "gelu"])
def test_backward(rows, cols, m, act):
    say(f"[gpu] case gated backward {act} {rows}x{cols} m={m}")
    rng = rng_of(11, rows, cols, m)
    gate, up = Coded(normal(rng, (rows, cols), 0.02)), Coded(normal(rng, (rows, cols), 0.02))
    dh = strided(normal(rng, (m, rows)), rows + 3, torch.float32)
    g = strided(normal(rng, (m, rows), 2.0), rows + 7, torch.bfloat16)
    u = strided(normal(rng, (m, rows), 2.0), rows + 7, torch.bfloat16)
    dh64, g64, u64 = (v[:m, :rows].cpu().double() for v in (dh, g, u))
    dx, dg, du = run_backward(gate, up, act, dh, (g, u), m, dx_stride=cols + 5)
    for name, got, want, big in (("dg", dg, dh64 * u64 * dact64(g64, act), (dh64 * u64).abs()),
                                 ("du", du, dh64 * act64(g64, act), (dh64 * g64).abs())):
        check(name, got, want, HALF_BF16 * want.abs() + 2.0 ** -18 * (1 + g64.abs()) * big)
    # dx from the dg and du it gave (BF16, the operands of its products)
    want = dg @ gate.w + du @ up.w
    e = gamma(2 * rows) * (dg.abs() @ gate.w.abs() + du.abs() @ up.w.abs())
    check("dx", dx, want, e + HALF_BF16 * (want.abs() + e))
    again, _, _ = run_backward(gate, up, act, dh, (g, u), m, keep_grads=False)
    assert torch.equal(again, dx)
    again, dg2, du2 = run_backward(gate, up, act, dh, (g, u), m, in_place=True)
    assert torch.equal(again, dx) and torch.equal(dg2, dg) and torch.equal(du2, du)


def test_backward_aligned_buffers_give_the_same_bits():
    """dg and du at 16-byte aligned rows, at odd ones and not kept at all."""
    rows, cols, m = 200, 128, 50
    rng = rng_of(19)
    gate, up = Coded(normal(rng, (rows, cols), 0.02)), Coded(normal(rng, (rows, cols), 0.02))
    dhv, gv, uv = normal(rng, (m, rows)), normal(rng, (m, rows)), normal(rng, (m, rows))
    got = [run_backward(gate, up, "silu", strided(dhv, s, torch.float32, shift=k),
                        (strided(gv, s, torch.bfloat16, shift=k), strided(uv, s, torch.bfloat16, shift=k)), m, keep)[0]
           for s, k, keep in ((rows, 0, True), (rows, 0, False), (rows + 8, 0, True), (rows + 1, 0, True),
                              (rows, 1, True))]
    for v in got[1:]:
        assert torch.equal(v, got[0])


def test_chain_of_differences():
    """dx against central differences of the whole block's scalar loss
    sum(dh h(x)) in 64 bits, x moved along random directions."""
    rows, cols, m = 48, 64, 9
    rng = rng_of(23)
    gate, up = Coded(normal(rng, (rows, cols), 0.1)), Coded(normal(rng, (rows, cols), 0.1))
    x = strided(normal(rng, (m, cols)), cols, torch.bfloat16)
    dh = strided(normal(rng, (m, rows)), rows, torch.float32)
    for act in ACTS:
        _, g, u = run_forward(gate, up, act, (x, m), True)
        dx, dg, du = run_backward(gate, up, act, dh, (strided(g, rows, torch.bfloat16), strided(u, rows, torch.bfloat16)), m)
        x64, dh64 = x[:m].cpu().double(), dh[:m].cpu().double()
        loss = lambda v: float((dh64 * act64(v @ gate.w.T, act) * (v @ up.w.T)).sum())  # noqa: E731
        # g and u were rounded to BF16 (half a step), |act''| <= 1 for these, dg and du and dx again
        gr, ur = x64 @ gate.w.T, x64 @ up.w.T
        step = HALF_BF16 * 1.01
        edg = dh64.abs() * (step * ur.abs() * 1.13 + ur.abs() * step * gr.abs()) * 1.02 + step * dg.abs()
        edu = dh64.abs() * 1.13 * step * gr.abs() * 1.02 + step * du.abs()
        edx = edg @ gate.w.abs() + edu @ up.w.abs() + step * dx.abs() + 1e-5
        for _ in range(4):
            v = torch.from_numpy(rng.standard_normal((m, cols)))
            s = 2.0 ** -12
            diff = (loss(x64 + s * v) - loss(x64 - s * v)) / (2 * s)
            assert abs(diff - float((dx * v).sum())) <= float((edx * v.abs()).sum()) + 1e-4


# ---------------------------------------------------------------------------
# transposed product
# ---------------------------------------------------------------------------
def run_t(mat, dv, m, add=None):
    """y = d W, or add + d W."""
    d = torch.full((m + 1, mat.rows), float("nan"), dtype=torch.bfloat16, device="cuda")  # NaN behind the last token
    d[:m] = torch.as_tensor(dv).bfloat16()
    y = torch.full((m + 1, mat.cols), -7.0, device="cuda")
    if add is not None:
        y[:m] = add
    n = afx.afx_restore_gemm_t_workspace(mat.rows, mat.cols, m)
    ws = workspace(n)
    afx.afx_restore_gemm_t_async(mat.info, mat.dev.data_ptr(), mat.rows, mat.cols, d.data_ptr(), m, y.data_ptr(),
                                 add is not None, ws.data_ptr(), n, stream())
    torch.cuda.synchronize()
    assert untouched(y, m, mat.cols)
    return y[:m].cpu().double(), d[:m].cpu().double()


T_SIZES = [(8, 8, 1), (8, 64, 2), (64, 8, 3), (72, 136, 5), (64, 256, 16), (128, 264, 63), (200, 512, 64),
           (1032, 256, 65), (5120, 264, 33), (136, 1000, 129), (64, 248, 256), (520, 328, 257), (4104, 72, 300)]


@pytest.mark.parametrize("rows,cols,m", T_SIZES)
def test_transposed_integers_exact(rows, cols, m):
    say(f"[gpu] case transposed integers {rows}x{cols} m={m}")
    rng = rng_of(31, rows, cols, m)
    mat = Coded(rng.integers(-3, 4, (rows, cols)).astype(np.float32))
    y, d = run_t(mat, rng.integers(-2, 3, (m, rows)).astype(np.float32), m)
    assert torch.equal(y, d @ mat.w)
    y0 = torch.from_numpy(rng.integers(-100, 100, (m, cols)).astype(np.float32)).cuda()
    y, d = run_t(mat, rng.integers(-2, 3, (m, rows)).astype(np.float32), m, y0)
    assert torch.equal(y, d @ mat.w + y0.cpu().double())


@pytest.mark.parametrize("rows,cols,m", [(5120, 520, 7), (2048, 256, 200), (5120, 1024, 300)])
def test_transposed_random_within_bound(rows, cols, m):
    say(f"[gpu] case transposed random {rows}x{cols} m={m}")
    rng = rng_of(37, rows, cols, m)
    mat = Coded(normal(rng, (rows, cols), 0.02))
    dv, y0 = normal(rng, (m, rows)), torch.from_numpy(normal(rng, (m, cols))).cuda()
    y, d = run_t(mat, dv, m, y0)
    c = y0.cpu().double()
    check("y", y, d @ mat.w + c, gamma(rows + 1) * (d.abs() @ mat.w.abs() + c.abs()))
    again, _ = run_t(mat, dv, m, y0)
    assert torch.equal(again, y)


def test_transposed_special_values_stay_in_their_columns():
    rows, cols, m = 72, 264, 20
    rng = rng_of(41)
    w = normal(rng, (rows, cols))
    w[70, 100] = np.inf  # in the last, partial k-tile and the middle of the columns
    mat = Coded(w)
    y, d = run_t(mat, np.abs(normal(rng, (m, rows))) + 0.1, m)
    cols_ok = [c for c in range(cols) if c != 100]
    assert bool(torch.isinf(y[:, 100]).all())
    check("y", y[:, cols_ok], d @ mat.w[:, cols_ok], gamma(rows) * (d.abs() @ mat.w[:, cols_ok].abs()))


# ---------------------------------------------------------------------------
# streams, graphs, several calls at once
# ---------------------------------------------------------------------------
def test_two_streams_with_a_workspace_each():
    rows, cols, m = 256, 512, 150
    rng = rng_of(43)
    gate, up = Coded(normal(rng, (rows, cols), 0.05)), Coded(normal(rng, (rows, cols), 0.05))
    xs = [torch.from_numpy(normal(rng, (m, cols))).bfloat16().cuda() for _ in range(2)]
    n = afx.afx_restore_gated_workspace(rows, cols, m)
    w = afx.gated_weights(gate.info, gate.dev.data_ptr(), up.info, up.dev.data_ptr(), rows, cols)
    want = [run_forward(gate, up, "silu", (x, m), False)[0] for x in xs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    hs = [torch.zeros(m, rows, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    spaces = [workspace(n) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, x, h, ws in zip(streams, xs, hs, spaces):
            afx.afx_restore_gated_async(w, m, x.data_ptr(), cols, h.data_ptr(), rows, 0, 0, 0, ws.data_ptr(), n,
                                        s.cuda_stream)
    torch.cuda.synchronize()
    for h, k in zip(hs, want):
        assert torch.equal(h.cpu().double(), k)


@pytest.mark.parametrize("m", [1, 24, 300])
def test_graph_replays(m):
    """Forward, backward and transposed product captured in one graph; every
    replay on new inputs gives the eager call's bits."""
    rows, cols = 264, 320
    rng = rng_of(47, m)
    gate, up = Coded(normal(rng, (rows, cols), 0.05)), Coded(normal(rng, (rows, cols), 0.05))
    w = afx.gated_weights(gate.info, gate.dev.data_ptr(), up.info, up.dev.data_ptr(), rows, cols)
    new = lambda k, std=1.0: torch.from_numpy(normal(rng, (m, k), std)).cuda()  # noqa: E731
    x, dh, d = new(cols).bfloat16(), new(rows), new(rows).bfloat16()
    bf = dict(dtype=torch.bfloat16, device="cuda")
    h, g, u, dg, du = (torch.zeros(m, rows, **bf) for _ in range(5))
    dx, y = torch.zeros(m, cols, **bf), torch.zeros(m, cols, device="cuda")
    sizes = [afx.afx_restore_gated_workspace(rows, cols, m), afx.afx_restore_gated_workspace(rows, cols, m, True),
             afx.afx_restore_gemm_t_workspace(rows, cols, m)]
    ws = workspace(max(sizes))  # one after another on one stream: they may share it

    def step():
        s = stream()
        afx.afx_restore_gated_async(w, m, x.data_ptr(), cols, h.data_ptr(), rows, g.data_ptr(), u.data_ptr(), rows,
                                    ws.data_ptr(), ws.numel(), s)
        afx.afx_restore_gated_backward_async(w, m, dh.data_ptr(), rows, g.data_ptr(), u.data_ptr(), rows,
                                             dx.data_ptr(), cols, dg.data_ptr(), du.data_ptr(), ws.data_ptr(),
                                             ws.numel(), s)
        afx.afx_restore_gemm_t_async(gate.info, gate.dev.data_ptr(), rows, cols, d.data_ptr(), m, y.data_ptr(), False,
                                     ws.data_ptr(), ws.numel(), s)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (h, g, u, dg, du, dx, y)
    for rep in range(3):
        x.copy_(new(cols)), dh.copy_(new(rows)), d.copy_(new(rows))
        step()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, k in zip(outs, want):
            assert torch.equal(o, k), f"replay {rep}"
