"""Buffers that are column ranges of one wider matrix (gate and up
projections kept as the halves of one, the norms' outputs side by side):
they share no byte, and give the bits that buffers of their own do."""
import numpy as np
import pytest

from lossless_bf16_weight_afx_amd import afx
from test_gpu_gated import Coded, normal, rng_of, say, stream, workspace

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


@pytest.mark.parametrize("rows,cols", [(136, 160), (51, 72), (64, 256)])
@pytest.mark.parametrize("m", [1, 3, 16, 64, 100, 300])
def test_gated_halves(m, rows, cols):
    say(f"[gpu] case interleaved {rows}x{cols} m={m}")
    rng = rng_of(91, rows, m)
    gate, up = (Coded(normal(rng, (rows, cols), 0.1)) for _ in range(2))
    w = afx.gated_weights(gate.info, gate.dev.data_ptr(), up.info, up.dev.data_ptr(), rows, cols)
    x = torch.from_numpy(normal(rng, (m, cols))).bfloat16().cuda()
    dh = torch.from_numpy(normal(rng, (m, rows))).cuda()
    ws = workspace(max(afx.afx_restore_gated_workspace(rows, cols, m, b) for b in (False, True)))
    n, gap = ws.numel(), 5

    def passes(h, g, u, dg, du):
        dx = torch.zeros(m, cols, dtype=torch.bfloat16, device="cuda")
        afx.afx_restore_gated_async(w, m, x.data_ptr(), cols, h.data_ptr(), h.stride(0), g.data_ptr(), u.data_ptr(),
                                    g.stride(0), ws.data_ptr(), n, stream())
        got = [t.clone() for t in (h, g, u)]
        afx.afx_restore_gated_backward_async(w, m, dh.data_ptr(), rows, g.data_ptr(), u.data_ptr(), g.stride(0),
                                             dx.data_ptr(), cols, dg.data_ptr(), du.data_ptr(), ws.data_ptr(), n,
                                             stream())
        torch.cuda.synchronize()
        return got + [t.clone() for t in (dg, du, dx)]

    new = lambda k: torch.full((m, k), -7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    want = passes(*(new(rows) for _ in range(5)))
    for in_place in (False, True):
        wide = new(5 * rows + gap)
        part = [wide[:, i * rows:(i + 1) * rows] for i in range(5)]
        got = passes(*part[:3], *(part[1:3] if in_place else part[3:]))
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        assert bool((wide[:, 5 * rows:] == -7.0).all()) and (not in_place or bool((wide[:, 3 * rows:] == -7.0).all()))


@pytest.mark.parametrize("d", [40, 600, 1001])
@pytest.mark.parametrize("m", [1, 9])
def test_norm_outputs_side_by_side(m, d):
    rng = rng_of(92, d, m)
    bf = lambda *s: torch.from_numpy(normal(rng, s)).bfloat16().cuda()  # noqa: E731
    b, w_post, w_pre, gate = torch.from_numpy(normal(rng, (m, d))).cuda(), bf(d), bf(d), bf(d)
    p = afx.block_norm(d, 1e-5, 0.5, afx.TYPE_BF16, w_post.data_ptr(), gate.data_ptr(), 0, w_pre.data_ptr())
    dxn, dro, r = bf(m, d), bf(m, d), bf(m, d)
    ws = workspace(afx.afx_block_norm_workspace(p, m))

    def passes(r_in, ro, xn, dr, db):
        afx.afx_block_norm_async(p, m, b.data_ptr(), d, r_in.data_ptr(), r_in.stride(0), ro.data_ptr(), ro.stride(0),
                                 xn.data_ptr(), xn.stride(0), stream())
        dw = [torch.zeros(d, device="cuda") for _ in range(3)]
        afx.afx_block_norm_backward_async(p, m, b.data_ptr(), d, ro.data_ptr(), ro.stride(0), dxn.data_ptr(), d,
                                          dro.data_ptr(), d, dr.data_ptr(), dr.stride(0), db.data_ptr(), db.stride(0),
                                          *(t.data_ptr() for t in dw), ws.data_ptr(), ws.numel(), stream())
        torch.cuda.synchronize()
        return [t.clone() for t in (ro, xn, dr, db, *dw)]

    new = lambda k: torch.full((m, k), -7.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    # (buffers of their own with the same row distance: it decides how a row's values are dealt to the lanes, and
    # with that the order of a row's sums)
    want = passes(r, *(new(5 * d + 3)[:, :d] for _ in range(4)))
    wide = new(5 * d + 3)
    part = [wide[:, i * d:(i + 1) * d] for i in range(5)]
    part[0].copy_(r)
    for a, k in zip(passes(*part), want):
        assert torch.equal(a, k)
    assert torch.equal(part[0], r) and bool((wide[:, 5 * d:] == -7.0).all())
