"""The gated block and the transposed product on a matrix of more than 2^32
weights: element offsets, byte offsets and row indices pass 32 bits. Small
integers keep every FP32 sum exact, and the weights repeat with a period prime
to the chunk size and the row length; the reference multiplies the matrix as
the library's restore gives it (held to the original bits here at both ends
and around element 2^32) in FP32."""
import sys

import numpy as np
import pytest

from lossless_bf16_weight_afx_amd import afx, synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def say(*a):
    print(*a, file=sys.stderr, flush=True)


@pytest.fixture(scope="module")
def matrix():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rows, cols, period = 1_048_640, 4096, (1 << 24) + 4099
    n = rows * cols
    vals = np.random.default_rng(98).integers(-3, 4, size=period).astype(np.float32)
    pat = synth.f32_to_bf16_bits(vals)
    say("[gpu] generate and encode 2^32+ weights")
    w = np.empty(n, np.uint16)
    for o in range(0, n, period):
        w[o:o + period] = pat[:min(period, n - o)]
    blob = afx.afx_encode(w, (rows, cols))
    info, dev = afx.afx_query(blob), afx.to_device(blob)
    wide = afx.decode(info, dev).view(torch.bfloat16)
    for a in (0, (1 << 32) - 5000, n - 5000):
        assert np.array_equal(wide[a:a + 5000].view(torch.int16).cpu().numpy().view(np.uint16), w[a:a + 5000])
    del w, blob
    yield info, dev, wide.view(rows, cols), rows, cols
    del dev, wide
    torch.cuda.empty_cache()


def blocks(rows, step=1 << 16):
    return [slice(a, min(a + step, rows)) for a in range(0, rows, step)]


@pytest.mark.parametrize("m", [2, 8, 130])
def test_gated(matrix, m):
    info, dev, wide, rows, cols = matrix
    say(f"[gpu] case gated block {rows}x{cols}, m={m}")
    x = torch.from_numpy(np.random.default_rng(m).integers(-2, 3, (m, cols))).to(torch.bfloat16).cuda()
    h, g, u = (torch.empty(m, rows, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    n = afx.afx_restore_gated_workspace(rows, cols, m)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    weights = afx.gated_weights(info, dev.data_ptr(), info, dev.data_ptr(), rows, cols)
    afx.afx_restore_gated_async(weights, m, x.data_ptr(), cols, h.data_ptr(), rows, g.data_ptr(), u.data_ptr(), rows,
                                ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(g, u)
    for b in blocks(rows):
        want = x.float() @ wide[b].float().t()  # exact: below 2^24
        assert torch.equal(g[:, b], want.to(torch.bfloat16)), f"rows from {b.start}"
        exact = want.double()  # h: half a BF16 step, and the FP32 activation's error as in test_gpu_gated.py
        err = (h[:, b].double() - exact * exact / (1 + torch.exp(-exact))).abs()
        assert bool((err <= (2.0 ** -8 + 2.0 ** -17 * (1 + exact.abs())) * exact * exact).all())


@pytest.mark.parametrize("m", [2, 20, 70])
def test_transposed(matrix, m):
    info, dev, wide, rows, cols = matrix
    say(f"[gpu] case transposed product {rows}x{cols}, m={m}")
    d = torch.from_numpy(np.random.default_rng(m).integers(-2, 3, (m, rows))).to(torch.bfloat16).cuda()
    y = torch.empty(m, cols, device="cuda")
    n = afx.afx_restore_gemm_t_workspace(rows, cols, m)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    afx.afx_restore_gemm_t_async(info, dev.data_ptr(), rows, cols, d.data_ptr(), m, y.data_ptr(), False,
                                 ws.data_ptr(), n, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    want = torch.zeros(m, cols, device="cuda")
    for b in blocks(rows):
        want += d[:, b].float() @ wide[b].float()
    assert float(want.abs().max()) < 2 ** 24
    assert torch.equal(y, want)
