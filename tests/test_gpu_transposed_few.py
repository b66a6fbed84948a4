"""GPU parity of the transposed products for few tokens (up to 64), where the coded matrix is multiplied as it is: small integers,
so that every FP32 sum is exact and the 64-bit result is the answer; and
infinities and NaN at the matrix's edges."""
import numpy as np
import pytest

from lossless_bf16_weight_afx_amd import afx
from test_gpu_gated import Coded, normal, rng_of, run_backward, say, stream, strided, workspace

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


# rows and columns that end inside a slab (32 x 128), one group, rows a wave's share does not reach, more column tiles
# than workgroups, more slabs down a tile than workgroups, segments that start in one chunk and end in the next
SHAPES = [(8, 32), (8, 256), (40, 96), (32, 128), (256, 160), (1000, 288), (72, 70016), (9000, 64), (520, 5152),
          (2056, 2080),
          # rows that start inside a group: fewer columns than one, windows of 96 of 128 decoded ones
          (8, 8), (48, 24), (40, 104), (1000, 296), (72, 70008), (9000, 72), (520, 5144), (2056, 2072)]


def product(mat, d, m, add):
    y = torch.full((m + 2, mat.cols), 5.0, device="cuda")
    n = afx.afx_restore_gemm_t_workspace(mat.rows, mat.cols, m)
    ws = workspace(n)
    afx.afx_restore_gemm_t_async(mat.info, mat.dev.data_ptr(), mat.rows, mat.cols, d.data_ptr(), m, y.data_ptr(), add,
                                 ws.data_ptr(), n, stream())
    torch.cuda.synchronize()
    assert bool((y[m:] == 5.0).all())
    return y[:m].cpu().double()


@pytest.mark.parametrize("m", [1, 5, 16, 17, 33, 64, 65])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_integers_exact(rows, cols, m):
    say(f"[gpu] case transposed product {rows}x{cols} m={m}")
    rng = rng_of(61, rows, cols, m)
    mat = Coded(rng.integers(-3, 4, (rows, cols)).astype(np.float32))
    d = torch.from_numpy(rng.integers(-2, 3, (m, rows))).to(torch.bfloat16).cuda()
    want = d.cpu().double() @ mat.w  # below 2^24
    assert torch.equal(product(mat, d, m, False), want)
    assert torch.equal(product(mat, d, m, True), want + 5)


@pytest.mark.parametrize("m", [20, 70, 300])
@pytest.mark.parametrize("cols", [136, 160])
def test_outputs_aligned_to_their_elements_only(cols, m):
    """y 4 bytes past a 16-byte boundary: the same bits as an aligned one."""
    rng = rng_of(64, cols, m)
    mat = Coded(normal(rng, (200, cols)))
    d = torch.from_numpy(normal(rng, (m, 200))).to(torch.bfloat16).cuda()
    n = afx.afx_restore_gemm_t_workspace(200, cols, m)
    ws, got = workspace(n), []
    for shift in (0, 1):
        for add in (False, True):
            y = torch.full((m * cols + 2,), 3.0, device="cuda")
            afx.afx_restore_gemm_t_async(mat.info, mat.dev.data_ptr(), 200, cols, d.data_ptr(), m,
                                         y.data_ptr() + 4 * shift, add, ws.data_ptr(), n, stream())
            torch.cuda.synchronize()
            assert bool((y[m * cols + shift:] == 3.0).all() and (y[:shift] == 3.0).all())
            got.append(y[shift:m * cols + shift].clone())
    assert torch.equal(got[0], got[2]) and torch.equal(got[1], got[3])


@pytest.mark.parametrize("m", [3, 40])
@pytest.mark.parametrize("rows,cols", [(40, 96), (200, 320), (40, 88), (200, 328)])
def test_infinities_and_nan_stay_in_their_columns(rows, cols, m):
    """Also in the last row, which the slab's rows past it repeat."""
    rng = rng_of(62, rows, m)
    w = rng.integers(-3, 4, (rows, cols)).astype(np.float32)
    w[rows - 1, 3], w[0, 40], w[rows - 1, cols - 1] = np.inf, -np.inf, np.nan
    mat = Coded(w)
    d = torch.from_numpy(rng.integers(1, 3, (m, rows))).to(torch.bfloat16).cuda()
    got, want = product(mat, d, m, False), d.cpu().double() @ mat.w
    assert torch.equal(torch.nan_to_num(got, nan=12345.0), torch.nan_to_num(want, nan=12345.0))


@pytest.mark.parametrize("m", [1, 20, 64])
@pytest.mark.parametrize("rows,cols,pad", [(24, 64, 0), (333, 2080, 0), (704, 96, 8), (704, 96, 3), (1, 8, 0),
                                           (35, 40, 0), (333, 2072, 5), (704, 104, 8)])
def test_both_matrices_of_a_gated_block(rows, cols, pad, m):
    """dx = dg Wg + du Wu from the dg and du that the call returns, whose BF16
    values are the product's operands: within the rounding of dx and of FP32
    sums of 2 rows terms."""
    say(f"[gpu] case gated gradient {rows}x{cols} m={m}")
    rng = rng_of(63, rows, cols, m)
    gate, up = (Coded(rng.standard_normal((rows, cols)).astype(np.float32) * 0.1) for _ in range(2))
    dh = strided(normal(rng, (m, rows)), rows, torch.float32)
    gu = [strided(normal(rng, (m, rows)), rows + pad, torch.bfloat16) for _ in range(2)]
    dx, dg, du = run_backward(gate, up, "silu", dh, gu, m)
    want = dg @ gate.w + du @ up.w
    size = dg.abs() @ gate.w.abs() + du.abs() @ up.w.abs()
    k = 2 * rows * 2.0 ** -24
    assert bool(((dx - want).abs() <= 2.0 ** -8 * want.abs() + 1.01 * k / (1 - k) * size).all())
