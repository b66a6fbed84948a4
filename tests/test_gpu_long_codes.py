"""GPU parity of the kernels that decode row segments (the gated block, its
gradients and the transposed product for few tokens) on matrices whose codes
are long: exponents spread over many values, and last rows of rare ones.

Every result here is one weight. A token that is 1 in one column (or a
gradient that is 1 in one row) picks it out, all other terms are zero times
a finite value, and BF16 and FP32 hold it exactly: results must be equal."""
import numpy as np
import pytest

from lossless_bf16_weight_afx_amd import afx, synth
from test_gpu_gated import Coded, rng_of, run_backward, run_forward, run_t, say, strided

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


def of_exponents(rng, exp):
    """Values of the given exponent fields, any sign and mantissa."""
    bits = (rng.integers(0, 2, exp.shape) << 15) | (exp << 7) | rng.integers(0, 128, exp.shape)
    return synth.bf16_bits_to_f32(bits.astype(np.uint16).ravel()).reshape(exp.shape)


def matrix(kind, rng, rows, cols):
    if kind == "spread":  # 160 exponents alike: more than 7 bits a code
        return of_exponents(rng, rng.integers(47, 207, (rows, cols)))
    exp = 120 + rng.integers(0, 2, (rows, cols))
    exp[-1] = rng.integers(60, 120, cols)  # rare ones: codes of up to 12 bits
    return of_exponents(rng, exp)


# a last segment that starts in one chunk and ends in the next, the tensor's last: of 256 columns (the gated block),
# of 128 and of a window of 128 that starts inside a group (the gradients); and others
SHAPES = [(19, 224), (37, 224), (43, 96), (3, 5472), (40, 104), (79, 104), (128, 256), (17, 40), (64, 1056)]


@pytest.mark.parametrize("m", [2, 16, 48, 64, 100, 128])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", ["spread", "rare last row"])
def test_forward_picks_columns(kind, rows, cols, m):
    say(f"[gpu] case long codes forward {kind} {rows}x{cols} m={m}")
    rng = rng_of(71, rows, cols)
    gate, up = (Coded(matrix(kind, rng, rows, cols)) for _ in range(2))
    for c0 in range(0, cols, m) if cols <= 1056 and m > 2 else (0, cols - m):
        at = np.arange(c0, c0 + m) % cols
        x = np.zeros((m, cols), np.float32)
        x[np.arange(m), at] = 1
        _, g, u = run_forward(gate, up, "silu", (strided(x, cols, torch.bfloat16), m), True)
        assert torch.equal(g, gate.w.T[at]) and torch.equal(u, up.w.T[at]), f"columns {c0}.."


def rows_of(rows, m):
    """Batches of m rows that reach all of them, or the first and last."""
    for r0 in range(0, rows, m) if m > 1 else (0, rows - 1):
        yield np.arange(r0, r0 + m) % rows


@pytest.mark.parametrize("m", [1, 5, 16, 17, 48, 64])
@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("kind", ["spread", "rare last row"])
def test_gradients_pick_rows(kind, rows, cols, m):
    """g = 0, u = 2: act' = 1/2 and act = 0, so dg = dh and du = 0. g = 32, u =
    0: the exact GELU is 32 there, so dg = 0 and du = 32 dh."""
    say(f"[gpu] case long codes backward {kind} {rows}x{cols} m={m}")
    rng = rng_of(72, rows, cols)
    gate, up = (Coded(matrix(kind, rng, rows, cols)) for _ in range(2))
    for at in rows_of(rows, m):
        for mat, g, u, one in ((gate, 0.0, 2.0, 1.0), (up, 32.0, 0.0, 1 / 32)):
            dh = np.zeros((m, rows), np.float32)
            dh[np.arange(m), at] = one
            gu = [strided(np.full((m, rows), v, np.float32), rows, torch.bfloat16) for v in (g, u)]
            dx, _, _ = run_backward(gate, up, "gelu", strided(dh, rows, torch.float32), gu, m)
            assert torch.equal(dx, mat.w[at]), f"rows {at[0]}.."


@pytest.mark.parametrize("m", [1, 5, 16, 17, 48, 64])
@pytest.mark.parametrize("rows,cols", [s for s in SHAPES if s[0] % 8 == 0] + [(8, 520), (24, 2744)])
@pytest.mark.parametrize("kind", ["spread", "rare last row"])
def test_transposed_product_picks_rows(kind, rows, cols, m):
    say(f"[gpu] case long codes transposed {kind} {rows}x{cols} m={m}")
    rng = rng_of(73, rows, cols)
    mat = Coded(matrix(kind, rng, rows, cols))
    for at in rows_of(rows, m):
        d = np.zeros((m, rows), np.float32)
        d[np.arange(m), at] = 1
        y, _ = run_t(mat, d, m)
        assert torch.equal(y, mat.w[at]), f"rows {at[0]}.."
