"""The gated block's gradients for pre-activations far from zero, up to the
largest BF16 value: act' is 0 or 1 there and act(g) is 0 or g, exactly (in
FP32 the sigmoids and the Gaussian are at their limits from |g| = 104 on)."""
import numpy as np
import pytest

from lossless_bf16_weight_afx_amd import afx
from test_gpu_gated import ACTS, Coded, normal, rng_of, run_backward, say, strided

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LARGEST = float(torch.finfo(torch.bfloat16).max)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


@pytest.mark.parametrize("m", [3, 70])
@pytest.mark.parametrize("act", list(ACTS))
def test_gradients_at_their_limits(act, m):
    say(f"[gpu] case far gradients {act} m={m}")
    rows, cols = 40, 64
    rng = rng_of(81, m)
    gate, up = (Coded(normal(rng, (rows, cols), 2.0 ** -10)) for _ in range(2))
    size = np.exp(rng.uniform(np.log(128.0), np.log(LARGEST), (m, rows)))
    size[0, :8] = [128, 1e5, 1e10, 1e12, 1.8e19, 1.9e19, 1e30, LARGEST]
    g = strided(np.where(rng.random((m, rows)) < 0.5, -size, size).astype(np.float32), rows, torch.bfloat16)
    g[0, :8] = g[0, :8].abs()
    u = strided(rng.integers(1, 5, (m, rows)).astype(np.float32), rows, torch.bfloat16)
    dh = strided(np.exp2(-rng.integers(0, 4, (m, rows))).astype(np.float32), rows, torch.float32)
    g64, u64, dh64 = (v[:m].cpu().double() for v in (g, u, dh))
    _, dg, du = run_backward(gate, up, act, dh, (g, u), m)
    on = (g64 > 0).double()
    assert torch.equal(dg, dh64 * u64 * on)
    assert torch.equal(du, dh64 * g64 * on)
