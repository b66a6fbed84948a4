"""Attention told more tokens and new tokens than there can be, where many
key-value heads leave a single row's tokens in one part."""
import pytest

from lossless_bf16_weight_afx_amd import afx
from test_gpu_attend import Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("max_len", [2 ** 31 - 1024, 2 ** 31, 2 ** 32 - 1])
def test_lengths_that_no_sequence_has(new, max_len):
    b = Batch(new, [700], [(0, new)], kv_heads=256, group=1, dim=8)
    b.upload()
    b.run(scale=0.3, max_len=max_len)
    b.check()
