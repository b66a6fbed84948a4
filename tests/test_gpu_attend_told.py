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


@pytest.mark.parametrize("new", [1, 4, 60])
@pytest.mark.parametrize("length, told", [(9000, 520), (9000, 1000), (9000, 4400), (4097, 1030), (1331, 1300), (5003, 5000)])
@pytest.mark.parametrize("window", [0, 4321])
def test_sequences_longer_than_was_told(new, length, told, window):
    """More tokens than the parts that were planned: they are shared out anew, over as many parts."""
    b = Batch(length + told + new, [length, 300, 1025], [(0, new), (1, min(new, 3)), (2, 1)], kv_heads=1, group=4, page=64,
              spread=1.5)
    b.upload()
    b.run(scale=0.125, max_len=told, window=window)
    b.check()
