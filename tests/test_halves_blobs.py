"""Blobs that a layer's halves refuse when they are made (CPU): kernels read as
many bytes as the info says, wherever the tensor ends."""
import pytest

from lossless_bf16_weight_afx_amd import attn, ffn
from test_attn import calls, info, paged, refused  # noqa: F401

torch = pytest.importorskip("torch")


def matrices(shapes, blobs):
    """(info, blob) of each shape, all infos of blobs of 640 bytes."""
    out = []
    for (rows, cols), blob in zip(shapes, blobs):
        i = info(rows, cols)
        i.blob_bytes = 640
        out.append((i, blob))
    return out


WHOLE = torch.zeros(640, dtype=torch.uint8)
BAD = [torch.zeros(639, dtype=torch.uint8), torch.zeros(159, dtype=torch.int32), torch.zeros(0, dtype=torch.uint8),
       torch.zeros(1280, dtype=torch.uint8)[::2]]
GOOD = [WHOLE, torch.zeros(160, dtype=torch.int32), torch.zeros(1000, dtype=torch.uint8)]


def attention(blobs):
    shapes = ((256, 256), (128, 256), (128, 256), (256, 256))
    return attn.Attention(*matrices(shapes, blobs), 256, paged(), 0, 4, torch.ones(256, dtype=torch.bfloat16))


def feed_forward(blobs):
    shapes = ((256, 64), (256, 64), (64, 256))
    return ffn.FeedForward(*matrices(shapes, blobs), 64, 256, torch.ones(64, dtype=torch.bfloat16), max_tokens=4)


@pytest.mark.parametrize("half, n", [(attention, 4), (feed_forward, 3)])
def test_blobs_that_are_not_whole(calls, half, n):  # noqa: F811
    for i in range(n):
        for bad in BAD:
            refused(calls, half, [bad if k == i else WHOLE for k in range(n)])
        for good in GOOD:
            half([good if k == i else WHOLE for k in range(n)])
