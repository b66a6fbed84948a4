"""The largest sizes that the attention over a paged cache takes, and the first
that it refuses, on the CPU: each call is refused before any HIP call, at the
limit for its query rows' alignment, which is looked at later."""
import pytest

from lossless_bf16_weight_afx_amd import afx, cache
from test_paged_abi import INVALID, MISALIGNED, UNSUPPORTED, at, call_attend, kv, refused, table

ROOM = 1024  # positions that the kernels may count behind a sequence's last


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_positions_stay_below_two_to_the_31(page):
    most = (2 ** 31 - ROOM) // page
    how = dict(kvp=kv(page_tokens=page), q=at(3) + 8)
    t = lambda n: table(page_tokens=page, max_pages=n, table_stride=n)  # noqa: E731
    refused(MISALIGNED, lambda: call_attend(t=t(most), **how))
    for n in (most + 1, (2 ** 31 - 16) // page):
        refused(UNSUPPORTED, lambda: call_attend(t=t(n), **how))
    how = dict(n_pages=4, page_tokens=page, max_seqs=1, max_tokens=1, device="meta")
    with pytest.raises(ValueError):
        cache.PagedCache(1, 1, 8, max_pages=most + 1, **how)


@pytest.mark.parametrize("dim, tile, most", [(64, 256, 2 ** 23), (128, 256, 2 ** 23), (136, 128, 2 ** 24),
                                             (256, 128, 2 ** 24)])
def test_one_launch_is_of_fewer_than_two_to_the_32_threads(dim, tile, most):
    """Two key-value heads of 256 query heads each; a prompt of m tokens has m 256 / tile tiles, and one for its end."""
    width = 512 * dim
    # (out is q, which is looked at later)
    how = dict(p=afx.attend(512, 0.1, True, 0, 2 ** 23, 1), kvp=kv(head_dim=dim), rows=1, qs=width, outs=width, out=at(3))
    m = (most // 2 - 2) * tile // 256
    while 2 * (m * 256 // tile + 1) < most:
        m += 1
    refused(UNSUPPORTED, lambda: call_attend(m=m, **how))
    refused(INVALID, lambda: call_attend(m=m - 1, **how))
