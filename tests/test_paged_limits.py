"""The largest sizes that the attention over a paged cache takes, and the first
that it refuses, on the CPU: each call is refused before any HIP call, at the
limit for its query rows' alignment, which is looked at later."""
import pytest

from lossless_bf16_weight_afx_amd import cache
from test_paged_abi import MISALIGNED, UNSUPPORTED, at, call_attend, kv, refused, table

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
