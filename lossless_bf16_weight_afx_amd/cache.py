"""A paged cache of keys and values, and the calls that grow, fork, trim and
compact it on the GPU:

    extend    afx_pages_extend_async    new tokens get slots, pages as needed
    fork      afx_pages_fork_async      sequences that share another's pages
    trim      afx_pages_trim_async      sequences keep their first tokens, or none
    compact   afx_pages_compact_async   the live pages move to the lowest ids

Which pages a sequence has, its length and the pages' counts live on the
device and are changed there: nothing waits, nothing is copied to the host,
and nothing is allocated after the constructor, so that a HIP graph may
capture whole steps of generation. Everything is enqueued on the current
stream; one cache serves one stream at a time.
"""
from __future__ import annotations

from typing import NamedTuple

from . import afx


class Step(NamedTuple):
    """The new tokens of one step: row r's are starts[r] .. starts[r + 1] - 1
    of m, and belong to sequence seqs[r]; max_new and max_len are the most of
    one row and the most tokens of one sequence after them. slots, pos and
    granted are views of the cache's buffers: a step ends with the cache's
    next call. A row whose granted is not its number of tokens was refused
    (see afx.h): its tokens have no slots, and what is computed for them is of
    no use; the same goes for tokens behind the last row's."""
    cache: "PagedCache"
    seqs: object
    starts: object
    m: int
    max_new: int
    slots: object
    pos: object
    granted: object
    number: int
    max_len: int


class PagedCache:
    """Keys and values of `layers` layers for max_seqs sequences of up to
    max_pages pages of page_tokens tokens, from a pool of n_pages; steps are
    of up to max_rows sequences and max_tokens new tokens. Sequences and rows
    are named by int32 device tensors."""

    def __init__(self, layers: int, kv_heads: int, head_dim: int, *, n_pages: int, page_tokens: int = 64,
                 max_seqs: int, max_pages: int, max_tokens: int, max_rows: int | None = None, device="cuda"):
        import torch

        max_rows = min(max_seqs, afx.MAX_PAGE_ROWS) if max_rows is None else max_rows
        if min(layers, kv_heads, head_dim, n_pages, max_seqs, max_pages, max_tokens, max_rows) < 1:
            raise ValueError("every size must be at least 1")
        if kv_heads > 1024 or head_dim % 8 or head_dim > afx.MAX_HEAD_DIM or page_tokens not in (16, 32, 64, 128, 256):
            raise ValueError(f"{kv_heads} heads of {head_dim} in pages of {page_tokens} tokens: at most 1024 heads, of a "
                             f"multiple of 8 up to {afx.MAX_HEAD_DIM}, and pages of 16, 32, 64, 128 or 256")
        if max_rows > afx.MAX_PAGE_ROWS or max_seqs > 1 << 20 or max_tokens > 1 << 23:
            raise ValueError(f"at most {afx.MAX_PAGE_ROWS} rows, 2^20 sequences and 2^23 tokens")
        if n_pages * page_tokens >= 1 << 31 or max_pages * page_tokens > (1 << 31) - 1024 or 2 * layers > 65535:
            raise ValueError("a pool is of fewer than 2^31 tokens, a sequence of up to 2^31 - 1024, and a cache of at most "
                             "32767 layers")
        self.layers, self.kv_heads, self.head_dim = layers, kv_heads, head_dim
        self.n_pages, self.page_tokens, self.max_pages = n_pages, page_tokens, max_pages
        self.max_seqs, self.max_rows, self.max_tokens = max_seqs, max_rows, max_tokens
        per_page = kv_heads * head_dim * page_tokens
        # planes 2 i and 2 i + 1: layer i's keys and values
        self.data = torch.empty((2 * layers, n_pages * per_page), dtype=torch.bfloat16, device=device)
        self.device = self.data.device
        new = lambda *n: torch.zeros(n, dtype=torch.int32, device=self.device)  # noqa: E731
        self.table, self.len, self.refs = new(max_seqs, max_pages).fill_(-1), new(max_seqs), new(n_pages)
        self.slots, self.pos, self.granted = new(max_tokens), new(max_tokens), new(max_rows)
        self.map, self.live = new(n_pages), new(1)
        self.number = 0  # calls so far
        self._scratch = {}
        self.pages = afx.page_table(self.table.data_ptr(), max_pages, self.len.data_ptr(), self.refs.data_ptr(), max_seqs,
                                    max_pages, n_pages, page_tokens)
        self.planes = afx.page_data(self.data.data_ptr(), 2 * per_page, 2 * per_page * n_pages, 2 * layers)
        sizes = [afx.afx_pages_extend_workspace(self.pages, n) for n in range(1, max_rows + 1)]
        sizes.append(afx.afx_pages_compact_workspace(self.pages))
        self.ws = torch.empty(max(max(sizes), 16), dtype=torch.uint8, device=self.device)

    def layer(self, i: int) -> afx.afx_kv_pages:
        """Layer i's keys and values (afx_heads_async, afx_attend_async)."""
        if not 0 <= i < self.layers:
            raise ValueError(f"layer {i} of {self.layers}")
        at = self.data.data_ptr() + 2 * i * self.planes.plane_stride
        return afx.kv_pages(at, at + self.planes.plane_stride, self.n_pages, self.page_tokens, self.kv_heads, self.head_dim)

    def scratch(self, what: str, n: int):
        """n bytes on the device for what a layer's pass over this cache forms
        and uses up. Passes follow one another on the cache's stream: those of
        all layers share them. For constructors: what a larger n replaces stays
        with those who hold it."""
        import torch

        if what not in self._scratch or self._scratch[what].numel() < n:
            self._scratch[what] = torch.empty(n, dtype=torch.uint8, device=self.device)
        return self._scratch[what][:n]

    def _list(self, t, what: str, n: int | None = None) -> int:
        import torch

        if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.device != self.device:
            raise ValueError(f"{what}: an int32 tensor [rows] on {self.device}, without gaps")
        if (n is None and not 1 <= t.numel() <= self.max_rows) or (n is not None and t.numel() != n):
            raise ValueError(f"{what}: {t.numel()} values" + (f", not 1 to {self.max_rows}" if n is None else f", not {n}"))
        return t.data_ptr()

    def _stream(self) -> int:
        import torch

        self.number += 1
        return torch.cuda.current_stream(self.device).cuda_stream

    def extend(self, seqs, starts, m: int, max_new: int | None = None, max_len: int | None = None) -> Step:
        """Sequences grow by the new tokens of their rows: row r's are
        starts[r] .. starts[r + 1] - 1 of m. max_new (m if not told) is the most
        of one row, max_len (all that the cache can hold of a sequence if not
        told) the most tokens of one sequence afterwards. Attention divides its
        work by them: rows and sequences that have more come out right too, but
        numbers far from the truth cost time, of single tokens over a long
        cache most of it. A captured step keeps the numbers that it was
        captured with: tell the most that its replays will meet."""
        import torch

        s, n = self._list(seqs, "seqs"), seqs.numel()
        at = self._list(starts, "starts", n + 1)
        if not 1 <= m <= self.max_tokens:
            raise ValueError(f"{m} tokens: the buffers are for 1 to {self.max_tokens}")
        max_new = m if max_new is None else max_new
        if not 1 <= max_new <= m:
            raise ValueError(f"at most {max_new} of {m} tokens in a row")
        most = self.max_pages * self.page_tokens
        max_len = most if max_len is None else max_len
        if not 1 <= max_len <= most:
            raise ValueError(f"at most {max_len} tokens of a sequence: the cache holds 1 to {most}")
        with torch.cuda.device(self.device):
            afx.afx_pages_extend_async(self.pages, self.planes, n, s, at, m, self.slots.data_ptr(), self.pos.data_ptr(),
                                       self.granted.data_ptr(), self.ws.data_ptr(), self.ws.numel(), self._stream())
        return Step(self, seqs, starts, m, max_new, self.slots[:m], self.pos[:m], self.granted[:n], self.number,
                    max_len)

    def fork(self, src, dst):
        """Sequences dst, which hold nothing, become copies of src that share
        its pages. Returns 1 or 0 a row (a view of this cache's buffer)."""
        import torch

        s, n = self._list(src, "src"), src.numel()
        d = self._list(dst, "dst", n)
        with torch.cuda.device(self.device):
            afx.afx_pages_fork_async(self.pages, n, s, d, self.granted.data_ptr(), self._stream())
        return self.granted[:n]

    def trim(self, seqs, lens) -> None:
        """Sequences keep their first lens tokens."""
        import torch

        s = self._list(seqs, "seqs")
        keep = self._list(lens, "lens", seqs.numel())
        with torch.cuda.device(self.device):
            afx.afx_pages_trim_async(self.pages, seqs.numel(), s, keep, self._stream())

    def free(self, seqs) -> None:
        """Sequences give up all of their pages."""
        import torch

        s = self._list(seqs, "seqs")
        with torch.cuda.device(self.device):
            afx.afx_pages_trim_async(self.pages, seqs.numel(), s, 0, self._stream())

    def compact(self):
        """The live pages move to the lowest ids. Returns each page's new id
        (-1: it was free) and their number (views of this cache's buffers)."""
        import torch

        with torch.cuda.device(self.device):
            afx.afx_pages_compact_async(self.pages, self.planes, self.map.data_ptr(), self.live.data_ptr(),
                                        self.ws.data_ptr(), self.ws.numel(), self._stream())
        return self.map, self.live
