"""The attention half of a decoder layer over coded weights and a paged cache,
from the library's entry points:

    xn      = norm(r; w_pre)                      afx_block_norm_async
    q, k, v = xn Wq^T, xn Wk^T, xn Wv^T           afx_restore_gemm_batch_async
    q, k    = rotate(norm(q; w_q)), .. (k; w_k),
              k and v to the cache                afx_heads_async
    a       = softmax(s q K^T) V                  afx_attend_async
    b       = a Wo^T                              afx_restore_gemm_async
    r'      = r + scale gate norm(b; w_post),
    xn'     = norm(r'; w_next)                    afx_block_norm_async

It stands before ffn.FeedForward in a layer: r' is that one's r. As there,
this module only holds buffers and makes calls: everything is enqueued on the
current stream, which a HIP graph may capture, nothing is allocated after the
constructor, and the objects over one cache serve one stream at a time: they
share the memory for the products' outputs and the attention's workspace.
"""
from __future__ import annotations

import math

from . import afx
from .cache import PagedCache, Step


class Attention:
    """q, k, v, o: (info, device blob) of [q_heads dim, d], [kv_heads dim, d]
    (two) and [d, q_heads dim] matrices, for layer `layer` of the cache, whose
    kv_heads and head_dim they have (d and q_heads dim multiples of 256,
    kv_heads dim of 64). w_pre, w_post, block_gate and w_next are BF16 device
    tensors [d], w_q and w_k BF16 [dim], the heads' norms; all but w_pre may be
    None. freq: FP32 [pairs], the radians by which the pairs of a head turn per
    position (None: none does); axis: uint8 [pairs], the axis of position that
    each turns with, of n_axes. softmax_scale is dim^-1/2 if not told. Buffers
    are for steps of up to max_tokens tokens (the cache's, if not told)."""

    def __init__(self, q, k, v, o, d: int, cache: PagedCache, layer: int, q_heads: int, w_pre, *, w_q=None, w_k=None,
                 freq=None, axis=None, n_axes: int = 1, pairing: int = afx.ROPE_HALVES, softmax_scale: float | None = None,
                 window: int = 0, w_post=None, block_gate=None, w_next=None, eps: float = 1e-6, scale: float = 1.0,
                 max_tokens: int | None = None):
        import torch

        dim, kv_heads, dev = cache.head_dim, cache.kv_heads, cache.device
        nq, nk = q_heads * dim, kv_heads * dim
        max_tokens = cache.max_tokens if max_tokens is None else max_tokens
        if q_heads < 1 or q_heads > 1024 or q_heads % kv_heads or q_heads // kv_heads > 256:
            raise ValueError(f"{q_heads} query heads over {kv_heads} heads of keys: a multiple of up to 256, 1024 at most")
        if d < 256 or d % 256 or nq % 256 or nk % 64:
            raise ValueError(f"d {d} and heads of {nq} and {nk} values: the products take multiples of 256, 256 and 64")
        for (info, blob), shape in ((q, (nq, d)), (k, (nk, d)), (v, (nk, d)), (o, (d, nq))):
            # (coded with another number of dimensions, the values are taken in order)
            if int(info.n_elems) != shape[0] * shape[1] or (info.ndim == 2 and tuple(info.shape[:2]) != shape):
                raise ValueError(f"a matrix is not one of {shape[0]} x {shape[1]} values")
            if blob.device != dev:
                raise ValueError("the matrices are on the cache's device")
            if not blob.is_contiguous() or blob.numel() * blob.element_size() < info.blob_bytes:
                raise ValueError(f"a blob of {info.blob_bytes} bytes is not whole in {blob.numel() * blob.element_size()}")
        if d > afx.MAX_NORM_WIDTH or not (0 < eps < math.inf and math.isfinite(scale)):
            raise ValueError(f"norms of up to {afx.MAX_NORM_WIDTH} values, eps {eps} above 0, scale {scale} finite")
        if not 1 <= max_tokens <= cache.max_tokens:
            raise ValueError(f"{max_tokens} tokens: the cache's steps are of 1 to {cache.max_tokens}")
        pairs = 0 if freq is None else freq.numel()
        if 2 * pairs > dim or not 1 <= n_axes <= 4 or pairing not in (afx.ROPE_HALVES, afx.ROPE_NEIGHBOURS) \
                or (axis is not None and freq is None) or window < 0:
            raise ValueError(f"{pairs} pairs of {dim} values turning with {n_axes} axes, window {window}")
        for t, n, kind in ((w_pre, d, torch.bfloat16), (w_post, d, torch.bfloat16), (block_gate, d, torch.bfloat16),
                           (w_next, d, torch.bfloat16), (w_q, dim, torch.bfloat16), (w_k, dim, torch.bfloat16),
                           (freq, pairs, torch.float32), (axis, pairs, torch.uint8)):
            if t is not None and (t.dtype != kind or t.shape != (n,) or not t.is_contiguous() or t.device != dev):
                raise ValueError(f"norm weights, the gate, frequencies and axes are contiguous tensors on {dev}: here "
                                 f"{kind} [{n}]")
        self.q, self.k, self.v, self.o, self.d, self.cache = q, k, v, o, d, cache
        self.vectors = (w_pre, w_post, block_gate, w_next, w_q, w_k, freq, axis)  # (kept: the structs hold addresses)
        addr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        self.kv, self.nq, self.nk, self.n_axes = cache.layer(layer), nq, nk, n_axes
        self.norm_in = afx.block_norm(d, eps, w_pre=addr(w_pre))
        self.norm_out = afx.block_norm(d, eps, scale, afx.TYPE_BF16, addr(w_post), addr(block_gate), 0, addr(w_next))
        self.heads = afx.heads(q_heads, kv_heads, dim, 2 * pairs, pairing, n_axes, eps, addr(w_q), addr(w_k), addr(freq),
                               addr(axis))
        self.softmax_scale = dim ** -0.5 if softmax_scale is None else softmax_scale
        self.q_heads, self.window, self.max_tokens = q_heads, window, max_tokens
        new = lambda n: torch.empty((max_tokens, n), dtype=torch.bfloat16, device=dev)  # noqa: E731
        self.xn, self.qn, self.a, self.r_out = new(d), new(nq), new(nq), new(d)
        self.xn_next = new(d) if w_next is not None else None
        # the products' FP32 outputs of a step of m tokens, cleared at once: m rows of q, of k, of v, of b
        self.y = cache.scratch("products", 4 * max_tokens * (nq + 2 * nk + d)).view(torch.float32)
        self.ws = cache.scratch("attention", max(max(self._workspaces()), 16))

    def _attend(self, max_new: int, max_len: int) -> afx.afx_attend:
        return afx.attend(self.q_heads, self.softmax_scale, True, self.window, max_new, max_len)

    def _plan(self, max_new: int, max_len: int, n: int, m: int) -> afx.afx_attend:
        """The attention of m new tokens of n sequences. Steps of unusual sizes, that the workspace was not made for,
        are cut into fewer parts, as if their sequences were shorter, or into one, which needs none."""
        size = lambda p: afx.afx_attend_workspace(p, self.kv, n, m)  # noqa: E731
        p = self._attend(max_new, max_len)
        if size(p) > self.ws.numel():
            shorter = (self._attend(max_new, max_len >> i) for i in range(1, max_len.bit_length()))
            p = next((s for s in shorter if 0 < size(s) <= self.ws.numel()), self._attend(max_new, 1))
        return p

    def _workspaces(self):
        """The workspaces of single tokens and of drafts of some tokens for every number of rows, and of prompts, over
        sequences of the cache's most tokens and of shorter ones (which may be cut into more parts)."""
        rows, whole = min(self.cache.max_rows, self.max_tokens), self.cache.max_pages * self.cache.page_tokens
        sizes = [(new, n, n * new) for n in range(1, rows + 1) for new in (1, 2, 4, 8) if n * new <= self.max_tokens]
        sizes += [(m, n, m) for m in {*range(16, self.max_tokens + 1, 16), self.max_tokens}
                  for n in {1, min(4, rows), min(64, rows), rows}]
        lens = [256 << i for i in range(whole.bit_length()) if 256 << i < whole] + [whole]
        for new, n, m in sizes:
            for length in lens:
                yield afx.afx_attend_workspace(self._attend(new, length), self.kv, n, m)

    def _own(self, ptr: int, ld: int, m: int) -> bool:
        """Whether rows of a stream lie in buffers that the pass writes before it has read them: all but r', which is
        written row by row in the places of its own rows."""
        end = ptr + 2 * ((m - 1) * ld + self.d)
        own = [self.xn, self.qn, self.a, self.xn_next, self.y, self.ws, self.cache.data]
        if ptr != self.r_out.data_ptr() or ld != self.d:
            own.append(self.r_out[:m])
        return any(t is not None and ptr < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < end
                   for t in own)

    def forward(self, r, step: Step, pos=None):
        """r' and xn' (None without w_next) for the residual stream r of a
        step's new tokens, in this object's buffers (views of its first rows);
        their keys and values are in the cache's layer afterwards. pos: int32
        [n_axes, tokens], the tokens' positions, if they are not their places
        in their sequences (each axis a row of its own in memory, also where
        axes agree). r may not lie in this object's buffers, but for r' of the
        last pass, from its first row on (or rows behind the new tokens')."""
        import torch

        m, c = r.shape[0], self.cache
        if r.dtype != torch.bfloat16 or r.dim() != 2 or r.shape[1] != self.d or r.stride(1) != 1 or r.device != c.device:
            raise ValueError(f"a residual stream is a BF16 [tokens, {self.d}] tensor on {c.device}, rows whole")
        if step.cache is not c or step.m != m:
            raise ValueError("the step is not one of this many tokens in this cache")
        if step.number != c.number:
            raise ValueError("the cache was called since the step began")
        if not 1 <= m <= self.max_tokens:
            raise ValueError(f"{m} tokens: the buffers are for 1 to {self.max_tokens}")
        if pos is None and self.n_axes > 1:
            raise ValueError(f"positions along {self.n_axes} axes have to be told")
        if pos is not None and (pos.dtype != torch.int32 or pos.shape != (self.n_axes, m) or pos.stride(1) != 1
                                or (self.n_axes > 1 and pos.stride(0) < m) or pos.device != c.device):
            raise ValueError(f"positions are an int32 [{self.n_axes}, {m}] tensor on {c.device}, rows whole and each in "
                             "memory of its own (not expanded)")
        r_ptr, ld = r.data_ptr(), r.stride(0) if m > 1 else self.d  # (one row's stride may be anything)
        if self._own(r_ptr, ld, m):
            raise ValueError("the residual stream lies in buffers that this object writes before it has read them")
        d, nq, nk, n = self.d, self.nq, self.nk, step.seqs.numel()
        y = self.y.data_ptr()
        q, k, v, b = y, y + 4 * m * nq, y + 4 * m * (nq + nk), y + 4 * m * (nq + 2 * nk)
        pos_ptr, pos_ld = (step.pos if pos is None else pos).data_ptr(), pos.stride(0) if self.n_axes > 1 else m
        xn, xn_next = self.xn.data_ptr(), 0 if self.xn_next is None else self.xn_next.data_ptr()
        p = self._plan(step.max_new, step.max_len, n, m)
        s = torch.cuda.current_stream(c.device).cuda_stream
        with torch.cuda.device(c.device):
            self.y[:m * (nq + 2 * nk + d)].zero_()
            afx.afx_block_norm_async(self.norm_in, m, 0, 0, r_ptr, ld, 0, 0, xn, d, s)
            afx.afx_restore_gemm_batch_async([(self.q[0], self.q[1].data_ptr(), nq, d, xn, q),
                                              (self.k[0], self.k[1].data_ptr(), nk, d, xn, k),
                                              (self.v[0], self.v[1].data_ptr(), nk, d, xn, v)], m, s)
            afx.afx_heads_async(self.heads, m, pos_ptr, pos_ld, q, nq, k, nk, v, nk, self.qn.data_ptr(), nq, 0, 0,
                                self.kv, step.slots.data_ptr(), s)
            afx.afx_attend_async(p, self.kv, c.pages, n, step.seqs.data_ptr(), step.starts.data_ptr(), m,
                                 self.qn.data_ptr(), nq, self.a.data_ptr(), nq, 0, self.ws.data_ptr(), self.ws.numel(), s)
            afx.afx_restore_gemm_async(self.o[0], self.o[1].data_ptr(), d, nq, self.a.data_ptr(), m, b, s)
            afx.afx_block_norm_async(self.norm_out, m, b, d, r_ptr, ld, self.r_out.data_ptr(), d, xn_next, d, s)
        return self.r_out[:m], None if self.xn_next is None else self.xn_next[:m]
