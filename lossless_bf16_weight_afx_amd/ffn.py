"""The feed-forward half of a decoder layer over coded weights, forward and
backward, from the library's entry points:

    xn  = norm(r; w_pre)                      afx_block_norm_async
    h   = act(xn Wg^T) * (xn Wu^T)            afx_restore_gated_async
    b   = h Wd^T                              afx_restore_gemm_async
    r'  = r + scale gate norm(b; w_post),
    xn' = norm(r'; w_next)                    afx_block_norm_async

and the gradients back from those of r' and xn' (the *_backward_async calls
and afx_restore_gemm_t_async). "Why Weight Offloading Slows Inference"
(section "Lossless compression") restores a weight's bits before the
computation that uses it; here that computation takes the coded weights
themselves, which are constants: only activations, norms and gates have
gradients.

This module only holds buffers and makes calls: everything is enqueued on the
current stream, which a HIP graph may capture, and nothing is allocated after
the constructor. One object serves one stream at a time, and with
training=True a forward() and its backward() take turns: backward() needs
what forward() kept, and writes over it.
"""
from __future__ import annotations

from . import afx


class FeedForward:
    """gate, up: (info, device blob) of [ff, d] matrices; down: of a [d, ff]
    one (d a multiple of 64, ff of 256). Norm weights and a gate are BF16
    device tensors [d]; w_post, block_gate and w_next may be None. All are on
    one device, where the calls run whichever device is current. Buffers are
    for up to max_tokens tokens; training keeps what backward() needs."""

    def __init__(self, gate, up, down, d: int, ff: int, w_pre, *, w_post=None, block_gate=None, w_next=None,
                 act: int = afx.ACT_SILU, eps: float = 1e-6, scale: float = 1.0, max_tokens: int, training=False):
        import torch

        if d % 64 or ff % 256 or d < 64 or ff < 256:
            raise ValueError(f"d {d} and ff {ff}: the down product takes multiples of 64 and 256")
        for (info, blob), shape in ((gate, (ff, d)), (up, (ff, d)), (down, (d, ff))):
            # (coded with another number of dimensions, the values are taken in order)
            if int(info.n_elems) != d * ff or (info.ndim == 2 and tuple(info.shape[:2]) != shape):
                raise ValueError(f"a matrix is not one of {shape[0]} x {shape[1]} values")
            if blob.device != w_pre.device:
                raise ValueError("the matrices and the norm weights are on one device")
            if not blob.is_contiguous() or blob.numel() * blob.element_size() < info.blob_bytes:
                raise ValueError(f"a blob of {info.blob_bytes} bytes is not whole in {blob.numel() * blob.element_size()}")
        if max_tokens < 1:
            raise ValueError("max_tokens must be at least 1")
        for t in (w_pre, w_post, block_gate, w_next):
            if t is not None and (t.dtype != torch.bfloat16 or t.shape != (d,) or not t.is_contiguous()
                                  or t.device != w_pre.device):
                raise ValueError(f"norm weights and the gate are contiguous BF16 [{d}] tensors on one device")
        self.gate, self.up, self.down, self.d, self.ff = gate, up, down, d, ff
        self.vectors = (w_pre, w_post, block_gate, w_next)  # (kept: the structs below hold addresses)
        addr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        self.weights = afx.gated_weights(gate[0], gate[1].data_ptr(), up[0], up[1].data_ptr(), ff, d, act)
        self.norm_in = afx.block_norm(d, eps, w_pre=addr(w_pre))
        self.norm_out = afx.block_norm(d, eps, scale, afx.TYPE_BF16, addr(w_post), addr(block_gate), 0, addr(w_next))
        self.max_tokens, dev = max_tokens, w_pre.device
        new = lambda n, t=torch.bfloat16: torch.empty((max_tokens, n), dtype=t, device=dev)  # noqa: E731
        self.xn, self.h, self.b, self.r_out = new(d), new(ff), new(d, torch.float32), new(d)
        self.xn_next = new(d) if w_next is not None else None
        # A workspace's size need not grow with the tokens: up to 128 of them other kernels take over, and from there
        # on the division of the work follows from how many tiles of 64, 128 and 256 tokens there are. It does grow
        # while the number of tiles of 64 stays, so the largest is at one of these.
        sizes = [afx.afx_restore_gated_workspace(ff, d, m) for m in self._sizes()]
        self.training = training
        self._kept = None  # training: the stream (address, stride, tokens) of the forward pass whose values are held
        self._captured = False  # whether that pass was captured into a graph
        if training:
            self.g, self.u, self.db, self.dxn, self.dr = new(ff), new(ff), new(d), new(d), new(d)
            self.dh = new(ff, torch.float32)
            vec = lambda t: None if t is None else torch.empty(d, device=dev)  # noqa: E731
            self.dw_pre, self.dw_post, self.dgate, self.dw_next = (vec(t) for t in self.vectors)
            for m in self._sizes():
                sizes += [afx.afx_restore_gated_workspace(ff, d, m, True), afx.afx_restore_gemm_t_workspace(d, ff, m),
                          afx.afx_block_norm_workspace(self.norm_in, m),
                          afx.afx_block_norm_workspace(self.norm_out, m)]
        self.ws = torch.empty(max(max(sizes), 16), dtype=torch.uint8, device=dev)

    def _sizes(self):
        n = self.max_tokens
        return sorted({*range(1, min(n, 256) + 1), *range(256, n + 1, 64), n})

    def _stream(self, m: int) -> int:
        import torch

        if not 1 <= m <= self.max_tokens:
            raise ValueError(f"{m} tokens: the buffers are for 1 to {self.max_tokens}")
        return torch.cuda.current_stream(self.ws.device).cuda_stream

    def _residual(self, t):
        import torch

        if t.dtype != torch.bfloat16 or t.dim() != 2 or t.shape[1] != self.d or t.stride(1) != 1 \
                or t.device != self.ws.device:
            raise ValueError(f"a residual stream is a BF16 [tokens, {self.d}] tensor on {self.ws.device}, rows whole")
        return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else self.d  # (one row's stride may be anything)

    def _own(self, ptr: int, ld: int, m: int) -> bool:
        """Whether rows of a stream lie in buffers that the passes write before they have read them: all, but r'
        without training."""
        end = ptr + 2 * ((m - 1) * ld + self.d)
        own = [self.xn, self.h, self.b, self.xn_next, self.ws]
        if self.training:
            own += [self.r_out, self.g, self.u, self.db, self.dxn, self.dr, self.dh]
        return any(t is not None and ptr < t.data_ptr() + t.numel() * t.element_size() and t.data_ptr() < end
                   for t in own)

    def forward(self, r):
        """r' and xn' (None without w_next) for the residual stream r, in this
        object's buffers (views of its first rows). r may not lie in them, but
        for r' of the last pass, without training (backward() reads r again)."""
        import torch

        m, (r_ptr, ld) = r.shape[0], self._residual(r)
        s, d, ff = self._stream(m), self.d, self.ff
        if self._own(r_ptr, ld, m):
            raise ValueError("the residual stream lies in buffers that this object writes before it has read them")
        g, u = (self.g.data_ptr(), self.u.data_ptr()) if self.training else (0, 0)
        xn_next = 0 if self.xn_next is None else self.xn_next.data_ptr()
        with torch.cuda.device(self.ws.device):
            if self.training:
                self._kept, self._captured = None, torch.cuda.is_current_stream_capturing()
            afx.afx_block_norm_async(self.norm_in, m, 0, 0, r_ptr, ld, 0, 0, self.xn.data_ptr(), d, s)
            afx.afx_restore_gated_async(self.weights, m, self.xn.data_ptr(), d, self.h.data_ptr(), ff, g, u, ff,
                                        self.ws.data_ptr(), self.ws.numel(), s)
            self.b[:m].zero_()
            afx.afx_restore_gemm_async(self.down[0], self.down[1].data_ptr(), d, ff, self.h.data_ptr(), m,
                                       self.b.data_ptr(), s)
            afx.afx_block_norm_async(self.norm_out, m, self.b.data_ptr(), d, r_ptr, ld, self.r_out.data_ptr(), d,
                                     xn_next, d, s)
        if self.training:
            self._kept = (r_ptr, ld, m)
        return self.r_out[:m], None if self.xn_next is None else self.xn_next[:m]

    def backward(self, r, dr_out, dxn_next=None):
        """dr, the gradient of r, from those of r' and xn', once after each
        forward(r), with the same r. dw_pre, dw_post, dgate and dw_next hold
        the vectors' gradients. (If a graph captured that pass, its replays
        are not seen here: they are taken to come before each backward() that
        is not captured.)"""
        import torch

        if not self.training:
            raise ValueError("the object was made without training=True")
        m, (r_ptr, ld), (dro, ld_dro) = r.shape[0], self._residual(r), self._residual(dr_out)
        dxo, ld_dxo = (0, 0) if dxn_next is None else self._residual(dxn_next)
        if dr_out.shape[0] != m or (dxn_next is not None and (dxn_next.shape[0] != m or self.xn_next is None)):
            raise ValueError("the gradients do not match the forward pass")
        s, d, ff, ws, n = self._stream(m), self.d, self.ff, self.ws.data_ptr(), self.ws.numel()
        if self._kept != (r_ptr, ld, m):
            raise ValueError("each backward() follows a forward() of its own" if self._kept is None else
                             "r is not the stream of the last forward pass")
        addr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
        with torch.cuda.device(self.ws.device):
            afx.afx_block_norm_backward_async(self.norm_out, m, self.b.data_ptr(), d, self.r_out.data_ptr(), d, dxo,
                                              ld_dxo, dro, ld_dro, self.dr.data_ptr(), d, self.db.data_ptr(), d,
                                              addr(self.dw_next), addr(self.dw_post), addr(self.dgate), ws, n, s)
            afx.afx_restore_gemm_t_async(self.down[0], self.down[1].data_ptr(), d, ff, self.db.data_ptr(), m,
                                         self.dh.data_ptr(), False, ws, n, s)
            if not self._captured or torch.cuda.is_current_stream_capturing():
                self._kept = None
            # dg and du take the places of g and u: with xn they give the gradients of the two matrices' products
            afx.afx_restore_gated_backward_async(self.weights, m, self.dh.data_ptr(), ff, self.g.data_ptr(),
                                                 self.u.data_ptr(), ff, self.dxn.data_ptr(), d, self.g.data_ptr(),
                                                 self.u.data_ptr(), ws, n, s)
            afx.afx_block_norm_backward_async(self.norm_in, m, 0, 0, r_ptr, ld, self.dxn.data_ptr(), d,
                                              self.dr.data_ptr(), d, self.dr.data_ptr(), d, 0, 0, addr(self.dw_pre), 0,
                                              0, ws, n, s)
        return self.dr[:m]
