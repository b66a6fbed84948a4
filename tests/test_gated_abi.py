"""The gated feed-forward block, the transposed product and the block norms on
the CPU: every refusal comes before any HIP call (the device addresses here
are made up and never dereferenced)."""
import ctypes

import numpy as np
import pytest

import oracle
from lossless_bf16_weight_afx_amd import afx, synth

MB = 1 << 20
# made-up, widely spaced, 256-byte aligned device addresses
GATE, UP, X, H, G, U, DH, DX, DG, DU, WS, Y = (i << 32 for i in range(1, 13))


@pytest.fixture(scope="module", autouse=True)
def L():
    return afx.lib()


def coded(rows, cols):
    w = synth.generate(synth.TensorSpec("w", (rows, cols), "normal", rows + cols))
    return afx.afx_query(oracle.encode(w, (rows, cols)))


@pytest.fixture(scope="module")
def infos():
    return coded(40, 64), coded(40, 64)


def status(call, *args):
    with pytest.raises(afx.AfxError) as e:
        call(*args)
    return e.value.status


# ---------------------------------------------------------------------------
# gated block
# ---------------------------------------------------------------------------
def forward(infos, rows=40, cols=64, act=0, gate=GATE, up=UP, m=3, x=X, xs=64, h=H, hs=40, g=G, u=U, gus=40, ws=WS,
            nws=64 * MB):
    w = afx.gated_weights(infos[0], gate, infos[1], up, rows, cols, act)
    return status(afx.afx_restore_gated_async, w, m, x, xs, h, hs, g, u, gus, ws, nws)


def backward(infos, rows=40, cols=64, act=0, m=3, dh=DH, dhs=40, g=G, u=U, gus=40, dx=DX, dxs=64, dg=DG, du=DU, ws=WS,
             nws=64 * MB):
    w = afx.gated_weights(infos[0], GATE, infos[1], UP, rows, cols, act)
    return status(afx.afx_restore_gated_backward_async, w, m, dh, dhs, g, u, gus, dx, dxs, dg, du, ws, nws)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=41), afx.AFX_E_INVALID_ARG),          # rows * cols != n_elems
    (dict(rows=20, cols=128), afx.AFX_E_INVALID_ARG),  # x_stride below the row
    (dict(rows=0, cols=64), afx.AFX_E_INVALID_ARG),
    (dict(rows=640, cols=4, xs=8), afx.AFX_E_UNSUPPORTED),  # cols not a multiple of 8
    (dict(act=3), afx.AFX_E_INVALID_ARG),
    (dict(gate=0), afx.AFX_E_INVALID_ARG),
    (dict(gate=GATE + 8), afx.AFX_E_MISALIGNED),
    (dict(up=UP + 8), afx.AFX_E_MISALIGNED),
    (dict(x=0), afx.AFX_E_INVALID_ARG),
    (dict(x=X + 2), afx.AFX_E_MISALIGNED),
    (dict(xs=68), afx.AFX_E_UNSUPPORTED),            # rows of x not 16-byte aligned
    (dict(xs=1 << 22), afx.AFX_E_UNSUPPORTED),
    (dict(h=0), afx.AFX_E_INVALID_ARG),
    (dict(h=H + 1), afx.AFX_E_MISALIGNED),
    (dict(hs=39), afx.AFX_E_INVALID_ARG),
    (dict(u=0), afx.AFX_E_INVALID_ARG),              # one of g, u
    (dict(g=0), afx.AFX_E_INVALID_ARG),
    (dict(gus=39), afx.AFX_E_INVALID_ARG),
    (dict(m=(1 << 23) + 1), afx.AFX_E_UNSUPPORTED),
    (dict(h=X), afx.AFX_E_INVALID_ARG),              # outputs over inputs
    (dict(h=GATE + 256), afx.AFX_E_INVALID_ARG),
    (dict(g=H), afx.AFX_E_INVALID_ARG),              # outputs over outputs
    (dict(u=G + 2 * 40), afx.AFX_E_INVALID_ARG),
])
def test_gated_forward_refusals(infos, kw, want):
    assert forward(infos, **kw) == want


def test_gated_workspace_is_required_in_full(infos):
    for m in (300, 3000):
        need = afx.afx_restore_gated_workspace(40, 64, m)
        if need:
            assert forward(infos, m=m, nws=need - 1) == afx.AFX_E_BUFFER_TOO_SMALL
            assert forward(infos, m=m, ws=0) == afx.AFX_E_INVALID_ARG
            assert forward(infos, m=m, ws=WS + 8) == afx.AFX_E_MISALIGNED
            assert forward(infos, m=m, ws=X) == afx.AFX_E_INVALID_ARG
    need = afx.afx_restore_gated_workspace(40, 64, 3, backward=True)
    assert need > 0
    assert backward(infos, nws=need - 1) == afx.AFX_E_BUFFER_TOO_SMALL
    assert backward(infos, ws=0) == afx.AFX_E_INVALID_ARG
    assert afx.afx_restore_gated_workspace(40, 64, 0, backward=True) == 0
    for bad in ((0, 64, 1), (40, 0, 1)):
        assert status(afx.afx_restore_gated_workspace, *bad) == afx.AFX_E_INVALID_ARG
    for bad in ((40, 60, 1), (1 << 21, 64, 1), (40, 1 << 22, 1), (40, 64, (1 << 23) + 1)):
        assert status(afx.afx_restore_gated_workspace, *bad) == afx.AFX_E_UNSUPPORTED


@pytest.mark.parametrize("kw,want", [
    (dict(rows=41), afx.AFX_E_INVALID_ARG),
    (dict(act=7), afx.AFX_E_INVALID_ARG),
    (dict(dh=0), afx.AFX_E_INVALID_ARG),
    (dict(dh=DH + 2), afx.AFX_E_MISALIGNED),
    (dict(dhs=39), afx.AFX_E_INVALID_ARG),
    (dict(g=0), afx.AFX_E_INVALID_ARG),
    (dict(u=0), afx.AFX_E_INVALID_ARG),
    (dict(gus=39), afx.AFX_E_INVALID_ARG),
    (dict(dx=0), afx.AFX_E_INVALID_ARG),
    (dict(dx=DX + 1), afx.AFX_E_MISALIGNED),
    (dict(dxs=63), afx.AFX_E_INVALID_ARG),
    (dict(du=0), afx.AFX_E_INVALID_ARG),             # one of dg, du
    (dict(dg=U), afx.AFX_E_INVALID_ARG),             # in place of the other one
    (dict(dg=G + 80), afx.AFX_E_INVALID_ARG),        # over g, but not in place
    (dict(dx=G), afx.AFX_E_INVALID_ARG),
    (dict(dx=DH), afx.AFX_E_INVALID_ARG),
    (dict(du=DG), afx.AFX_E_INVALID_ARG),
    (dict(ws=U), afx.AFX_E_INVALID_ARG),
    (dict(dxs=1 << 22), afx.AFX_E_UNSUPPORTED),
])
def test_gated_backward_refusals(infos, kw, want):
    assert backward(infos, **kw) == want


def test_no_tokens_is_nothing_to_do(infos):
    w = afx.gated_weights(infos[0], GATE, infos[1], UP, 40, 64)
    afx.afx_restore_gated_async(w, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    afx.afx_restore_gated_backward_async(w, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    afx.afx_restore_gemm_t_async(infos[0], GATE, 40, 64, 0, 0, 0, False, 0, 0)
    p = afx.block_norm(64, 1e-6, w_pre=X)
    afx.afx_block_norm_async(p, 0, 0, 0, 0, 0, 0, 0, H, 64)


def test_counts_beyond_32_bits_are_refused_by_the_binding(infos):
    with pytest.raises(ValueError):
        afx.afx_restore_gemm_t_async(infos[0], GATE, 40, 64, X, 1 << 32, Y, False, WS, 64 * MB)
    with pytest.raises(ValueError):
        afx.afx_restore_gated_workspace(40, 64, -1)


# ---------------------------------------------------------------------------
# transposed product
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kw,want", [
    (dict(rows=41), afx.AFX_E_INVALID_ARG),
    (dict(rows=20, cols=128), afx.AFX_E_UNSUPPORTED),  # rows not a multiple of 8
    (dict(d=0), afx.AFX_E_INVALID_ARG),
    (dict(d=X + 2), afx.AFX_E_MISALIGNED),
    (dict(y=0), afx.AFX_E_INVALID_ARG),
    (dict(y=Y + 2), afx.AFX_E_MISALIGNED),
    (dict(y=X), afx.AFX_E_INVALID_ARG),
    (dict(y=GATE), afx.AFX_E_INVALID_ARG),
    (dict(ws=0), afx.AFX_E_INVALID_ARG),
    (dict(ws=X), afx.AFX_E_INVALID_ARG),
    (dict(ws=Y), afx.AFX_E_INVALID_ARG),
    (dict(nws=255), afx.AFX_E_BUFFER_TOO_SMALL),
    (dict(m=(1 << 23) + 1), afx.AFX_E_UNSUPPORTED),
])
def test_gemm_t_refusals(infos, kw, want):
    a = dict(rows=40, cols=64, d=X, m=3, y=Y, ws=WS, nws=64 * MB)
    a.update(kw)
    assert status(afx.afx_restore_gemm_t_async, infos[0], GATE, a["rows"], a["cols"], a["d"], a["m"], a["y"], False,
                  a["ws"], a["nws"]) == want


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------
B, R, RO, XN, WPOST, WGATE, WPRE, DXN, DRO, DR, DB, DW1 = (i << 32 for i in range(1, 13))
D = 48


def norm_params(**kw):
    a = dict(d=D, eps=1e-6, scale=0.5, r_type=afx.TYPE_BF16, w_post=WPOST, gate=WGATE, gate_stride=0, w_pre=WPRE)
    a.update(kw)
    return afx.block_norm(**a)


BAD_PARAMS = [
    (dict(d=0), afx.AFX_E_INVALID_ARG),
    (dict(d=afx.MAX_NORM_WIDTH + 1), afx.AFX_E_UNSUPPORTED),
    (dict(eps=0.0), afx.AFX_E_INVALID_ARG),
    (dict(eps=-1.0), afx.AFX_E_INVALID_ARG),
    (dict(eps=float("nan")), afx.AFX_E_INVALID_ARG),
    (dict(eps=float("inf")), afx.AFX_E_INVALID_ARG),
    (dict(scale=float("inf")), afx.AFX_E_INVALID_ARG),
    (dict(r_type=2), afx.AFX_E_INVALID_ARG),
    (dict(w_post=WPOST + 1), afx.AFX_E_MISALIGNED),
    (dict(gate_stride=D - 1), afx.AFX_E_INVALID_ARG),
]


@pytest.mark.parametrize("kw,want", BAD_PARAMS)
def test_norm_parameter_refusals(kw, want):
    p = norm_params(**kw)
    s = 40000  # a stride that no width refuses
    assert status(afx.afx_block_norm_async, p, 3, B, s, R, s, RO, s, XN, s) == want
    assert status(afx.afx_block_norm_workspace, p, 3) == want
    assert status(afx.afx_block_norm_backward_async, p, 3, B, s, RO, s, DXN, s, DRO, s, DR, s, DB, s, DW1, 0, 0,
                  WS + (1 << 40), MB) == want


@pytest.mark.parametrize("kw,want", [
    (dict(b_stride=D - 1), afx.AFX_E_INVALID_ARG),
    (dict(r=0), afx.AFX_E_INVALID_ARG),
    (dict(r_stride=D - 1), afx.AFX_E_INVALID_ARG),
    (dict(ro=0), afx.AFX_E_INVALID_ARG),             # b needs somewhere to write r'
    (dict(xn=0), afx.AFX_E_INVALID_ARG),             # w_pre without xn
    (dict(b=0, ro=0, xn=0), afx.AFX_E_INVALID_ARG),
    (dict(ro=R, ro_stride=D + 8), afx.AFX_E_INVALID_ARG),  # in place only with the same stride
    (dict(ro=R + 2 * D), afx.AFX_E_INVALID_ARG),
    (dict(xn=R), afx.AFX_E_INVALID_ARG),
    (dict(xn=RO), afx.AFX_E_INVALID_ARG),
    (dict(xn=WPRE), afx.AFX_E_INVALID_ARG),
    (dict(b=B + 2), afx.AFX_E_MISALIGNED),
    (dict(r=R + 1), afx.AFX_E_MISALIGNED),
    (dict(b_stride=1 << 28), afx.AFX_E_UNSUPPORTED),
])
def test_norm_forward_refusals(kw, want):
    a = dict(b=B, b_stride=D, r=R, r_stride=D, ro=RO, ro_stride=D, xn=XN, xn_stride=D)
    a.update(kw)
    assert status(afx.afx_block_norm_async, norm_params(), 3, *a.values()) == want


@pytest.mark.parametrize("params,kw,want", [
    ({}, dict(ro=0), afx.AFX_E_INVALID_ARG),
    ({}, dict(dxn_stride=D - 1), afx.AFX_E_INVALID_ARG),
    ({}, dict(dr=0, db=0, dw_pre=0, dw_post=0, dgate=0), afx.AFX_E_INVALID_ARG),  # nothing to write
    (dict(w_pre=0), {}, afx.AFX_E_INVALID_ARG),      # dxn without w_pre
    (dict(w_post=0), {}, afx.AFX_E_INVALID_ARG),     # dw_post without w_post
    (dict(gate=0), {}, afx.AFX_E_INVALID_ARG),       # dgate without a gate
    ({}, dict(b=0), afx.AFX_E_INVALID_ARG),          # db without b
    ({}, dict(dr=DRO, dr_stride=D + 8), afx.AFX_E_INVALID_ARG),
    ({}, dict(db=B), afx.AFX_E_INVALID_ARG),
    ({}, dict(dw_pre=DR), afx.AFX_E_INVALID_ARG),
    ({}, dict(dw_post=DW1), afx.AFX_E_INVALID_ARG),  # the same buffer twice
    ({}, dict(dgate=(14 << 32) + 2), afx.AFX_E_MISALIGNED),
    ({}, dict(ws=0), afx.AFX_E_INVALID_ARG),
    ({}, dict(ws=(15 << 32) + 8), afx.AFX_E_MISALIGNED),
    ({}, dict(ws=B), afx.AFX_E_INVALID_ARG),
    ({}, dict(nws=3), afx.AFX_E_BUFFER_TOO_SMALL),
])
def test_norm_backward_refusals(params, kw, want):
    a = dict(b=B, b_stride=D, ro=RO, ro_stride=D, dxn=DXN, dxn_stride=D, dro=DRO, dro_stride=D, dr=DR, dr_stride=D,
             db=DB, db_stride=D, dw_pre=DW1, dw_post=13 << 32, dgate=14 << 32, ws=15 << 32, nws=MB)
    a.update(kw)
    assert status(afx.afx_block_norm_backward_async, norm_params(**params), 3, *a.values()) == want


def test_null_structures_are_refused(L):
    n = ctypes.c_size_t()
    assert L.afx_restore_gated_async(None, 1, X, 64, H, 40, None, None, 0, WS, MB, None) == afx.AFX_E_INVALID_ARG
    assert L.afx_restore_gated_workspace(40, 64, 1, 0, None) == afx.AFX_E_INVALID_ARG
    assert L.afx_restore_gemm_t_workspace(40, 64, 1, None) == afx.AFX_E_INVALID_ARG
    assert L.afx_restore_gemm_t_async(None, GATE, 40, 64, X, 1, Y, 0, WS, MB, None) == afx.AFX_E_INVALID_ARG
    assert L.afx_block_norm_workspace(None, 1, ctypes.byref(n)) == afx.AFX_E_INVALID_ARG
    assert L.afx_block_norm_async(None, 1, B, D, R, D, RO, D, XN, D, None) == afx.AFX_E_INVALID_ARG
    w = afx.afx_gated()
    assert L.afx_restore_gated_async(ctypes.byref(w), 1, X, 64, H, 40, None, None, 0, WS, MB, None) == \
        afx.AFX_E_INVALID_ARG
