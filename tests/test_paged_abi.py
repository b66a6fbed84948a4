"""Refusals of the calls on a paged cache, on the CPU: each is decided before
any HIP call, so that made-up addresses are never reached."""
import math

import pytest

from lossless_bf16_weight_afx_amd import afx

INVALID, SMALL, MISALIGNED, UNSUPPORTED = -1, -5, -6, -8
MB = 1 << 20


def at(i):
    """Address of made-up buffer i, far from the others."""
    return (i + 1) << 36


def refused(status, call, *args):
    with pytest.raises(afx.AfxError) as e:
        call(*args)
    assert e.value.status == status, e.value


def kv(**new):
    a = dict(k_dev=at(0), v_dev=at(1), n_pages=64, page_tokens=16, kv_heads=2, head_dim=64)
    a.update(new)
    return afx.kv_pages(**a)


def heads(**new):
    a = dict(q_heads=4, kv_heads=2, head_dim=64, rot_dim=64, pairing=afx.ROPE_HALVES, n_axes=1, eps=1e-6, w_q=at(20),
             w_k=at(21), freq=at(22), axis=0)
    a.update(new)
    return afx.heads(**a)


def table(**new):
    a = dict(table_dev=at(30), table_stride=8, len_dev=at(31), refs_dev=at(32), n_seqs=5, max_pages=8, n_pages=64,
             page_tokens=16)
    a.update(new)
    return afx.page_table(**a)


def data(**new):
    a = dict(data_dev=at(40), page_bytes=4096, plane_stride=64 * 4096, n_planes=3)
    a.update(new)
    return afx.page_data(**a)


NONE = object()


def call_heads(p=None, m=3, kvp=NONE, **new):
    a = dict(pos=at(2), pos_stride=3, q=at(3), qs=256, k=at(4), ks=128, v=at(5), vs=128, qo=at(6), qos=256, ko=0, kos=0,
             slots=at(7))
    a.update(new)
    afx.afx_heads_async(p or heads(), m, a["pos"], a["pos_stride"], a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"],
                        a["qo"], a["qos"], a["ko"], a["kos"], kv() if kvp is NONE else kvp, a["slots"])


def call_grad(p=None, m=3, **new):
    a = dict(pos=at(2), pos_stride=3, q=at(3), qs=256, k=at(4), ks=128, dq=at(5), dqs=256, dk=at(6), dks=128, qi=at(7),
             qis=256, ki=at(8), kis=128, wq=at(9), wk=at(10), ws=at(11), n=MB)
    a.update(new)
    afx.afx_heads_backward_async(p or heads(), m, a["pos"], a["pos_stride"], a["q"], a["qs"], a["k"], a["ks"], a["dq"],
                                 a["dqs"], a["dk"], a["dks"], a["qi"], a["qis"], a["ki"], a["kis"], a["wq"], a["wk"],
                                 a["ws"], a["n"])


def call_attend(p=None, kvp=None, t=None, rows=5, m=3, **new):
    a = dict(seqs=0, starts=at(2), q=at(3), qs=256, out=at(4), outs=256, lse=at(5), ws=at(6), n=64 * MB)
    a.update(new)
    afx.afx_attend_async(p or afx.attend(4, 0.125, True, 0, 1, 100), kvp or kv(), t or table(), rows, a["seqs"],
                         a["starts"], m, a["q"], a["qs"], a["out"], a["outs"], a["lse"], a["ws"], a["n"])


@pytest.mark.parametrize("status, new", [
    (INVALID, dict(q_heads=0)), (INVALID, dict(kv_heads=0)), (INVALID, dict(q_heads=1025)), (INVALID, dict(head_dim=0)),
    (UNSUPPORTED, dict(head_dim=60, rot_dim=0)), (UNSUPPORTED, dict(head_dim=264, rot_dim=0)),
    (INVALID, dict(rot_dim=66)), (INVALID, dict(rot_dim=31)), (INVALID, dict(pairing=2)), (INVALID, dict(n_axes=0)),
    (INVALID, dict(n_axes=5)), (INVALID, dict(freq=0)), (INVALID, dict(eps=0.0)), (INVALID, dict(eps=math.nan)),
    (INVALID, dict(eps=math.inf)), (MISALIGNED, dict(w_q=at(20) + 1)), (MISALIGNED, dict(freq=at(22) + 2)),
])
def test_head_parameters(status, new):
    p = heads(**new)
    refused(status, call_heads, p)
    refused(status, call_grad, p)
    refused(status, afx.afx_heads_workspace, p, 3)


@pytest.mark.parametrize("status, new", [
    (INVALID, dict(q=0, k=0, v=0)), (INVALID, dict(q=0)), (INVALID, dict(qo=0)), (INVALID, dict(slots=0)),
    (INVALID, dict(kvp=None)), (INVALID, dict(kvp=None, slots=0)), (INVALID, dict(pos=0)),
    (INVALID, dict(qs=255)), (INVALID, dict(ks=127)), (INVALID, dict(vs=120)), (INVALID, dict(qos=128)),
    (INVALID, dict(ko=at(8), kos=127)), (INVALID, dict(k=0, ko=at(8), kos=128)), (UNSUPPORTED, dict(qs=1 << 28)),
    (MISALIGNED, dict(q=at(3) + 2)), (MISALIGNED, dict(qo=at(6) + 1)), (MISALIGNED, dict(slots=at(7) + 2)),
    (MISALIGNED, dict(pos=at(2) + 1)), (UNSUPPORTED, dict(m=(1 << 23) + 1)),
    (INVALID, dict(p=heads(n_axes=2), pos_stride=2)),
    (INVALID, dict(kvp=kv(kv_heads=4))), (INVALID, dict(kvp=kv(head_dim=128))), (INVALID, dict(kvp=kv(n_pages=0))),
    (UNSUPPORTED, dict(kvp=kv(page_tokens=8))), (UNSUPPORTED, dict(kvp=kv(page_tokens=24))),
    (UNSUPPORTED, dict(kvp=kv(page_tokens=512))), (UNSUPPORTED, dict(kvp=kv(n_pages=1 << 27))),
    (MISALIGNED, dict(kvp=kv(k_dev=at(0) + 8))), (INVALID, dict(kvp=kv(v_dev=0))),
    # outputs on inputs, and on each other
    (INVALID, dict(qo=at(3))), (INVALID, dict(kvp=kv(k_dev=at(3)))), (INVALID, dict(kvp=kv(v_dev=at(0)))),
    (INVALID, dict(ko=at(6) + 512 * 2, kos=128)), (INVALID, dict(kvp=kv(k_dev=at(7)))), (INVALID, dict(qo=at(22))),
    (INVALID, dict(kvp=kv(v_dev=at(2) & ~15))),
])
def test_heads_arguments(status, new):
    refused(status, lambda: call_heads(**new))


def test_heads_of_no_tokens():
    call_heads(m=0, q=0, k=0, v=0, qo=0, slots=0, kvp=None)  # does nothing


@pytest.mark.parametrize("status, new", [
    (INVALID, dict(dq=0)), (INVALID, dict(q=0)), (INVALID, dict(k=0)), (INVALID, dict(dk=0)), (INVALID, dict(pos=0)),
    (INVALID, dict(qi=0, ki=0, wq=0, wk=0)), (INVALID, dict(p=heads(w_q=0))), (INVALID, dict(p=heads(w_k=0))),
    (INVALID, dict(ws=0)), (SMALL, dict(n=4 * 64 * 2 - 1)), (MISALIGNED, dict(ws=at(11) + 8)),
    (MISALIGNED, dict(wq=at(9) + 2)), (INVALID, dict(qis=255)), (INVALID, dict(dks=127)),
    (INVALID, dict(qi=at(3))), (INVALID, dict(qi=at(5), qis=512)), (INVALID, dict(qi=at(5) + 2)),
    (INVALID, dict(ki=at(5))), (INVALID, dict(wq=at(10))), (INVALID, dict(wk=at(11))), (INVALID, dict(wk=at(8))),
    (UNSUPPORTED, dict(m=(1 << 23) + 1)),
])
def test_heads_backward_arguments(status, new):
    refused(status, lambda: call_grad(**new))


@pytest.mark.parametrize("status, new", [
    (INVALID, dict(p=afx.attend(3, 1.0))), (INVALID, dict(p=afx.attend(0, 1.0))),
    (INVALID, dict(p=afx.attend(4, math.nan))), (INVALID, dict(p=afx.attend(4, math.inf))),
    (INVALID, dict(p=afx.attend(2 * 257, 1.0))), (INVALID, dict(kvp=kv(n_pages=63))),
    (INVALID, dict(kvp=kv(page_tokens=32, n_pages=64))), (INVALID, dict(starts=0)), (INVALID, dict(q=0)),
    (INVALID, dict(out=0)), (INVALID, dict(qs=248)), (INVALID, dict(outs=248)), (MISALIGNED, dict(qs=260)),
    (MISALIGNED, dict(outs=257)), (MISALIGNED, dict(q=at(3) + 8)), (MISALIGNED, dict(lse=at(5) + 2)),
    (UNSUPPORTED, dict(qs=1 << 28)), (UNSUPPORTED, dict(m=(1 << 23) + 1)), (UNSUPPORTED, dict(rows=(1 << 16) + 1)),
    (INVALID, dict(rows=6)),  # the sixth sequence of five
    (INVALID, dict(out=at(3))), (INVALID, dict(out=at(0))), (INVALID, dict(lse=at(4))), (INVALID, dict(lse=at(31))),
    (INVALID, dict(t=table(table_dev=0))), (INVALID, dict(t=table(len_dev=0))), (INVALID, dict(t=table(n_seqs=0))),
    (INVALID, dict(t=table(table_stride=7))), (UNSUPPORTED, dict(t=table(max_pages=1 << 27, table_stride=1 << 27))),
    (UNSUPPORTED, dict(t=table(n_seqs=(1 << 20) + 1))), (MISALIGNED, dict(t=table(len_dev=at(31) + 1))),
])
def test_attend_arguments(status, new):
    refused(status, lambda: call_attend(**new))


def test_attend_of_no_tokens():
    call_attend(m=0, starts=0, q=0, out=0)
    call_attend(rows=0, starts=0, q=0, out=0)
    call_attend(m=0, t=table(refs_dev=0))  # (it does not read the counts)


def pages_calls(t, d):
    yield lambda: afx.afx_pages_fork_async(t, 2, at(2), at(3), at(4))
    yield lambda: afx.afx_pages_trim_async(t, 2, at(2), at(3))
    yield lambda: afx.afx_pages_extend_async(t, d, 2, at(2), at(3), 4, at(4), at(5), at(6), at(7), MB)
    yield lambda: afx.afx_pages_compact_async(t, d, at(2), at(3), at(4), MB)


@pytest.mark.parametrize("status, new", [
    (INVALID, dict(table_dev=0)), (INVALID, dict(len_dev=0)), (INVALID, dict(refs_dev=0)), (INVALID, dict(n_seqs=0)),
    (INVALID, dict(max_pages=0)), (INVALID, dict(n_pages=0)), (INVALID, dict(table_stride=7)),
    (UNSUPPORTED, dict(page_tokens=17)), (UNSUPPORTED, dict(page_tokens=8)), (UNSUPPORTED, dict(page_tokens=512)),
    (UNSUPPORTED, dict(n_seqs=(1 << 20) + 1)), (UNSUPPORTED, dict(n_pages=1 << 27)),
    (UNSUPPORTED, dict(max_pages=1 << 27, table_stride=1 << 27)), (UNSUPPORTED, dict(table_stride=1 << 28)),
    (MISALIGNED, dict(refs_dev=at(32) + 2)),
])
def test_page_tables(status, new):
    for call in pages_calls(table(**new), data(plane_stride=1 << 45)):
        refused(status, call)


@pytest.mark.parametrize("new", [dict(len_dev=at(30)), dict(refs_dev=at(31)), dict(refs_dev=at(30)),
                                 dict(refs_dev=at(2)), dict(len_dev=at(3)), dict(table_dev=at(3))])
def test_page_tables_on_other_buffers(new):
    for call in pages_calls(table(**new), data()):
        refused(INVALID, call)


@pytest.mark.parametrize("status, new", [
    (INVALID, dict(data_dev=0)), (INVALID, dict(page_bytes=0)), (INVALID, dict(n_planes=0)),
    (UNSUPPORTED, dict(page_bytes=4104)), (UNSUPPORTED, dict(n_planes=65536)),
    (UNSUPPORTED, dict(page_bytes=(1 << 30) + 16)), (INVALID, dict(plane_stride=64 * 4096 - 16)),
    (UNSUPPORTED, dict(plane_stride=64 * 4096 + 8)), (MISALIGNED, dict(data_dev=at(40) + 8)),
    (INVALID, dict(data_dev=at(2))), (INVALID, dict(data_dev=at(3))),
])
def test_page_data(status, new):
    t, d = table(), data(**new)
    for call in list(pages_calls(t, d))[2:]:
        refused(status, call)
    refused(status, afx.afx_pages_copy_async, d, 64, 2, at(2), at(3))


def test_page_lists():
    t, d = table(), data()
    refused(UNSUPPORTED, afx.afx_pages_fork_async, t, 1025, at(2), at(3), 0)
    refused(UNSUPPORTED, afx.afx_pages_trim_async, t, 1025, at(2), 0)
    refused(UNSUPPORTED, afx.afx_pages_extend_workspace, t, 1025)
    refused(UNSUPPORTED, afx.afx_pages_extend_async, t, d, 1025, at(2), at(3), 4, at(4), 0, 0, at(7), MB)
    refused(UNSUPPORTED, afx.afx_pages_extend_async, t, d, 1, at(2), at(3), (1 << 23) + 1, at(4), 0, 0, at(7), MB)
    for src, dst, granted, status in ((0, at(3), 0, INVALID), (at(2), 0, 0, INVALID), (at(2) + 2, at(3), 0, MISALIGNED),
                                      (at(2), at(3), at(3), INVALID), (at(2), at(3), at(4) + 1, MISALIGNED)):
        refused(status, afx.afx_pages_fork_async, t, 2, src, dst, granted)
    refused(INVALID, afx.afx_pages_trim_async, t, 2, 0, 0)
    good = dict(seqs=at(2), starts=at(3), m=4, slots=at(4), pos=at(5), granted=at(6), ws=at(7), n=MB)
    for new, status in ((dict(seqs=0), INVALID), (dict(starts=0), INVALID), (dict(slots=0), INVALID),
                        (dict(ws=0), INVALID), (dict(n=2 * 16 + 64 * 4 - 1), SMALL), (dict(ws=at(7) + 8), MISALIGNED),
                        (dict(pos=at(4)), INVALID), (dict(granted=at(2)), INVALID), (dict(slots=at(3) - 4), INVALID)):
        a = {**good, **new}
        refused(status, afx.afx_pages_extend_async, t, d, 2, *a.values())
    refused(INVALID, afx.afx_pages_extend_async, t, d, 0, 0, 0, 4, at(4), 0, 0, 0, 0)  # tokens of no row
    refused(INVALID, afx.afx_pages_compact_async, t, d, 0, 0, at(4), MB)
    refused(INVALID, afx.afx_pages_compact_async, t, d, at(2), at(2), at(4), MB)
    refused(SMALL, afx.afx_pages_compact_async, t, d, at(2), 0, at(4), 4 * (2 + 2 * 64) - 1)
    refused(INVALID, afx.afx_pages_copy_async, d, 64, 2, 0, at(3))
    refused(INVALID, afx.afx_pages_copy_async, d, 0, 2, at(2), at(3))
    refused(MISALIGNED, afx.afx_pages_copy_async, d, 64, 2, at(2) + 1, at(3))


def test_page_calls_of_no_rows():
    t, d = table(), data()
    afx.afx_pages_fork_async(t, 0, 0, 0, 0)
    afx.afx_pages_trim_async(t, 0, 0, 0)
    afx.afx_pages_extend_async(t, d, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    afx.afx_pages_copy_async(d, 64, 0, 0, 0)


def test_counts_that_do_not_fit():
    for call in (lambda: kv(n_pages=1 << 32), lambda: heads(q_heads=-1), lambda: table(n_seqs=1 << 32),
                 lambda: data(n_planes=-1), lambda: afx.attend(4, 1.0, True, 1 << 32), lambda: call_heads(m=1 << 32),
                 lambda: call_attend(rows=-1), lambda: call_grad(m=-1)):
        with pytest.raises(ValueError):
            call()
