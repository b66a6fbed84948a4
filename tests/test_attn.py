"""attn.Attention's and cache.PagedCache's own part (buffers, checks, order and
arguments of calls) on the CPU: the library's calls that would run on the GPU
are recorded instead."""
import contextlib

import pytest

from lossless_bf16_weight_afx_amd import afx, attn, cache

torch = pytest.importorskip("torch")

CALLS = ("afx_pages_extend_async", "afx_pages_fork_async", "afx_pages_trim_async", "afx_pages_compact_async",
         "afx_block_norm_async", "afx_restore_gemm_batch_async", "afx_heads_async", "afx_attend_async",
         "afx_restore_gemm_async")


class Stream:
    cuda_stream = 0


@pytest.fixture
def calls(monkeypatch):
    """The library's calls, in order: name and arguments."""
    made = []
    for name in CALLS:
        monkeypatch.setattr(afx, name, lambda *a, name=name: made.append((name, a)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    monkeypatch.setattr(torch.cuda, "device", contextlib.nullcontext)
    return made


def refused(calls, f, *args, **kw):
    """ValueError, and nothing was called."""
    n = len(calls)
    with pytest.raises(ValueError):
        f(*args, **kw)
    assert len(calls) == n


def paged(**kw):
    how = dict(layers=2, kv_heads=2, head_dim=64, n_pages=20, page_tokens=16, max_seqs=6, max_pages=8, max_tokens=40,
               max_rows=5, device="cpu")
    how.update(kw)
    return cache.PagedCache(how.pop("layers"), how.pop("kv_heads"), how.pop("head_dim"), **how)


def info(rows, cols):
    i = afx.afx_info()
    i.n_elems, i.ndim = rows * cols, 2
    i.shape[0], i.shape[1] = rows, cols
    return i


def half(c, d=256, q_heads=4, layer=0, shapes=None, **kw):
    nq, nk = q_heads * c.head_dim, c.kv_heads * c.head_dim
    shapes = shapes or ((nq, d), (nk, d), (nk, d), (d, nq))
    blob = torch.zeros(16, dtype=torch.uint8)
    return attn.Attention(*((info(*s), blob) for s in shapes), d, c, layer, q_heads,
                          torch.ones(d, dtype=torch.bfloat16), **kw)


def ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_the_cache_describes_its_buffers(calls):
    c = paged()
    page = 2 * 2 * 64 * 16
    assert c.data.numel() * 2 == 4 * 20 * page
    assert (c.planes.page_bytes, c.planes.plane_stride, c.planes.n_planes) == (page, 20 * page, 4)
    for i in (0, 1):
        kv = c.layer(i)
        assert kv.k_dev == c.data.data_ptr() + 2 * i * 20 * page and kv.v_dev == kv.k_dev + 20 * page
        assert (kv.n_pages, kv.page_tokens, kv.kv_heads, kv.head_dim) == (20, 16, 2, 64)
    assert bool((c.table == -1).all()) and bool((c.len == 0).all()) and bool((c.refs == 0).all())
    assert (c.pages.n_seqs, c.pages.max_pages, c.pages.n_pages, c.pages.table_stride) == (6, 8, 20, 8)
    need = max([afx.afx_pages_extend_workspace(c.pages, n) for n in range(1, 6)]
               + [afx.afx_pages_compact_workspace(c.pages), 16])
    assert c.ws.numel() == need
    for i in (-1, 2):
        refused(calls, c.layer, i)


@pytest.mark.parametrize("kw", [dict(layers=0), dict(kv_heads=1025), dict(head_dim=4), dict(head_dim=264),
                                dict(page_tokens=8), dict(page_tokens=48), dict(n_pages=0), dict(max_seqs=0),
                                dict(max_pages=0), dict(max_tokens=0), dict(max_rows=1025), dict(layers=32768),
                                dict(max_pages=1 << 27), dict(max_seqs=(1 << 20) + 1)])
def test_caches_that_are_refused(calls, kw):
    refused(calls, paged, **kw)


def test_calls_of_the_cache(calls):
    c = paged()
    seqs, starts = ints(3, 1), ints(0, 2, 7)
    step = c.extend(seqs, starts, 7, 5)
    name, a = calls[-1]
    assert name == CALLS[0] and a[2:6] == (2, seqs.data_ptr(), starts.data_ptr(), 7)
    assert a[6:9] == (c.slots.data_ptr(), c.pos.data_ptr(), c.granted.data_ptr())
    assert (step.m, step.max_new, step.slots.numel(), step.pos.numel(), step.granted.numel()) == (7, 5, 7, 7, 2)
    assert c.extend(seqs, starts, 7).max_new == 7
    assert c.fork(seqs, ints(0, 2)).numel() == 2
    assert calls[-1][0] == CALLS[1]
    lens = ints(4, 0)
    c.trim(seqs, lens)
    assert calls[-1] == (CALLS[2], (c.pages, 2, seqs.data_ptr(), lens.data_ptr(), 0))
    c.free(seqs)
    assert calls[-1] == (CALLS[2], (c.pages, 2, seqs.data_ptr(), 0, 0))
    where, live = c.compact()
    assert calls[-1][0] == CALLS[3] and where.numel() == 20 and live.numel() == 1


def test_lists_that_are_refused(calls):
    c = paged()
    two, starts = ints(0, 1), ints(0, 1, 2)
    for bad in (two.long(), two.float(), two[None], ints(*range(6)), torch.zeros(4, dtype=torch.int32)[::2], ints()):
        refused(calls, c.extend, bad, torch.zeros(bad.numel() + 1, dtype=torch.int32), 2)
        refused(calls, c.free, bad)
        refused(calls, c.trim, two, bad if bad.numel() != 2 or bad.dtype != torch.int32 or bad.dim() != 1
                or not bad.is_contiguous() else ints(0))
        refused(calls, c.fork, two, bad if bad.numel() != 2 or bad.dtype != torch.int32 or bad.dim() != 1
                or not bad.is_contiguous() else ints(0))
    refused(calls, c.extend, two, two, 2)  # starts has one more
    for m, new in ((0, None), (41, None), (2, 3), (2, 0)):
        refused(calls, c.extend, two, starts, m, new)


def test_order_and_buffers_of_a_step(calls):
    c = paged()
    t = half(c, layer=1, w_next=torch.ones(256, dtype=torch.bfloat16), freq=torch.ones(16))
    r = torch.ones(7, 256, dtype=torch.bfloat16)
    step = c.extend(ints(3, 1), ints(0, 2, 7), 7, 5)
    r1, xn = t.forward(r, step)
    assert [n for n, _ in calls] == [CALLS[0], CALLS[4], CALLS[5], CALLS[6], CALLS[7], CALLS[8], CALLS[4]]
    assert r1.data_ptr() == t.r_out.data_ptr() and r1.shape == (7, 256) and xn.data_ptr() == t.xn_next.data_ptr()
    y = t.y.data_ptr()
    q, k, v, b = y, y + 4 * 7 * 256, y + 4 * 7 * 384, y + 4 * 7 * 512
    jobs = calls[2][1][0]
    assert [j[5] for j in jobs] == [q, k, v] and all(j[4] == t.xn.data_ptr() for j in jobs)
    a = calls[3][1]
    assert a[1:10] == (7, step.pos.data_ptr(), 7, q, 256, k, 128, v, 128) and a[15] == step.slots.data_ptr()
    assert a[14].k_dev == c.layer(1).k_dev and t.heads.rot_dim == 32
    a = calls[4][1]
    assert a[3:9] == (2, step.seqs.data_ptr(), step.starts.data_ptr(), 7, t.qn.data_ptr(), 256)
    assert (a[0].max_new, a[0].max_len, a[0].causal) == (5, 128, 1) and abs(a[0].scale - 0.125) < 1e-7
    assert calls[5][1][4:7] == (t.a.data_ptr(), 7, b)
    assert bool((t.y[:7 * (256 + 256 + 256)] == 0).all())
    t.forward(t.r_out[:7], c.extend(ints(3, 1), ints(0, 2, 7), 7))  # r' of the last pass


def test_steps_that_are_refused(calls):
    c, other = paged(), paged()
    t = half(c)
    r = torch.ones(7, 256, dtype=torch.bfloat16)
    seqs, starts = ints(3, 1), ints(0, 2, 7)
    refused(calls, t.forward, r, other.extend(seqs, starts, 7))
    step = c.extend(seqs, starts, 7)
    for bad in (r[:6], r.float(), r[0], torch.ones(7, 512, dtype=torch.bfloat16), r.t(), t.xn[:7], t.qn[:7, :256],
                t.ws.new_zeros(7 * 512).view(torch.bfloat16).view(7, 256)[:, :128],
                c.data[0, :7 * 256].view(7, 256)):
        refused(calls, t.forward, bad, step)
    for pos in (ints(*range(7)), ints(*range(7))[None].long(), ints(*range(6))[None], ints(*range(14)).view(2, 7)):
        refused(calls, t.forward, r, step, pos)
    t.forward(r, step, ints(*range(7))[None])
    t.forward(r, step)  # a second layer's, or the same again
    c.free(seqs)
    refused(calls, t.forward, r, step)  # the cache has moved on
    axes = half(c, freq=torch.ones(16), axis=torch.zeros(16, dtype=torch.uint8), n_axes=3)
    step = c.extend(seqs, starts, 7)
    refused(calls, axes.forward, r, step)
    axes.forward(r, step, torch.zeros(3, 7, dtype=torch.int32))
    small = half(c, max_tokens=6)
    refused(calls, small.forward, r, step)


@pytest.mark.parametrize("kw", [dict(d=128), dict(d=320), dict(q_heads=3), dict(q_heads=2), dict(layer=2), dict(window=-1),
                                dict(max_tokens=41), dict(max_tokens=0), dict(n_axes=5), dict(n_axes=0), dict(pairing=2),
                                dict(freq=torch.ones(33)), dict(freq=torch.ones(4).double()),
                                dict(axis=torch.zeros(4, dtype=torch.uint8)),
                                dict(freq=torch.ones(4), axis=torch.zeros(3, dtype=torch.uint8)),
                                dict(w_q=torch.ones(63, dtype=torch.bfloat16)), dict(w_k=torch.ones(64)),
                                dict(w_next=torch.ones(128, dtype=torch.bfloat16)),
                                dict(shapes=((256, 256), (128, 256), (256, 128), (256, 256))),
                                dict(shapes=((256, 256), (128, 256), (128, 256), (256, 512)))])
def test_halves_that_are_refused(calls, kw):
    refused(calls, half, paged(), **kw)


def test_a_step_of_any_size_has_its_workspace(calls, monkeypatch):
    """Sizes that the workspace was not made for are taken in one part, which needs none."""
    c = paged(max_seqs=40, max_rows=40, max_tokens=300, n_pages=2000, max_pages=512)
    t = half(c)
    usual = 0
    for n in (1, 2, 3, 17, 40):
        for m in (n, n + 1, 4 * n, 299):
            for new in {1, 2, 3, 8, m}:
                if n > m or new > m or n * new < m:
                    continue
                starts = torch.linspace(0, m, n + 1).int()
                t.forward(torch.ones(m, 256, dtype=torch.bfloat16),
                          c.extend(torch.arange(n, dtype=torch.int32), starts, m, new))
                p = calls[-3][1][0]
                assert afx.afx_attend_workspace(p, t.kv, n, m) <= t.ws.numel() and p.max_new == new
                usual += p.max_len == 512 * 16
    assert usual > 20
    monkeypatch.setattr(t, "ws", t.ws[:16])
    t.forward(torch.ones(1, 256, dtype=torch.bfloat16), c.extend(ints(0), ints(0, 1), 1))
    p = calls[-3][1][0]
    assert p.max_len == 1 and afx.afx_attend_workspace(p, t.kv, 1, 1) == 0
