"""ffn.FeedForward's own part (buffers, checks, order of calls) on the CPU:
the library's calls that would run on the GPU are recorded instead."""
import contextlib

import pytest

from lossless_bf16_weight_afx_amd import afx, ffn

torch = pytest.importorskip("torch")


def info(rows, cols):
    i = afx.afx_info()
    i.n_elems, i.ndim = rows * cols, 2
    i.shape[0], i.shape[1] = rows, cols
    return i


def matrices(d, ff):
    blob = torch.zeros(16, dtype=torch.uint8)
    return [(info(ff, d), blob), (info(ff, d), blob), (info(d, ff), blob)]


def block(d, ff, max_tokens, training=False, **kw):
    return ffn.FeedForward(*matrices(d, ff), d, ff, torch.ones(d, dtype=torch.bfloat16), max_tokens=max_tokens,
                           training=training, **kw)


@pytest.mark.parametrize("training", [False, True])
@pytest.mark.parametrize("d,ff,max_tokens", [(768, 1024, 641), (768, 14336, 700), (1024, 1536, 321), (2048, 768, 500),
                                             (1024, 2816, 1024), (256, 512, 700), (64, 256, 3), (128, 8192, 70),
                                             (5120, 17408, 450), (320, 2560, 1300)])
def test_workspace_holds_every_token_count(d, ff, max_tokens, training):
    t = block(d, ff, max_tokens, training)
    need = 0
    for m in range(1, max_tokens + 1):
        need = max(need, afx.afx_restore_gated_workspace(ff, d, m))
        if training:
            need = max(need, afx.afx_restore_gated_workspace(ff, d, m, True),
                       afx.afx_restore_gemm_t_workspace(d, ff, m), afx.afx_block_norm_workspace(t.norm_in, m),
                       afx.afx_block_norm_workspace(t.norm_out, m))
    assert t.ws.numel() == max(need, 16)


# ---------------------------------------------------------------------------
# what the buffers hold between forward() and backward()
# ---------------------------------------------------------------------------
CALLS = ("afx_block_norm_async", "afx_restore_gated_async", "afx_restore_gemm_async", "afx_block_norm_backward_async",
         "afx_restore_gemm_t_async", "afx_restore_gated_backward_async")


class Stream:
    cuda_stream = 0


@pytest.fixture
def calls(monkeypatch):
    """The names of the library's calls, in order; `capturing` as a graph's capture would have it."""
    made = []
    for name in CALLS:
        monkeypatch.setattr(afx, name, lambda *a, name=name: made.append(name))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "device", contextlib.nullcontext)
    return made


def values(m, d=64):
    return torch.ones(m, d, dtype=torch.bfloat16)


def refused(calls, f, *args):
    """ValueError, and nothing was called."""
    n = len(calls)
    with pytest.raises(ValueError):
        f(*args)
    assert len(calls) == n


def test_backward_takes_the_kept_values_once(calls):
    """dg and du take the places of g and u: a second backward() would take
    them for g and u."""
    t, r = block(64, 256, 8, True), values(8)
    refused(calls, t.backward, r, r)  # no forward pass yet
    t.forward(r)
    t.backward(r, r)
    refused(calls, t.backward, r, r)
    t.forward(r)
    refused(calls, t.backward, r, values(7))  # refused arguments leave the kept values
    t.backward(r, r)
    assert calls == (list(CALLS[:3]) + [CALLS[0]] + list(CALLS[3:]) + [CALLS[3]]) * 2


def test_backward_is_of_the_last_forward_pass(calls):
    t, r, wide = block(64, 256, 8, True), values(8), torch.ones(8, 128, dtype=torch.bfloat16)
    t.forward(r)
    for other in (values(8), r[:5], r[1:], wide[:, :64]):
        refused(calls, t.backward, other, values(other.shape[0]))
    t.backward(r[:], values(8))  # a view of the same rows
    t.forward(wide[:, 64:])
    refused(calls, t.backward, wide[:, :64], r)
    t.forward(r[2:3])
    refused(calls, t.backward, r[:1], r[:1])
    t.backward(r[2:3], r[:1])


def test_training_does_not_overwrite_the_stream(calls):
    """backward() reads r once more: it may not lie in the object's own buffers."""
    w = torch.ones(64, dtype=torch.bfloat16)
    t, r = block(64, 256, 8, True, w_next=w), values(8)
    t.forward(r)
    for own in (t.r_out, t.r_out[2:5], t.xn, t.xn_next, t.h[:, :64], t.g[:, 64:128], t.u[:3, :64], t.db, t.dxn, t.dr):
        refused(calls, t.forward, own)
    t.backward(r, r)  # what the last forward pass kept is still there
    other = block(64, 256, 8)
    ro, _ = other.forward(r)
    other.forward(ro)  # without training, in place
    t.forward(ro)  # another object's output
    t.backward(ro, t.dr)


def test_a_captured_forward_pass_may_be_replayed_between_backward_calls(calls, monkeypatch):
    """Replays are not seen here, so what they keep is taken to be there;
    not so after a graph of both passes."""
    t, r = block(64, 256, 8, True), values(8)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    t.forward(r)
    t.backward(r, r)
    refused(calls, t.backward, r, r)
    t.forward(r)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    t.backward(r, r)
    t.backward(r, r)
    refused(calls, t.backward, values(8), r)
    t.forward(r)
    t.backward(r, r)
    refused(calls, t.backward, r, r)


# ---------------------------------------------------------------------------
# matrices and devices
# ---------------------------------------------------------------------------
def test_matrices_of_another_shape_are_refused():
    d, ff, w, blob = 64, 256, torch.ones(64, dtype=torch.bfloat16), torch.zeros(16, dtype=torch.uint8)
    gate, up, down = matrices(d, ff)
    for bad in ([(info(d, ff), blob), up, down], [gate, (info(128, 128), blob), down], [gate, up, (info(ff, d), blob)],
                [gate, up, (info(d, 2 * ff), blob)]):
        with pytest.raises(ValueError):
            ffn.FeedForward(*bad, d, ff, w, max_tokens=4)
    flat = info(d, ff)  # coded without a shape of two dimensions: taken as the matrix, as the library's calls do
    flat.ndim, flat.shape[0], flat.shape[1] = 1, d * ff, 0
    ffn.FeedForward(gate, up, (flat, blob), d, ff, w, max_tokens=4)


def test_matrices_on_another_device_are_refused():
    gate, up, down = matrices(64, 256)
    away = torch.zeros(16, dtype=torch.uint8, device="meta")
    for bad in ([(gate[0], away), up, down], [gate, (up[0], away), down], [gate, up, (down[0], away)]):
        with pytest.raises(ValueError):
            ffn.FeedForward(*bad, 64, 256, torch.ones(64, dtype=torch.bfloat16), max_tokens=4)


def test_calls_run_on_the_buffers_device(calls, monkeypatch):
    """Whichever device is current: a default stream is the current device's."""
    current = []

    class Device:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            current.append(self.device)

        def __exit__(self, *a):
            current.pop()

    monkeypatch.setattr(torch.cuda, "device", Device)
    for name in CALLS:
        monkeypatch.setattr(afx, name, lambda *a, name=name: calls.append((name, list(current))))
    t, r = block(64, 256, 8, True), values(8)
    t.forward(r)
    t.backward(r, r)
    assert len(calls) == 8 and all(on == [t.ws.device] for _, on in calls) and not current


def test_a_stream_in_the_buffers_is_refused_without_training_too(calls):
    """The gated block would write over it before the residual is added; only
    r' itself may be the next pass's stream."""
    t, r = block(64, 256, 8, w_next=torch.ones(64, dtype=torch.bfloat16)), values(8)
    ro, xn = t.forward(r)
    for own in (t.h[:, :64], t.h[:3, 64:128], t.xn, xn):
        refused(calls, t.forward, own)
    t.forward(ro)
