"""The values of a head that do not turn: they stay what the norm made them,
whatever the values beside them hold, in both directions."""
import math

import pytest

from lossless_bf16_weight_afx_amd import afx
from test_gpu_heads import Heads, forward

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


def strange(x, dim, rot):
    """Infinities, NaN and zeros of both signs among the values behind rot of each head [m, heads * dim]."""
    x = x.reshape(x.shape[0], -1, dim)
    for i, v in enumerate((math.inf, -math.inf, math.nan, -0.0, 0.0)):
        x[i::7, :, rot + (5 * i) % (dim - rot)] = v


def bits(t):
    return t.contiguous().view(torch.int16)


def same(got, want):
    """Bit for bit, but for a NaN's."""
    return bool(((bits(got) == bits(want)) | (torch.isnan(got) & torch.isnan(want))).all())


@pytest.mark.parametrize("pairing", [afx.ROPE_HALVES, afx.ROPE_NEIGHBOURS])
@pytest.mark.parametrize("dim, rot", [(64, 0), (64, 16), (128, 64), (80, 42), (256, 128), (24, 10)])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("m", [1, 35])
def test_forward(pairing, dim, rot, shift, m):
    t = Heads(dim + rot + m, m, dim, rot, pairing=pairing, w_q=False, w_k=False, shift=shift)
    clean = {n: t.want(n) for n in "qk"}
    for n in "qk":
        x = t.x[n].clone()
        strange(x, dim, rot)
        t.x[n][:] = x
    out, pages = forward(t)
    for n in "qk":
        heads = t.x[n].reshape(m, -1, dim)
        got = out[n][:, :heads.shape[1] * dim].cpu().reshape(m, -1, dim)
        assert same(got[..., rot:], heads[..., rot:].bfloat16())
        want, bound = clean[n]
        assert bool(((got.double() - want).abs() <= bound)[..., :rot].all())
    page, off = t.slots.long() // t.page, t.slots.long() % t.page
    cached = pages[0].cpu()[page, :, :, off].reshape(m, -1, dim)
    assert same(cached[..., rot:], t.x["k"].reshape(m, -1, dim)[..., rot:].bfloat16())


@pytest.mark.parametrize("pairing", [afx.ROPE_HALVES, afx.ROPE_NEIGHBOURS])
@pytest.mark.parametrize("dim, rot", [(64, 0), (64, 16), (128, 64), (80, 42), (256, 128), (24, 10)])
@pytest.mark.parametrize("m", [1, 35])
def test_backward(pairing, dim, rot, m):
    t = Heads(dim + rot + m, m, dim, rot, pairing=pairing, w_q=False, w_k=False)
    clean = {n: t.want_grad(n) for n in "qk"}
    dev = {}
    for n in "qk":
        x = t.dy[n].clone()
        strange(x, dim, rot)
        t.dy[n] = x
        dev[n] = x.cuda()
    p, pos = t.params(), t.pos.cuda()
    got = {n: torch.full_like(dev[n], 7.0) for n in "qk"}
    afx.afx_heads_backward_async(p, m, pos.data_ptr(), pos.stride(0), 0, 0, 0, 0, dev["q"].data_ptr(),
                                 dev["q"].stride(0), dev["k"].data_ptr(), dev["k"].stride(0), got["q"].data_ptr(),
                                 got["q"].stride(0), got["k"].data_ptr(), got["k"].stride(0), 0, 0, 0, 0,
                                 torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for n in "qk":
        g, dy = got[n].cpu().reshape(m, -1, dim), t.dy[n].reshape(m, -1, dim)
        assert same(g[..., rot:], dy[..., rot:])
        want, bound = clean[n][:2]
        assert bool(((g.double() - want).abs() <= bound)[..., :rot].all())
