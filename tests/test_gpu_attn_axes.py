"""attn.Attention with positions along several axes, a norm after the block, a
gate and a residual scale, over prompts and single tokens of two sequences,
against the formulas in 64 bits. Tolerance as in tests/test_gpu_attn_run.py:
the products' result is within 8 roundings of its norm; the norm after it and
the gate multiply what is left by between LO and HI, the residual add rounds
once more, and xn' once."""
import numpy as np
import pytest

import oracle
from lossless_bf16_weight_afx_amd import afx, attn, cache, synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

D, HEADS, KV, DIM, EPS, SCALE = 256, 4, 2, 64, 1e-6, 0.5
STEP, LO, HI = 2.0 ** -8, 0.8 ** 2, 1.2 ** 2


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    afx.lib()


def unit(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


@pytest.mark.parametrize("pairing", [afx.ROPE_HALVES, afx.ROPE_NEIGHBOURS])
@pytest.mark.parametrize("axes, pairs", [(1, 32), (3, 32), (2, 20), (4, 9)])
def test_positions_along_axes(pairing, axes, pairs):
    rng = np.random.default_rng(100 * axes + pairs + pairing)
    mats, wide = [], []
    for rows, cols in ((HEADS * DIM, D), (KV * DIM, D), (KV * DIM, D), (D, HEADS * DIM)):
        bits = synth.f32_to_bf16_bits((rng.standard_normal(rows * cols) * cols ** -0.5).astype(np.float32))
        blob = oracle.encode(bits, (rows, cols))
        mats.append((afx.afx_query(blob), afx.to_device(blob)))
        wide.append(torch.from_numpy(synth.bf16_bits_to_f32(bits).reshape(rows, cols).astype(np.float64)))
    vec = lambda n: torch.from_numpy(rng.uniform(0.8, 1.2, n)).bfloat16().cuda()  # noqa: E731
    w = {n: vec(d) for n, d in dict(pre=D, post=D, gate=D, nxt=D, q=DIM, k=DIM).items()}
    f = {n: t.cpu().double() for n, t in w.items()}
    freq = torch.tensor([100.0 ** (-i / pairs) for i in range(pairs)], device="cuda")
    axis = torch.from_numpy(rng.integers(0, axes, pairs)).to(torch.uint8).cuda()
    c = cache.PagedCache(1, KV, DIM, n_pages=12, page_tokens=16, max_seqs=2, max_pages=6, max_tokens=64)
    c.data.fill_(float("nan"))
    half = attn.Attention(*mats, D, c, 0, HEADS, w["pre"], w_q=w["q"], w_k=w["k"], freq=freq, axis=axis, n_axes=axes,
                          pairing=pairing, w_post=w["post"], block_gate=w["gate"], w_next=w["nxt"], eps=EPS, scale=SCALE)
    one, two = (slice(0, pairs), slice(pairs, 2 * pairs)) if pairing == afx.ROPE_HALVES else \
        (slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2))

    def turn(x, pos):
        t = (pos.double()[axis.cpu().long()].t() * freq.cpu().double())[:, None]
        y = x.clone()
        y[..., one] = x[..., one] * t.cos() - x[..., two] * t.sin()
        y[..., two] = x[..., two] * t.cos() + x[..., one] * t.sin()
        return y

    held = {s: (torch.zeros(0, KV, DIM).double(),) * 2 for s in range(2)}
    for rows in ([(1, 37), (0, 20)], [(0, 1), (1, 1)], [(1, 3), (0, 1)]):
        starts = np.concatenate([[0], np.cumsum([n for _, n in rows])])
        m = int(starts[-1])
        r = torch.from_numpy(rng.standard_normal((m, D))).bfloat16().cuda()
        # the axes' rows lie apart in one wider tensor
        pos = torch.from_numpy(rng.integers(-50, 3000, (axes, m + 9))).int().cuda()[:, 4:4 + m]
        step = c.extend(torch.tensor([s for s, _ in rows], dtype=torch.int32, device="cuda"),
                        torch.from_numpy(starts).int().cuda(), m)
        r1, xn1 = half.forward(r, step, pos)
        x, p = r.cpu().double(), pos.cpu()
        q, k, v = (unit(x, f["pre"]) @ t.t() for t in wide[:3])
        q = turn(unit(q.view(m, HEADS, DIM), f["q"]), p)
        k = turn(unit(k.view(m, KV, DIM), f["k"]), p)
        a = torch.zeros(m, HEADS * DIM).double()
        for (s, n), at in zip(rows, starts):
            part = slice(int(at), int(at) + n)
            hk, hv = torch.cat([held[s][0], k[part]]), torch.cat([held[s][1], v[part].view(n, KV, DIM)])
            held[s] = hk, hv
            seen = torch.arange(len(hk))[None] <= torch.arange(len(hk) - n, len(hk))[:, None]
            for h in range(HEADS):
                score = (q[part, h] @ hk[:, h // 2].t() * DIM ** -0.5).masked_fill(~seen, -torch.inf)
                a[part, h * DIM:(h + 1) * DIM] = torch.softmax(score, -1) @ hv[:, h // 2]
        b = SCALE * f["gate"] * unit(a @ wide[3].t(), f["post"])
        want, got = x + b, r1.cpu().double()
        assert (got - want).norm() <= 8 * STEP * HI / LO * b.norm() + STEP * want.norm()
        want = unit(want, f["nxt"])
        assert (xn1.cpu().double() - want).norm() <= (10 * HI / LO) * STEP * want.norm()
