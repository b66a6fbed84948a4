"""The operators of a decoder layer's feed-forward block, as a user's program
calls them, and in plain torch.

gated     h = act(x Wg^T) * (x Wu^T) for two coded weight matrices
gated_bwd its gradients: dg, du of the two projections, and dx = dg Wg + du Wu
gemm_t    y = d W (the input gradient of a product with a coded matrix)
norm      r' = r + s gate * norm(b; w_post), xn = norm(r'; w_pre): what stands
          between two blocks of a decoder layer (RMS norms)
norm_bwd  its gradients, of both norms' weights and of the gate too

Weights live in their coded form (the framework's storage format); the plain
forms multiply with the same values as BF16 matrices. Sizes are those of the
Qwen3-14B-shaped layer (hidden 5120, feed-forward 17408, heads of 128) and
odd ones around them.
"""
import math

import torch

own = False

DEV = "cuda"
THREADS = 16  # host threads of the encoder


def listed():
    return [
        # one token through the full-size block: token-by-token generation
        {"name": "gated m=1", "op": "gated", "m": 1, "rows": 17408, "cols": 5120, "act": "silu", "save": False},
        # a small odd-sized block, three tokens, the tanh form of GELU
        {"name": "gated m=3 odd", "op": "gated", "m": 3, "rows": 5461, "cols": 2056, "act": "gelu_tanh", "save": False},
        # a serving batch: 48 sequences, one token each
        {"name": "gated m=48", "op": "gated", "m": 48, "rows": 17408, "cols": 5120, "act": "silu", "save": False},
        # a prompt of 2048 tokens whose pre-activations are kept for the backward pass
        {"name": "gated m=2048", "op": "gated", "m": 2048, "rows": 17408, "cols": 5120, "act": "silu", "save": True},
        # gradients of a short odd-sized sequence, exact GELU
        {"name": "gated_bwd m=37 odd", "op": "gated_bwd", "m": 37, "rows": 4100, "cols": 1528, "act": "gelu"},
        # gradients of a training sequence through the full-size block
        {"name": "gated_bwd m=1024", "op": "gated_bwd", "m": 1024, "rows": 17408, "cols": 5120, "act": "silu"},
        # the down projection's input gradient for a handful of tokens
        {"name": "gemm_t m=16", "op": "gemm_t", "m": 16, "rows": 5120, "cols": 17408},
        # the query projection's input gradient for a sequence of 1000 tokens
        {"name": "gemm_t m=1000", "op": "gemm_t", "m": 1000, "rows": 5120, "cols": 5120},
        # between two blocks, one token: latency
        {"name": "norm m=1", "op": "norm", "m": 1, "d": 5120, "r_type": "bf16", "post": True, "gate": "none"},
        # between two blocks, a prompt of 4096 tokens, FP32 residual stream, gated
        {"name": "norm m=4096", "op": "norm", "m": 4096, "d": 5120, "r_type": "fp32", "post": True, "gate": "channel"},
        # the gradients of the same over a training sequence
        {"name": "norm_bwd m=4096", "op": "norm_bwd", "m": 4096, "d": 5120, "r_type": "fp32", "post": True,
         "gate": "channel"},
        # an odd row count and width with a gate per token
        {"name": "norm_bwd m=777 odd", "op": "norm_bwd", "m": 777, "d": 1023, "r_type": "bf16", "post": False,
         "gate": "token"},
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, even over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(("gated", "gated", "gated_bwd", "gemm_t", "norm", "norm_bwd"))
    if op in ("gated", "gated_bwd"):
        case = {"op": op, "m": _log(rng, 1, 2048 if op == "gated" else 1024), "rows": _log(rng, 64, 17408),
                "cols": _log(rng, 64, 5120, 8), "act": rng.choice(("silu", "gelu_tanh", "gelu"))}
        if op == "gated":
            case["save"] = rng.random() < 0.5
        return case
    if op == "gemm_t":
        return {"op": op, "m": _log(rng, 1, 2048), "rows": _log(rng, 64, 5120, 8), "cols": _log(rng, 64, 17408, 8)}
    return {"op": op, "m": _log(rng, 1, 4096), "d": _log(rng, 64, 5120), "r_type": rng.choice(("bf16", "fp32")),
            "post": rng.random() < 0.7, "gate": rng.choice(("none", "channel", "token"))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
EPS, SCALE = 1e-6, 0.75
_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _inputs(case, seed):
    """The tensors that a call reads, from the seed alone."""
    gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=DEV) * std + mean).to(dtype)

    op, m = case["op"], case["m"]
    if op in ("norm", "norm_bwd"):
        d, r_type = case["d"], _TYPES[case["r_type"]]
        gate = {"none": None, "channel": (d,), "token": (m, d)}[case["gate"]]
        t = {"b": normal(m, d, std=1.5, dtype=torch.float32),  # a product's FP32 output
             "r": normal(m, d, std=2.0, dtype=r_type),
             "w_post": normal(d, std=0.2, mean=1.0) if case["post"] else None,
             "gate": normal(*gate, std=0.5) if gate else None,
             "w_pre": normal(d, std=0.2, mean=1.0)}
        if op == "norm_bwd":  # here r is the stream after the block, as the forward pass left it
            t["dxn"] = normal(m, d, std=1e-2)
            t["dr_out"] = normal(m, d, std=1e-2, dtype=r_type)
        return t
    rows, cols = case["rows"], case["cols"]
    if op == "gemm_t":
        return {"w": normal(rows, cols, std=0.02), "d": normal(m, rows, std=1e-2)}
    t = {"wg": normal(rows, cols, std=0.02), "wu": normal(rows, cols, std=0.02)}
    if op == "gated":
        t["x"] = normal(m, cols)
    else:
        pre = 0.02 * math.sqrt(cols)  # the spread of a projection of normalised tokens
        t["g"], t["u"] = normal(m, rows, std=pre), normal(m, rows, std=pre)
        t["dh"] = normal(m, rows, std=1e-2, dtype=torch.float32)
    return t


def _coded(w):
    """A weight matrix as a user of the framework holds it: its coded blob on
    the GPU and what afx_query says of it."""
    from lossless_bf16_weight_afx_amd import afx

    blob = afx.afx_encode(w.view(torch.int16).cpu().numpy(), tuple(w.shape), threads=THREADS)
    return afx.afx_query(blob), afx.to_device(blob)


def prepare(case, seed):
    t = _inputs(case, seed)
    s = {"case": case, "t": t}
    if not own:
        return s
    from lossless_bf16_weight_afx_amd import afx

    op, m = case["op"], case["m"]

    def buf(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    if op in ("gated", "gated_bwd"):
        rows, cols = case["rows"], case["cols"]
        s["wg"], s["wu"] = _coded(t.pop("wg")), _coded(t.pop("wu"))
        s["w"] = afx.gated_weights(s["wg"][0], s["wg"][1].data_ptr(), s["wu"][0], s["wu"][1].data_ptr(), rows, cols,
                                   {"silu": afx.ACT_SILU, "gelu_tanh": afx.ACT_GELU_TANH,
                                    "gelu": afx.ACT_GELU}[case["act"]])
        s["ws"] = buf(afx.afx_restore_gated_workspace(rows, cols, m, backward=op == "gated_bwd"), dtype=torch.uint8)
        s["gu"] = [buf(m, rows), buf(m, rows)]
        s["out"] = buf(m, rows) if op == "gated" else buf(m, cols)
    elif op == "gemm_t":
        rows, cols = case["rows"], case["cols"]
        s["w"] = _coded(t.pop("w"))
        s["ws"] = buf(afx.afx_restore_gemm_t_workspace(rows, cols, m), dtype=torch.uint8)
        s["out"] = buf(m, cols, dtype=torch.float32)
    else:
        d, gate = case["d"], t["gate"]
        s["p"] = afx.block_norm(d, EPS, SCALE, afx.TYPE_FP32 if case["r_type"] == "fp32" else afx.TYPE_BF16,
                                w_post=_ptr(t["w_post"]), gate=_ptr(gate),
                                gate_stride=d if case["gate"] == "token" else 0, w_pre=_ptr(t["w_pre"]))
        s["xn"], s["r_out"] = buf(m, d), buf(m, d, dtype=t["r"].dtype)
        if op == "norm_bwd":
            s["ws"] = buf(afx.afx_block_norm_workspace(s["p"], m), dtype=torch.uint8)
            s["dw"] = [buf(d, dtype=torch.float32), buf(d, dtype=torch.float32) if case["post"] else None,
                       buf(*gate.shape, dtype=torch.float32) if gate is not None else None]
    return s


def _ptr(t):
    return 0 if t is None else t.data_ptr()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from lossless_bf16_weight_afx_amd import afx

    case, t = s["case"], s["t"]
    op, m = case["op"], case["m"]
    stream = torch.cuda.current_stream().cuda_stream
    if op == "gated":
        rows, cols = case["rows"], case["cols"]
        g, u = s["gu"] if case["save"] else (None, None)
        afx.afx_restore_gated_async(s["w"], m, t["x"].data_ptr(), cols, s["out"].data_ptr(), rows, _ptr(g), _ptr(u),
                                    rows, s["ws"].data_ptr(), s["ws"].numel(), stream)
        return {"h": s["out"], "g": g, "u": u} if case["save"] else {"h": s["out"]}
    if op == "gated_bwd":
        rows, cols = case["rows"], case["cols"]
        dg, du = s["gu"]
        afx.afx_restore_gated_backward_async(s["w"], m, t["dh"].data_ptr(), rows, t["g"].data_ptr(),
                                             t["u"].data_ptr(), rows, s["out"].data_ptr(), cols, dg.data_ptr(),
                                             du.data_ptr(), s["ws"].data_ptr(), s["ws"].numel(), stream)
        return {"dx": s["out"], "dg": dg, "du": du}
    if op == "gemm_t":
        info, blob = s["w"]
        afx.afx_restore_gemm_t_async(info, blob.data_ptr(), case["rows"], case["cols"], t["d"].data_ptr(), m,
                                     s["out"].data_ptr(), False, s["ws"].data_ptr(), s["ws"].numel(), stream)
        return {"y": s["out"]}
    d = case["d"]
    if op == "norm":
        afx.afx_block_norm_async(s["p"], m, t["b"].data_ptr(), d, t["r"].data_ptr(), d, s["r_out"].data_ptr(), d,
                                 s["xn"].data_ptr(), d, stream)
        return {"xn": s["xn"], "r_out": s["r_out"]}
    dw_pre, dw_post, dgate = s["dw"]
    afx.afx_block_norm_backward_async(s["p"], m, t["b"].data_ptr(), d, t["r"].data_ptr(), d, t["dxn"].data_ptr(), d,
                                      t["dr_out"].data_ptr(), d, s["r_out"].data_ptr(), d, s["xn"].data_ptr(), d,
                                      _ptr(dw_pre), _ptr(dw_post), _ptr(dgate), s["ws"].data_ptr(), s["ws"].numel(),
                                      stream)
    return {"dr": s["r_out"], "db": s["xn"], "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}


def _act(g, kind):
    """act(g) and its derivative."""
    if kind == "silu":
        sig = torch.sigmoid(g)
        return g * sig, sig * (1 + g * (1 - sig))
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        th = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + th), 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)
    cdf = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))


def _run_plain(s):
    case, t = s["case"], s["t"]
    op = case["op"]
    f = lambda v: v.float()  # noqa: E731
    if op == "gated":
        x = f(t["x"])
        g, u = x @ f(t["wg"]).t(), x @ f(t["wu"]).t()
        h = (_act(g, case["act"])[0] * u).bfloat16()
        return {"h": h, "g": g.bfloat16(), "u": u.bfloat16()} if case["save"] else {"h": h}
    if op == "gated_bwd":
        dh, u = t["dh"], f(t["u"])
        a, da = _act(f(t["g"]), case["act"])
        dg, du = dh * u * da, dh * a
        return {"dx": (dg @ f(t["wg"]) + du @ f(t["wu"])).bfloat16(), "dg": dg.bfloat16(), "du": du.bfloat16()}
    if op == "gemm_t":
        return {"y": f(t["d"]) @ f(t["w"])}
    b, r, w_pre = t["b"], f(t["r"]), f(t["w_pre"])
    w_post = f(t["w_post"]) if case["post"] else None
    gate = f(t["gate"]) if t["gate"] is not None else 1.0
    if op == "norm":
        if w_post is not None:
            b = b * torch.rsqrt((b * b).mean(-1, keepdim=True) + EPS) * w_post
        r = r + SCALE * gate * b
        xn = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * w_pre
        return {"xn": xn.bfloat16(), "r_out": r.to(t["r"].dtype)}
    # norm_bwd: with n = v / sqrt(mean(v^2) + eps) and dn the gradient of n,
    # dv = (dn - n mean(dn n)) / sqrt(mean(v^2) + eps)
    dxn, dr_out = f(t["dxn"]), f(t["dr_out"])
    k = torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS)
    n, dn = r * k, dxn * w_pre
    dr = dr_out + (dn - n * (dn * n).mean(-1, keepdim=True)) * k
    dw_pre = (dxn * n).sum(0)
    dbhat = SCALE * gate * dr
    bhat, db, dw_post = b, dbhat, None
    if w_post is not None:
        k = torch.rsqrt((b * b).mean(-1, keepdim=True) + EPS)
        n, dn = b * k, dbhat * w_post
        bhat, dw_post = n * w_post, (dbhat * n).sum(0)
        db = (dn - n * (dn * n).mean(-1, keepdim=True)) * k
    dgate = None
    if case["gate"] != "none":
        dgate = SCALE * bhat * dr
        dgate = dgate.sum(0) if case["gate"] == "channel" else dgate
    return {"dr": dr.to(t["r"].dtype), "db": db.bfloat16(), "dw_pre": dw_pre, "dw_post": dw_post, "dgate": dgate}


# ---------------------------------------------------------------------------
# the definition in 64 bits, and the work of a pass
# ---------------------------------------------------------------------------
def exact(case, seed):
    """From the formulas, with derivatives taken by torch's autograd of the
    forward formula in 64 bits."""
    t = {k: (v.double() if v is not None else None) for k, v in _inputs(case, seed).items()}
    op = case["op"]
    if op == "gemm_t":
        return {"y": torch.matmul(t["d"], t["w"])}

    def act(v):
        if case["act"] == "silu":
            return v / (1 + torch.exp(-v))
        if case["act"] == "gelu_tanh":
            return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
        return v * torch.special.ndtr(v)

    if op == "gated":
        g, u = torch.matmul(t["x"], t["wg"].t()), torch.matmul(t["x"], t["wu"].t())
        return {"h": act(g) * u, "g": g, "u": u} if case["save"] else {"h": act(g) * u}
    if op == "gated_bwd":
        g, u = t["g"].requires_grad_(), t["u"].requires_grad_()
        dg, du = torch.autograd.grad(act(g) * u, (g, u), t["dh"])
        return {"dx": torch.matmul(torch.cat((dg, du), 1), torch.cat((t["wg"], t["wu"]), 0)), "dg": dg, "du": du}

    def rms(v, w):
        return v / torch.sqrt(v.square().sum(-1, keepdim=True) / case["d"] + EPS) * w

    def step(b, w_post, gate):
        b = b if w_post is None else rms(b, w_post)
        return SCALE * (b if gate is None else b * gate)

    if op == "norm":
        r = t["r"] + step(t["b"], t["w_post"], t["gate"])
        return {"xn": rms(r, t["w_pre"]), "r_out": r}
    r, w_pre = t["r"].requires_grad_(), t["w_pre"].requires_grad_()
    dr, dw_pre = torch.autograd.grad(rms(r, w_pre), (r, w_pre), t["dxn"])
    dr = dr + t["dr_out"]
    names = [k for k in ("b", "w_post", "gate") if t[k] is not None]
    for k in names:
        t[k].requires_grad_()
    got = dict(zip(names, torch.autograd.grad(step(t["b"], t["w_post"], t["gate"]), [t[k] for k in names], dr)))
    return {"dr": dr, "db": got["b"], "dw_pre": dw_pre, "dw_post": got.get("w_post"), "dgate": got.get("gate")}


# Bytes of a coded N(0, 0.02) weight: sign and mantissa, 2.59 bits of exponent
# code, 16 bits of group start per 32 values, 64 bits per 4096.
CODED = 1 + 2.59 / 8 + 2 / 32 + 8 / 4096


def work(case):
    op, m = case["op"], case["m"]
    if op in ("gated", "gated_bwd"):
        rows, cols = case["rows"], case["cols"]
        n = 2 * CODED * rows * cols
        if op == "gated":
            n += 2 * m * cols + 2 * m * rows * (3 if case["save"] else 1)
        else:
            n += 2 * m * cols + (4 + 2 + 2 + 2 + 2) * m * rows
        return {"bytes": n, "flops": 4.0 * m * rows * cols}
    if op == "gemm_t":
        rows, cols = case["rows"], case["cols"]
        return {"bytes": CODED * rows * cols + 2 * m * rows + 4 * m * cols, "flops": 2.0 * m * rows * cols}
    d, r = case["d"], 4 if case["r_type"] == "fp32" else 2
    per_token = 2 if case["gate"] == "token" else 0
    if op == "norm":
        return {"bytes": m * d * (4 + r + r + 2 + per_token), "flops": 10.0 * m * d}
    per_token *= 3  # the gate and its FP32 gradient
    return {"bytes": m * d * (4 + r + 2 + r + r + 2 + per_token) + 12 * d, "flops": 25.0 * m * d}
