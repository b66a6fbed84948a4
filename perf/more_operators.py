"""The operators of a decoder layer's attention half over a paged cache, as a
user's program calls them, and in plain torch.

heads      what stands between the q, k, v products and the attention: the
           heads' norms, rotary positions with one or more axes, and the write
           of keys and values to the cache's pages
heads_bwd  the gradients of norms and rotation
attend     attention of new tokens (one, a few drafted ones, a prompt's chunk)
           over the cached ones of their sequences
pages      the cache's pages: branches of sequences forked, grown by new tokens
           (copying a shared last page) and freed; live pages compacted

Sizes are those of the Qwen3-14B-shaped layer (40 query heads and 8 key and
value heads of 128) and odd ones around them.

A page holds page_tokens tokens of every key-value head: keys as
[kv_heads, dim / 8, page_tokens, 8], values as [kv_heads, page_tokens / 8, dim, 8].
"""
import math
import random

import torch

own = False

DEV = "cuda"


def listed():
    full = {"q_heads": 40, "kv_heads": 8, "dim": 128}
    return [
        # one token of token-by-token generation, far into its sequence: latency
        {"name": "heads m=1", "op": "heads", "m": 1, **full, "rot": 128, "axes": 1, "pairing": "halves", "norm": True,
         "page": 16},
        # a prompt of 4096 tokens with images: time, height and width axes
        {"name": "heads m=4096 axes", "op": "heads", "m": 4096, **full, "rot": 128, "axes": 3, "pairing": "halves",
         "norm": True, "page": 32},
        # the gradients of a training sequence
        {"name": "heads_bwd m=2048", "op": "heads_bwd", "m": 2048, **full, "rot": 128, "axes": 1,
         "pairing": "halves", "norm": True},
        # an odd token count, part of each small head rotated, neighbouring pairs, two axes
        {"name": "heads_bwd m=333 odd", "op": "heads_bwd", "m": 333, "q_heads": 12, "kv_heads": 4, "dim": 80,
         "rot": 40, "axes": 2, "pairing": "neighbours", "norm": True},
        # one token over a short sequence: latency
        {"name": "attend 1 over 500", "op": "attend", "seqs": 1, "new": 1, "len": 500, "ragged": False, **full,
         "page": 16, "window": 0},
        # a serving batch: 64 sequences of up to 8192 tokens, one new token each
        {"name": "attend 64x1 over 8192", "op": "attend", "seqs": 64, "new": 1, "len": 8192, "ragged": True, **full,
         "page": 16, "window": 0},
        # one token over one very long sequence
        {"name": "attend 1 over 131072", "op": "attend", "seqs": 1, "new": 1, "len": 131072, "ragged": False, **full,
         "page": 64, "window": 0},
        # drafted tokens of 24 sequences (0 to 6 each), odd small heads, a window
        {"name": "attend 24x6 window", "op": "attend", "seqs": 24, "new": 6, "len": 3001, "ragged": True,
         "q_heads": 12, "kv_heads": 4, "dim": 80, "page": 32, "window": 1000},
        # a chunk of a long prompt: 2048 new tokens, the last of 16384
        {"name": "attend 2048 over 16384", "op": "attend", "seqs": 1, "new": 2048, "len": 16384, "ragged": False,
         **full, "page": 32, "window": 0},
        # three branches of one short sequence in a few layers: latency
        {"name": "pages branch 3", "op": "branch", "parents": 1, "branches": 3, "new": 1, "len": 200, "planes": 4,
         "kv_heads": 8, "dim": 128, "page": 16},
        # a beam step: 64 branches of 8 sequences over 40 layers, the old ones freed
        {"name": "pages branch 64", "op": "branch", "parents": 8, "branches": 64, "new": 2, "len": 1024,
         "planes": 80, "kv_heads": 8, "dim": 128, "page": 16},
        # half the sequences have gone: the live pages of 40 layers move to the front
        {"name": "pages compact", "op": "compact", "seqs": 24, "len": 700, "planes": 80, "kv_heads": 8, "dim": 128,
         "page": 16},
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, even over its logarithm, a multiple of step."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(("heads", "heads_bwd", "attend", "attend", "attend", "branch", "compact"))
    q_heads, kv_heads = rng.choice(((40, 8), (8, 8), (12, 4), (5, 1), (16, 2)))
    dim, page = rng.choice((64, 80, 96, 128, 128, 192, 256)), rng.choice((16, 32, 64, 128))
    if op in ("heads", "heads_bwd"):
        if q_heads * dim > 5120:
            dim = 128
        case = {"op": op, "m": _log(rng, 1, 4096 if op == "heads" else 2048), "q_heads": q_heads,
                "kv_heads": kv_heads, "dim": dim, "rot": rng.choice((dim, dim, dim // 2)),
                "axes": rng.choice((1, 1, 2, 3)), "pairing": rng.choice(("halves", "halves", "neighbours")),
                "norm": rng.random() < 0.7}
        if op == "heads":
            case["page"] = page
        return case
    if op == "attend":
        if q_heads * dim > 5120:
            dim = 128
        new = rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 16, 2048)))
        seqs = _log(rng, 1, max(1, min(64, 4096 // new)))
        most = min(131072, 2 ** 28 // (kv_heads * dim * seqs), 31 * 10 ** 6 // (seqs * new))
        return {"op": op, "seqs": seqs, "new": new, "len": _log(rng, max(new, 16), max(new, most)),
                "ragged": rng.random() < 0.7, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page,
                "window": rng.choice((0, 0, _log(rng, 16, 4096)))}
    size = page * kv_heads * dim * 2
    planes = 2 * _log(rng, 1, 40)
    if op == "branch":
        parents, branches = _log(rng, 1, 8), _log(rng, 1, 64)
        length = _log(rng, 20, max(20, min(1024, 6 * 10 ** 8 // (size * planes * parents) * page)))
        return {"op": op, "parents": parents, "branches": branches, "new": rng.choice((1, 1, 2, 5)), "len": length,
                "planes": max(2, min(planes, 6 * 10 ** 8 // (size * (branches + parents)) // 2 * 2)),
                "kv_heads": kv_heads, "dim": dim, "page": page}
    seqs = _log(rng, 2, 24)
    return {"op": op, "seqs": seqs, "len": _log(rng, 20, max(20, min(4096, 10 ** 9 // (size * planes * seqs) * page))),
            "planes": planes, "kv_heads": kv_heads, "dim": dim, "page": page}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
EPS, BASE = 1e-6, 1e6


def _lengths(n, most, ragged):
    """Lengths of n sequences of up to `most` tokens, the first the longest."""
    return [most if not ragged or s == 0 else max(1, int(most * (0.37 + 0.618034 * s) % most)) for s in range(n)]


def _fresh(case):
    """(length, new tokens) of each sequence of an attend case; a ragged
    batch has sequences without new tokens too."""
    lens = _lengths(case["seqs"], case["len"], case["ragged"])
    new = case["new"]
    if not case["ragged"] or new == 1:
        return [(n, min(new, n)) for n in lens]
    return [(n, min(n, (7 * s + new) % (new + 1))) for s, n in enumerate(lens)]


def _up(a, b):
    return -(-a // b)


def _tables(pages, n_pages, order):
    """Page tables [sequences, widest], -1 behind the last page, from an
    order of the cache's pages."""
    table = torch.full((len(pages), max(pages)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = order[at:at + n].int()
        at += n
    assert at <= n_pages
    return table.to(DEV)


def _inputs(case, seed):
    """The tensors that a call reads, from the seed alone."""
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    cpu = torch.Generator().manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=DEV) * std + mean).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=DEV)

    op = case["op"]
    if op in ("heads", "heads_bwd"):
        m, d, rot, axes = case["m"], case["dim"], case["rot"], case["axes"]
        pairs = rot // 2
        first = int(torch.randint(0, 100000, (1,), generator=cpu))
        pos = torch.arange(m)[None].repeat(axes, 1) + first
        for a in range(1, axes):  # inside images the other axes run over rows and columns
            pos[a] = first + (torch.arange(m) // (1 if a == axes - 1 else 32)) % 32
        # pairs in sections, one per axis
        axis = torch.arange(pairs, dtype=torch.int64) * axes // max(pairs, 1)
        t = {"q": normal(m, case["q_heads"] * d, std=1.5, dtype=torch.float32),  # products' FP32 outputs
             "k": normal(m, case["kv_heads"] * d, std=1.5, dtype=torch.float32),
             "pos": pos.int().to(DEV), "axis": axis.to(torch.uint8).to(DEV),
             "freq": (BASE ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float().to(DEV),
             "w_q": normal(d, std=0.2, mean=1.0) if case["norm"] else None,
             "w_k": normal(d, std=0.2, mean=1.0) if case["norm"] else None}
        if op == "heads_bwd":
            t["dq"] = normal(m, case["q_heads"] * d, std=1e-2)
            t["dk"] = normal(m, case["kv_heads"] * d, std=1e-2)
            return t
        t["v"] = normal(m, case["kv_heads"] * d, dtype=torch.float32)
        page = case["page"]
        n_pages = _up(m, page) + 3
        order = torch.randperm(n_pages, generator=cpu)
        at = first % page + torch.arange(m)  # the first tokens continue a page
        t["slots"] = (order[at // page] * page + at % page).int().to(DEV)
        t["k_pages"], t["v_pages"] = _pages(case, n_pages, normal)
        return t
    if op == "attend":
        fresh, page = _fresh(case), case["page"]
        need = [_up(n, page) for n, _ in fresh]
        n_pages = sum(need) + 2
        t = {"q": normal(sum(n for _, n in fresh), case["q_heads"] * case["dim"], std=2.0),
             "table": _tables(need, n_pages, torch.randperm(n_pages, generator=cpu)),
             "len": ints([n for n, _ in fresh]),
             "starts": ints([sum(n for _, n in fresh[:s]) for s in range(len(fresh) + 1)])}
        t["k_pages"], t["v_pages"] = _pages(case, n_pages, normal)
        return t
    page, elems = case["page"], case["page"] * case["kv_heads"] * case["dim"]
    if op == "branch":
        lens, n = _lengths(case["parents"], case["len"], True), case["branches"]
        need = [_up(v, page) for v in lens]
        n_pages = sum(need) + n * (1 + _up(case["new"], page)) + 1
        wide = max(need) + _up(case["new"], page)
        table = torch.full((case["parents"] + n, wide), -1, dtype=torch.int32, device=DEV)
        table[:case["parents"], :max(need)] = _tables(need, n_pages, torch.randperm(n_pages, generator=cpu))
        t = {"table": table, "len": ints(lens + [0] * n),
             "src": torch.randint(0, case["parents"], (n,), generator=cpu).int().to(DEV),
             "dst": case["parents"] + torch.randperm(n, generator=cpu).int().to(DEV),
             "starts": ints([case["new"] * b for b in range(n + 1)])}
    else:
        # sequences grown together, a page at a time; every other one has gone
        lens = _lengths(case["seqs"], case["len"], True)
        need = [_up(v, page) for v in lens]
        n_pages = sum(need) + 5
        grown = sorted((j, random.Random(f"{seed} {s} {j}").random(), s) for s in range(len(need))
                       for j in range(need[s]))
        table = torch.full((len(need), max(need)), -1, dtype=torch.int32)
        for i, (j, _, s) in enumerate(grown):
            if s % 2 == 0:
                table[s, j] = i
        t = {"table": table.to(DEV), "len": ints([v if s % 2 == 0 else 0 for s, v in enumerate(lens)])}
    used = t["table"][t["table"] >= 0].long()
    t["refs"] = torch.zeros(n_pages, dtype=torch.int32, device=DEV)
    t["refs"][used] = 1
    t["data"] = torch.randint(-2 ** 15, 2 ** 15, (case["planes"], n_pages, elems), generator=gen, device=DEV,
                              dtype=torch.int16)
    return t


def _pages(case, n_pages, normal):
    h, d, page = case["kv_heads"], case["dim"], case["page"]
    return normal(n_pages, h, d // 8, page, 8), normal(n_pages, h, page // 8, d, 8)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def prepare(case, seed):
    t = _inputs(case, seed)
    s = {"case": case, "t": t}
    op = case["op"]
    if op == "compact":  # what the tables were before: each pass starts from them
        s["was"] = {k: t[k].clone() for k in ("table", "len", "refs")}
    if not own:
        return s
    from lossless_bf16_weight_afx_amd import afx

    def buf(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=DEV)

    if op in ("heads", "heads_bwd"):
        s["p"] = afx.heads(case["q_heads"], case["kv_heads"], case["dim"], case["rot"],
                           {"halves": afx.ROPE_HALVES, "neighbours": afx.ROPE_NEIGHBOURS}[case["pairing"]],
                           case["axes"], EPS, _ptr(t["w_q"]), _ptr(t["w_k"]), _ptr(t["freq"]), _ptr(t["axis"]))
        s["q_out"] = buf(*t["q"].shape)
        if op == "heads":
            s["kv"] = _kv(case, t)
        else:
            s["k_out"] = buf(*t["k"].shape)
            s["dw"] = [buf(case["dim"], dtype=torch.float32) if case["norm"] else None for _ in range(2)]
            s["ws"] = buf(afx.afx_heads_workspace(s["p"], case["m"]), dtype=torch.uint8)
    elif op == "attend":
        m = t["q"].shape[0]
        s["kv"] = _kv(case, t)
        s["table"] = afx.page_table(t["table"].data_ptr(), t["table"].stride(0), t["len"].data_ptr(), 0, case["seqs"],
                                    t["table"].shape[1], t["k_pages"].shape[0], case["page"])
        s["p"] = afx.attend(case["q_heads"], case["dim"] ** -0.5, True, case["window"], case["new"], case["len"])
        s["out"], s["lse"] = buf(*t["q"].shape), buf(m, case["q_heads"], dtype=torch.float32)
        s["ws"] = buf(afx.afx_attend_workspace(s["p"], s["kv"], case["seqs"], m), dtype=torch.uint8)
    else:
        planes, n_pages, elems = t["data"].shape
        s["table"] = afx.page_table(t["table"].data_ptr(), t["table"].stride(0), t["len"].data_ptr(),
                                    t["refs"].data_ptr(), t["table"].shape[0], t["table"].shape[1], n_pages,
                                    case["page"])
        s["data"] = afx.page_data(t["data"].data_ptr(), 2 * elems, 2 * elems * n_pages, planes)
        if op == "branch":
            n = case["branches"]
            s["slots"], s["pos"] = buf(n * case["new"], dtype=torch.int32), buf(n * case["new"], dtype=torch.int32)
            s["granted"] = buf(n, dtype=torch.int32)
            s["ws"] = buf(afx.afx_pages_extend_workspace(s["table"], n), dtype=torch.uint8)
        else:
            s["map"], s["live"] = buf(n_pages, dtype=torch.int32), buf(1, dtype=torch.int32)
            s["ws"] = buf(afx.afx_pages_compact_workspace(s["table"]), dtype=torch.uint8)
    return s


def _kv(case, t):
    from lossless_bf16_weight_afx_amd import afx

    return afx.kv_pages(t["k_pages"].data_ptr(), t["v_pages"].data_ptr(), t["k_pages"].shape[0], case["page"],
                        case["kv_heads"], case["dim"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from lossless_bf16_weight_afx_amd import afx

    case, t = s["case"], s["t"]
    op = case["op"]
    stream = torch.cuda.current_stream().cuda_stream
    if op in ("heads", "heads_bwd"):
        m, nq, nk = case["m"], case["q_heads"] * case["dim"], case["kv_heads"] * case["dim"]
        if op == "heads":
            afx.afx_heads_async(s["p"], m, t["pos"].data_ptr(), m, t["q"].data_ptr(), nq, t["k"].data_ptr(), nk,
                                t["v"].data_ptr(), nk, s["q_out"].data_ptr(), nq, 0, 0, s["kv"],
                                t["slots"].data_ptr(), stream)
            return {"q": s["q_out"], "k_pages": t["k_pages"], "v_pages": t["v_pages"]}
        dw_q, dw_k = s["dw"]
        afx.afx_heads_backward_async(s["p"], m, t["pos"].data_ptr(), m, t["q"].data_ptr(), nq, t["k"].data_ptr(), nk,
                                     t["dq"].data_ptr(), nq, t["dk"].data_ptr(), nk, s["q_out"].data_ptr(), nq,
                                     s["k_out"].data_ptr(), nk, _ptr(dw_q), _ptr(dw_k), s["ws"].data_ptr(),
                                     s["ws"].numel(), stream)
        return {"dq": s["q_out"], "dk": s["k_out"], "dw_q": dw_q, "dw_k": dw_k}
    if op == "attend":
        n = case["q_heads"] * case["dim"]
        afx.afx_attend_async(s["p"], s["kv"], s["table"], case["seqs"], 0, t["starts"].data_ptr(), t["q"].shape[0],
                             t["q"].data_ptr(), n, s["out"].data_ptr(), n, s["lse"].data_ptr(), s["ws"].data_ptr(),
                             s["ws"].numel(), stream)
        return {"out": s["out"], "lse": s["lse"]}
    if op == "branch":
        n = case["branches"]
        afx.afx_pages_trim_async(s["table"], n, t["dst"].data_ptr(), 0, stream)
        afx.afx_pages_fork_async(s["table"], n, t["src"].data_ptr(), t["dst"].data_ptr(), 0, stream)
        afx.afx_pages_extend_async(s["table"], s["data"], n, t["dst"].data_ptr(), t["starts"].data_ptr(),
                                   n * case["new"], s["slots"].data_ptr(), s["pos"].data_ptr(),
                                   s["granted"].data_ptr(), s["ws"].data_ptr(), s["ws"].numel(), stream)
        return {"table": t["table"], "len": t["len"], "refs": t["refs"], "data": t["data"], "slots": s["slots"],
                "pos": s["pos"], "granted": s["granted"]}
    for k, v in s["was"].items():
        t[k].copy_(v)
    afx.afx_pages_compact_async(s["table"], s["data"], s["map"].data_ptr(), s["live"].data_ptr(),
                                s["ws"].data_ptr(), s["ws"].numel(), stream)
    return {"table": t["table"], "refs": t["refs"], "data": t["data"], "map": s["map"], "live": s["live"]}


def _turn(x, case, angle_cos, angle_sin, back=False):
    """Heads x [m, heads, dim] turned by their angles [m, pairs]."""
    rot, y = case["rot"], x.clone()
    if case["pairing"] == "halves":
        a, b = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        a, b = slice(0, rot, 2), slice(1, rot, 2)
    c, s = angle_cos[:, None], angle_sin[:, None] * (-1 if back else 1)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def _run_plain(s):
    case, t = s["case"], s["t"]
    op = case["op"]
    if op in ("heads", "heads_bwd"):
        m, d = case["m"], case["dim"]
        angle = t["pos"].double()[t["axis"].long()].t() * t["freq"].double()  # far positions: 64 bits
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        out = {}
        for name in ("q", "k"):
            x, w = t[name].view(m, -1, d), t["w_" + name]
            k = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
            if op == "heads":
                out[name] = _turn(x if w is None else x * k * w.float(), case, cos, sin).bfloat16()
                continue
            dn, dw = _turn(t["d" + name].float().view(m, -1, d), case, cos, sin, back=True), None
            if w is not None:
                n = x * k
                dw = (dn * n).sum((0, 1))
                dn = dn * w.float()
                dn = (dn - n * (dn * n).mean(-1, keepdim=True)) * k
            out["d" + name], out["dw_" + name] = dn.reshape(m, -1).bfloat16(), dw
        if op == "heads_bwd":
            return out
        page, off = t["slots"].long() // case["page"], t["slots"].long() % case["page"]
        t["k_pages"][page, :, :, off] = out["k"].view(m, -1, d // 8, 8)
        t["v_pages"][page, :, off // 8, :, off % 8] = t["v"].view(m, -1, d).bfloat16()
        return {"q": out["q"].reshape(m, -1), "k_pages": t["k_pages"], "v_pages": t["v_pages"]}
    if op == "attend":
        h, d, group = case["kv_heads"], case["dim"], case["q_heads"] // case["kv_heads"]
        q, out, lse = t["q"], [], []
        at = 0
        for i, (length, n) in enumerate(_fresh(case)):
            if n == 0:
                continue
            pages = t["table"][i, :_up(length, case["page"])].long()
            k = t["k_pages"][pages].permute(1, 0, 3, 2, 4).reshape(h, -1, d)[:, :length].float()
            v = t["v_pages"][pages].permute(1, 0, 2, 4, 3).reshape(h, -1, d)[:, :length].float()
            x = q[at:at + n].float().view(n, h, group, d).permute(1, 2, 0, 3).reshape(h, group * n, d)
            at += n
            score = torch.matmul(x, k.transpose(1, 2)).view(h, group, n, length) * d ** -0.5
            p, j = torch.arange(length - n, length, device=DEV)[:, None], torch.arange(length, device=DEV)[None]
            seen = j <= p
            if case["window"]:
                seen = seen & (j > p - case["window"])
            score = torch.where(seen, score, -math.inf)
            top = score.amax(-1, keepdim=True)
            e = torch.exp(score - top)
            total = e.sum(-1, keepdim=True)
            o = torch.matmul(e.view(h, group * n, length), v).view(h, group, n, d) / total
            out.append(o.permute(2, 0, 1, 3).reshape(n, -1).bfloat16())
            lse.append((top + torch.log(total))[..., 0].permute(2, 0, 1).reshape(n, -1))
        return {"out": torch.cat(out), "lse": torch.cat(lse)}
    page, table, length, refs, data = case["page"], t["table"], t["len"], t["refs"], t["data"]
    if op == "compact":
        for k, v in s["was"].items():
            t[k].copy_(v)
        live = refs > 0
        n = int(live.sum())
        holes, movers = (~live[:n]).nonzero()[:, 0], live[n:].nonzero()[:, 0] + n
        moved = torch.where(live, torch.arange(len(refs), device=DEV), -1)
        moved[movers] = holes
        data[:, holes] = data[:, movers]
        refs[holes] = refs[movers]
        refs[movers] = 0
        table.copy_(torch.where(table >= 0, moved[table.long().clamp(min=0)].int(), -1))
        return {"table": table, "refs": refs, "data": data, "map": moved.int(),
                "live": torch.full((1,), n, dtype=torch.int32, device=DEV)}
    src, dst, new, rows = t["src"].long(), t["dst"].long(), case["new"], case["branches"]
    # the old branches go
    old = table[dst]
    refs.index_add_(0, old[old >= 0].long(), torch.full_like(old[old >= 0], -1))
    # the new ones share their parents' pages
    table[dst] = table[src]
    length[dst] = length[src]
    taken = table[dst]
    refs.index_add_(0, taken[taken >= 0].long(), torch.ones_like(taken[taken >= 0]))
    # and grow, in their order: a shared page that is partly filled is copied for all but its last holder
    had = length[dst].long()
    last = table[dst, (had - 1).clamp(min=0) // page].long()
    partly = had % page > 0
    row = torch.arange(rows, device=DEV)
    before = ((last[:, None] == last[None]) & partly[:, None] & partly[None] & (row[None] < row[:, None])).sum(1)
    copied = partly & (refs[last.clamp(min=0)] - before > 1)
    need = (had + new + page - 1) // page - (had + page - 1) // page + copied
    free = (refs == 0).nonzero()[:, 0]
    fits = need.cumsum(0) <= len(free)
    need = torch.where(fits, need, 0)
    copied = copied & fits
    of = torch.repeat_interleave(row, need)
    nth = torch.arange(len(of), device=DEV) - (need.cumsum(0) - need)[of]
    ids = free[:len(of)]
    table[dst[of], (had + page - 1)[of] // page - copied[of].long() + nth] = ids.int()
    refs[ids] = 1
    refs.index_add_(0, last[copied], torch.full_like(last[copied], -1, dtype=torch.int32))
    data[:, ids[(nth == 0) & copied[of]]] = data[:, last[copied]]
    length[dst] = (had + new * fits).int()
    pos = (had[:, None] + torch.arange(new, device=DEV)[None]).reshape(-1)
    at = torch.repeat_interleave(row, new)
    slots = table[dst[at], (pos // page).clamp(max=table.shape[1] - 1)] * page + pos % page
    return {"table": table, "len": length, "refs": refs, "data": data,
            "slots": torch.where(fits[at], slots, -1).int(), "pos": torch.where(fits[at], pos, 0).int(),
            "granted": (new * fits).int()}


# ---------------------------------------------------------------------------
# the definition in 64 bits, and the work of a pass
# ---------------------------------------------------------------------------
def exact(case, seed):
    """From the formulas, gradients taken by torch's autograd of the forward
    formula in 64 bits, rotations as products of complex numbers, attention
    a head at a time. (Pages hold no computed numbers.)"""
    op = case["op"]
    if op in ("branch", "compact"):
        return None
    t = _inputs(case, seed)
    d = case["dim"]
    if op == "attend":
        h, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
        q = t["q"].double().view(-1, h, group, d)
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:3], dtype=torch.float64, device=DEV)
        starts, table, page = t["starts"].tolist(), t["table"].tolist(), case["page"]
        for i, (length, n) in enumerate(_fresh(case)):
            if n == 0:
                continue
            ids = torch.tensor(table[i][:_up(length, page)], device=DEV)
            at = slice(starts[i], starts[i] + n)
            far = torch.arange(length, device=DEV)[None] - torch.arange(length - n, length, device=DEV)[:, None]
            hidden = (far > 0) | (far <= -case["window"]) if case["window"] else far > 0
            for g in range(h):
                k = t["k_pages"][ids, g].transpose(1, 2).reshape(-1, d)[:length].double()
                v = t["v_pages"][ids, g].transpose(2, 3).reshape(-1, d)[:length].double()
                for a in range(group):
                    score = (q[at, g, a] @ k.t()).div_(math.sqrt(d)).masked_fill_(hidden, -math.inf)
                    lse[at, g, a] = torch.logsumexp(score, -1)
                    out[at, g, a] = torch.exp(score - lse[at, g, a][:, None]) @ v
        return {"out": out.flatten(1), "lse": lse.flatten(1)}
    m, rot = case["m"], case["rot"]
    angle = torch.stack([t["pos"][a].double() for a in t["axis"].tolist()], 1) * t["freq"].double()[None]
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def heads(x, w):
        x = x.view(m, -1, d)
        if w is not None:
            x = x / (x.square().sum(-1, keepdim=True) / d + EPS).sqrt() * w
        if case["pairing"] == "halves":
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            y = torch.cat((z.real, z.imag, x[..., rot:]), -1)
        else:
            z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn
            y = torch.cat((torch.view_as_real(z).flatten(-2), x[..., rot:]), -1)
        return y

    if op == "heads":
        q, k = (heads(t[n].double(), None if t["w_" + n] is None else t["w_" + n].double()) for n in "qk")
        k_pages, v_pages = t["k_pages"].double(), t["v_pages"].double()
        v = t["v"].double().view(m, -1, d)
        slots = t["slots"].long()
        ids, off = slots // case["page"], slots % case["page"]
        for c in range(0, d // 8):
            k_pages[ids, :, c, off] = k[..., 8 * c:8 * c + 8]
        for e in range(8):
            here = off % 8 == e
            v_pages[ids[here], :, off[here] // 8, :, e] = v[here]
        return {"q": q.reshape(m, -1), "k_pages": k_pages, "v_pages": v_pages}
    out = {}
    for n in "qk":
        x = t[n].double().requires_grad_()
        w = None if t["w_" + n] is None else t["w_" + n].double().requires_grad_()
        got = torch.autograd.grad(heads(x, w), [x] if w is None else [x, w], t["d" + n].double().view(m, -1, d))
        out["d" + n], out["dw_" + n] = got[0], None if w is None else got[1]
    return out


def work(case):
    op = case["op"]
    if op in ("heads", "heads_bwd"):
        m, d, q, kv = case["m"], case["dim"], case["q_heads"], case["kv_heads"]
        extra = 4 * case["axes"] * m + 5 * case["rot"] // 2 + (4 * d if case["norm"] else 0)
        if op == "heads":
            return {"bytes": m * d * (q + 2 * kv) * (4 + 2) + 4 * m + extra, "flops": 8.0 * m * d * (q + kv)}
        return {"bytes": m * d * (q + kv) * (4 + 2 + 2) + extra + (8 * d if case["norm"] else 0),
                "flops": 15.0 * m * d * (q + kv)}
    if op == "attend":
        d, tokens, pairs, new = case["dim"], 0, 0, 0
        for length, n in _fresh(case):
            new += n
            if n == 0:
                continue
            first = max(0, length - n + 1 - case["window"]) if case["window"] else 0
            tokens += length - first
            pairs += sum(min(p + 1, case["window"] or p + 1) for p in range(length - n, length))
        return {"bytes": 4 * d * case["kv_heads"] * tokens + new * case["q_heads"] * (4 * d + 4),
                "flops": 4.0 * d * case["q_heads"] * pairs}
    size = 2 * case["page"] * case["kv_heads"] * case["dim"] * case["planes"]
    if op == "compact":
        need = [_up(v, case["page"]) for v in _lengths(case["seqs"], case["len"], True)]
        live, n_pages = sum(need[::2]), sum(need) + 5
        moved = live * (1 - live / n_pages)  # live pages behind the first `live` places, about
        return {"bytes": 2 * size * moved + 8 * n_pages + 8 * len(need) * max(need), "flops": 0.0}
    # nearly every branch copies its parent's last page; its table is read and written
    wide = _up(case["len"], case["page"])
    return {"bytes": case["branches"] * (2 * size + 16 * wide), "flops": 0.0}
