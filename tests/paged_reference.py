"""What the calls on a paged cache should give, in 64 bits or whole numbers,
on the CPU, from their definitions in include/afx.h."""
import math

import torch

U = 2.0 ** -24  # half a step of FP32


def k_to_pages(k, pages, off, cache):
    """Keys [m, heads, dim] to their pages of cache [pages, heads, dim / 8, size, 8]."""
    cache[pages, :, :, off] = k.reshape(k.shape[0], k.shape[1], k.shape[2] // 8, 8)


def v_to_pages(v, pages, off, cache):
    """Values [m, heads, dim] to their pages of cache [pages, heads, size / 8, dim, 8]."""
    cache[pages, :, off // 8, :, off % 8] = v


def attend(q, k, v, p, lo, hi, scale):
    """One sequence and key-value head: queries q [n, dim] that see positions
    lo[i] .. hi[i] - 1 of k and v [tokens, dim], p the tokens that are there
    (bool). Returns out, lse, and bounds of their errors:

    A score is a sum of dim exact products in FP32 (dim + 2 roundings with the
    scale), its power of two has an argument rounded once or twice and 2^-22 of
    its own, and is formed again where the running maximum moves (at most 16
    times here) or parts are joined: e bounds its relative error. The weights
    are rounded to BF16 (2^-8 of each), sums over n tokens in FP32, the output
    to BF16."""
    q, k, v = q.double(), k.double(), v.double()
    j = torch.arange(k.shape[0])[None]
    seen = (j >= lo[:, None]) & (j < hi[:, None]) & p[None]
    # (what is not seen takes no part, whatever it holds)
    score = torch.zeros(q.shape[0], k.shape[0], dtype=torch.float64)
    size = torch.zeros_like(score)
    for i in range(q.shape[0]):
        score[i, seen[i]] = scale * (k[seen[i]] @ q[i])
        size[i, seen[i]] = abs(scale) * (k[seen[i]].abs() @ q[i].abs())
    score[~seen] = -math.inf
    lse = torch.logsumexp(score, -1)
    out, spread = torch.zeros(q.shape[0], v.shape[1], dtype=torch.float64), None
    spread = torch.zeros_like(out)
    for i in range(q.shape[0]):
        if not bool(seen[i].any()) or lse[i] == -math.inf:
            continue
        w = torch.exp(score[i, seen[i]] - lse[i])
        out[i] = w @ v[seen[i]]
        spread[i] = w @ v[seen[i]].abs()
    known = torch.where(torch.isfinite(score), score.abs(), 0.0)
    size = torch.where(torch.isfinite(score), size, 0.0)  # (an infinite score has no error)
    e = ((q.shape[1] + 2) * U * size + 4 * U * known).amax(-1) + 20 * 2.0 ** -22
    n = k.shape[0] + 64
    bound = (2.0 ** -8 + 2 * e[:, None] + 2 * n * U) * 1.02 * spread + 2.0 ** -8 * out.abs() + 1e-30
    return out, lse, bound, e + 2 * n * U + 8 * U * lse.abs().nan_to_num(0, 0, 0)


class Pages:
    """The page calls' state and rules on lists of whole numbers."""

    def __init__(self, n_seqs, max_pages, n_pages, size):
        self.table = [[-1] * max_pages for _ in range(n_seqs)]
        self.len, self.refs, self.size = [0] * n_seqs, [0] * n_pages, size
        self.copies = []  # (from, to) in their order

    def up(self, tokens):
        return -(-tokens // self.size)

    def ok(self, s):
        return 0 <= s < len(self.len)

    def fork(self, src, dst):
        granted = []
        for r, (s, d) in enumerate(zip(src, dst)):
            good = self.ok(s) and self.ok(d) and d not in dst[:r] and s not in dst and self.len[d] == 0
            granted.append(int(good))
            if good:
                self.len[d] = self.len[s]
                for i in range(self.up(self.len[s])):
                    self.table[d][i] = self.table[s][i]
                    self.refs[self.table[s][i]] += 1
        return granted

    def trim(self, seqs, lens=None):
        for r, s in enumerate(seqs):
            if not self.ok(s) or s in seqs[:r]:
                continue
            keep = max(0, lens[r]) if lens is not None else 0
            if keep >= self.len[s]:
                continue
            for i in range(self.up(keep), self.up(self.len[s])):
                self.refs[self.table[s][i]] -= 1
                self.table[s][i] = -1
            self.len[s] = keep

    def extend(self, seqs, starts, m):
        slots, pos, granted = [-1] * m, [0] * m, []
        free = [i for i, c in enumerate(self.refs) if c == 0]
        full = False
        for r, s in enumerate(seqs):
            n = starts[r + 1] - starts[r]
            if not self.ok(s) or s in seqs[:r] or self.len[s] + n > len(self.table[s]) * self.size:
                granted.append(0)
                continue
            had = self.len[s]
            last = self.table[s][had // self.size] if had % self.size and n else -1
            copy = last >= 0 and self.refs[last] > 1
            need = self.up(had + n) - self.up(had) + copy
            full = full or need > len(free)
            if full:
                granted.append(0)
                continue
            ids, free = free[:need], free[need:]
            if copy:
                self.refs[last] -= 1
                self.copies.append((last, ids[0]))
            for i, page in enumerate(ids):
                self.table[s][self.up(had) - copy + i] = page
                self.refs[page] = 1
            self.len[s] = had + n
            for i in range(n):
                slots[starts[r] + i] = self.table[s][(had + i) // self.size] * self.size + (had + i) % self.size
                pos[starts[r] + i] = had + i
            granted.append(n)
        return slots, pos, granted

    def compact(self):
        live = sum(c > 0 for c in self.refs)
        holes = [i for i in range(live) if self.refs[i] == 0]
        movers = [i for i in range(live, len(self.refs)) if self.refs[i] > 0]
        moved = [i if c > 0 else -1 for i, c in enumerate(self.refs)]
        for a, b in zip(movers, holes):
            moved[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
            self.copies.append((a, b))
        self.table = [[moved[e] if e >= 0 else -1 for e in row] for row in self.table]
        return moved, live
