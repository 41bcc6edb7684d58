"""Plain 64-bit forms of the decoder-layer operators (rotary positions, paged attention, cache pages) and the bounds
their f32 / bf16 / f16 kernels are held to.  Test code only; shares nothing with the library."""
import math

import numpy as np
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
CODE = {"f32": 0, "f16": 1, "bf16": 2}
#: half the spacing of the type, relative to the value
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
#: half the spacing below the smallest normal value
TINY = {"f32": 2.0 ** -150, "f16": 2.0 ** -25, "bf16": 2.0 ** -134}


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def rotary(x, cos, sin, positions, layout, inverse=False):
    """x [T, H, D], cos and sin [n_pos, r / 2], all f64; returns (y, |a c| + |b s| of each value)."""
    y, mag = x.copy(), np.zeros_like(x)
    r = 2 * cos.shape[1]
    for i in range(r // 2):
        a, b = (i, i + r // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = cos[positions, i][:, None], sin[positions, i][:, None] * (-1 if inverse else 1)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        mag[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        mag[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, mag


def rotary_bound(y, mag, dtype):
    """Two f32 products and a sum (each rounding within 2^-24 of mag), then one rounding to dtype."""
    return 3 * 2.0 ** -24 * mag + 1.01 * ROUND[dtype] * np.abs(y) + TINY[dtype]


def attention(q, k, v, first, scale, causal, window):
    """One sequence and one head: q [n, d] at positions first .., k and v [len, d], f64.
    Returns o, lse and the bounds on their errors as a function of the type."""
    n, d = q.shape
    length = k.shape[0]
    o, lse = np.zeros((n, v.shape[1])), np.full(n, -np.inf)
    bo = {t: np.zeros_like(o) for t in DT}
    bl = np.zeros(n)
    for i in range(n):
        pos = first + i
        hi = min(length, pos + 1) if causal else length
        lo = max(0, pos - window + 1) if window else 0
        if hi <= lo:
            for t in DT:
                bo[t][i] = 0.0
            continue
        kk, vv = k[lo:hi], v[lo:hi]
        s = kk @ q[i] * scale
        m = s.max()
        p = np.exp(s - m)
        total = p.sum()
        w = p / total
        o[i] = w @ vv
        lse[i] = m + math.log(total)
        # scores: d products summed in f32 and scaled; exponent: f32 argument and a 2^-22 exponential
        score = (d + 4) * 2.0 ** -24 * (np.abs(kk) @ np.abs(q[i])).max() * abs(scale)
        delta = score + 2.0 ** -22 * (np.abs(s).max() + abs(m) + 8) + 2.0 ** -21
        spread = w @ np.abs(vv)
        for t in DT:
            # p rounded to the type for the product with V (f32: not), the sums in f32, one rounding of o
            pr = 0.0 if t == "f32" else ROUND[t]
            lost = (hi - lo) * TINY[t] * np.abs(vv).max() if t == "f16" else 0.0
            bo[t][i] = spread * (pr + 2 * delta + (hi - lo + 64) * 2.0 ** -24) + 1.01 * ROUND[t] * np.abs(o[i]) + lost + TINY[t]
        bl[i] = delta + (hi - lo + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(lse[i])
    return o, lse, bo, bl


class Pages:
    """A cache's bookkeeping and pages as plain lists: the meaning of fork, resize and compact."""

    def __init__(self, refs, tables, lens, page_size, pool):
        self.refs, self.tables, self.lens = [int(x) for x in refs], [[int(p) for p in r] for r in tables], [int(x) for x in lens]
        self.ps, self.pool = page_size, pool.copy()  # pool [planes, pages, n]

    def held(self, n):
        return -(-n // self.ps)

    def fork(self, src, dst):
        rows, lens = [list(self.tables[a]) for a in src], [self.lens[a] for a in src]
        for row, n in zip(rows, lens):
            for p in row[:self.held(n)]:
                self.refs[p] += 1
        for b in dst:
            for p in self.tables[b][:self.held(self.lens[b])]:
                self.refs[p] -= 1
        for b, row, n in zip(dst, rows, lens):
            self.tables[b] = row[:self.held(n)] + [-1] * (len(row) - self.held(n))
            self.lens[b] = n

    def resize(self, seqs, new_lens):
        """False if the pages do not suffice (nothing changes)."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        plan, need = [], 0
        for b, n in zip(seqs, new_lens):
            had, want = self.held(self.lens[b]), self.held(n)
            split = n > self.lens[b] and self.lens[b] % self.ps != 0 and self.refs[self.tables[b][had - 1]] > 1
            plan.append((b, n, had, want, split))
            need += max(0, want - had) + int(split)
        if need > len(free):
            return False
        copies, drop = [], []
        for b, n, had, want, split in plan:
            if split:
                old = self.tables[b][had - 1]
                new = free.pop(0)
                copies.append((old, new))
                drop.append(old)
                self.refs[new] = 1
                self.tables[b][had - 1] = new
            for c in range(had, want):
                p = free.pop(0)
                self.refs[p] = 1
                self.tables[b][c] = p
            for c in range(want, had):
                drop.append(self.tables[b][c])
                self.tables[b][c] = -1
            self.lens[b] = n
        for p in drop:
            self.refs[p] -= 1
        before = self.pool.copy()
        for old, new in copies:
            self.pool[:, new] = before[:, old]
        return True

    def compact(self):
        live = sum(r > 0 for r in self.refs)
        src = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] == 0]
        name = dict(zip(src, dst))
        for a, b in name.items():
            self.pool[:, b] = self.pool[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for row, n in zip(self.tables, self.lens):
            for c in range(self.held(n)):
                row[c] = name.get(row[c], row[c])
        return live, len(src)
