"""Plain 64-bit forms of the serving step (tables from lengths, appended rows,
attention with shared prefixes) and seeded inputs for its tests.  Everything
here is numpy on the host and knows nothing of the library; values that a type
rounds are passed in as the values they stand for."""
from __future__ import annotations

import dataclasses
import math
from typing import List, Optional

import numpy as np


def build_tables(page, have, add, held_lists, free, clamp=2**31 - 1):
    """ctx, tok_off, pg_off, ids, slots, totals by walking the requests."""
    ctx, tok_off, pg_off, ids, slots = [], [0], [0], [], []
    used = 0
    for r, a in enumerate(add):
        h = max(int(have[r]), 0) if have is not None else 0
        a = min(max(int(a), 0), clamp - h)
        keep = -(-h // page)
        mine = [int(held_lists[r][k]) if k < len(held_lists[r]) else -1 for k in range(keep)] \
            if have is not None else []
        while len(mine) < -(-(h + a) // page):
            mine.append(int(free[used]) if used < len(free) else -1)
            used += 1
        for t in range(h, h + a):
            p = mine[t // page]
            slots.append(-1 if p < 0 else p * page + t % page)
        ids += mine
        ctx.append(h + a)
        tok_off.append(len(slots))
        pg_off.append(len(ids))
    return dict(ctx=ctx, tok_off=tok_off, pg_off=pg_off, ids=ids, slots=slots,
                totals=[len(slots), len(ids), used, max(0, used - len(free))])


@dataclasses.dataclass
class Batch:
    """An attention batch: rows of K and V are read through lookup(list, t),
    which gives the flat row of token t or None where its page is out of range."""
    page: int
    num_pages: int
    new: List[int]                      # query tokens per request
    ctx: List[int]                      # own context per request
    pg_off: np.ndarray
    ids: np.ndarray
    members: Optional[List[int]] = None  # group boundaries over the requests
    prefix: Optional[List[int]] = None
    pre_off: Optional[np.ndarray] = None
    pre_ids: Optional[np.ndarray] = None

    def rows(self, off, ids, n):
        out = []
        for t in range(n):
            i = int(off) + t // self.page
            p = int(ids[i]) if 0 <= i < len(ids) else -1
            out.append(p * self.page + t % self.page if 0 <= p < self.num_pages else None)
        return out

    def group_of(self, r):
        if self.members is None:
            return None
        return max(g for g in range(len(self.prefix)) if self.members[g] <= r)

    def skipped(self):
        """Out-of-range keys, once per context and once per prefix with queries."""
        n = sum(x is None for r, c in enumerate(self.ctx) if self.new[r] > 0
                for x in self.rows(self.pg_off[r], self.ids, c))
        if self.members is not None:
            for g, p in enumerate(self.prefix):
                if sum(self.new[self.members[g]:self.members[g + 1]]) > 0:
                    n += sum(x is None for x in self.rows(self.pre_off[g], self.pre_ids, p))
        return n


def attend(b: Batch, q, k, v, scale, causal=True):
    """out [T, Hq, D], lse [T, Hq] and for the error bound the weighted sums of
    |v| and the largest sum of |q_i k_i| * scale, all in 64 bits; q [T, Hq, D],
    k and v [rows, H, D]."""
    q = q.astype(np.float64)
    T, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    mass, size, seen = np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros(T, int)
    t0 = 0
    for r, n in enumerate(b.new):
        pre = []
        g = b.group_of(r)
        if g is not None:
            pre = b.rows(b.pre_off[g], b.pre_ids, b.prefix[g])
        own = b.rows(b.pg_off[r], b.ids, b.ctx[r])
        for i in range(n):
            lim = b.ctx[r] - n + i + 1 if causal else b.ctx[r]
            keys = [x for x in pre + own[:max(lim, 0)] if x is not None]
            seen[t0 + i] = len(keys)
            if not keys:
                continue
            kk, vv = k[keys].astype(np.float64), v[keys].astype(np.float64)
            kk, vv = np.repeat(kk, G, 1), np.repeat(vv, G, 1)         # [n, Hq, D]
            x = np.einsum("hd,nhd->hn", q[t0 + i], kk) * scale
            size[t0 + i] = np.einsum("hd,nhd->hn", np.abs(q[t0 + i]), np.abs(kk)).max(1) * scale
            m = x.max(1)
            with np.errstate(invalid="ignore"):
                p = np.exp(x - m[:, None])
                l = p.sum(1)
                out[t0 + i] = np.einsum("hn,nhd->hd", p, vv) / l[:, None]
                mass[t0 + i] = np.einsum("hn,nhd->hd", p, np.abs(vv)) / l[:, None]
                lse[t0 + i] = m + np.log(l)
        t0 += n
    return out, lse, mass, size, seen


HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}     # half a step, relative


def bounds(dtype, dim, out, lse, mass, size, seen, vmax):
    """Largest errors of out and lse that the arithmetic can make.

    A score is a sum of `dim` products in 32 bits: off by e = (dim + 8) 2^-24
    times the sum of |q_i k_i| scale (the 8: scale, its product with log2 e,
    the exponent's sum).  A weight is then off by e, and by 2 steps of the
    exponential; l and o sum `seen` of them (2^-24 each), and out divides the
    two, so the relative error of a weight counts twice.  For the second
    product a weight is rounded to the type (half a step of it; in f16 at
    least 2^-25, where it is subnormal, and the largest weights are at least 2^8), and out once more at the end."""
    u = HALF[dtype]
    e = (dim + 8) * 2.0 ** -24 * size + 2.0 ** -22 + (seen[:, None] + 64) * 2.0 ** -24
    tiny = seen * 2.0 ** -33 * vmax if dtype == "f16" else seen * 2.0 ** -126 * vmax
    # a result below the type's normal range is off by half its smallest step
    floor = 2.0 ** -25 if dtype == "f16" else 2.0 ** -126
    tol = u * np.abs(out) * 1.01 + (u + 2 * e[..., None]) * mass + tiny[:, None, None] + floor
    tol_lse = e + 2.0 ** -22 * (np.where(np.isfinite(lse), np.abs(lse), 0) + 4)
    return tol, tol_lse
