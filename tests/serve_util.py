"""Seeded attention batches on the device for the serving tests."""
from __future__ import annotations

import numpy as np
import torch

import scatter_kvx_gather_amd as kvx
from tests import serve_ref as ref

DEV = torch.device("cuda:0")
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.float8_e4m3fn}


def ints(x, dtype):
    return torch.tensor(np.ascontiguousarray(x), dtype=dtype, device=DEV)


def offsets(counts):
    return np.concatenate([[0], np.cumsum(np.asarray(counts, dtype=np.int64))]).astype(np.int64)


class Case:
    """A batch with its pool.  `values` keeps K and V as [rows, heads, dim] in
    the order of the flat rows, whatever the blocks' layout."""

    def __init__(self, seed, new, ctx, H, G, D, dtype="bf16", pool="", page=16, layout="nhd",
                 members=None, prefix=None, bad=0.0, amp=1.0, layers=1, layer=0, joint=False,
                 k_scale=1.0, v_scale=1.0, extra_pages=5, poison=True):
        rng = np.random.default_rng(seed)
        pool = pool or dtype
        self.dtype, self.pool_type, self.layout, self.layer = dtype, pool, layout, layer
        self.H, self.G, self.D, self.page = H, G, D, page
        self.k_scale, self.v_scale = k_scale, v_scale
        npg = [-(-c // page) for c in ctx]
        ppg = [-(-p // page) for p in (prefix or [])]
        total = sum(npg) + sum(ppg)
        self.num_pages = total + extra_pages
        perm = rng.permutation(self.num_pages).astype(np.int32)
        ids, pre_ids = perm[:sum(npg)].copy(), perm[sum(npg):total].copy()
        for a in (ids, pre_ids):
            if bad and a.size:
                m = rng.random(a.size) < bad
                a[m] = rng.choice([-1, -7, self.num_pages, 2**31 - 1], m.sum())
        self.b = ref.Batch(page, self.num_pages, list(new), list(ctx), offsets(npg), ids, members,
                           prefix, offsets(ppg), pre_ids)
        T, rows = sum(new), self.num_pages * page
        g = torch.Generator().manual_seed(seed)
        t = TORCH[dtype]
        self.q = (torch.randn(T, H * G, D, generator=g) * amp).to(t)
        kv = [torch.randn(rows, H, D, generator=g) for _ in range(2)]
        if pool == "fp8":
            kv = [(x / s).clamp(-448, 448).to(TORCH["fp8"]) for x, s in zip(kv, (k_scale, v_scale))]
        else:
            kv = [x.to(t) for x in kv]
        self.kv = kv
        # rows that no list holds a token in are NaN: nothing may come of them
        if poison:
            used = np.zeros(rows, bool)
            for r, c in enumerate(ctx):
                used[[x for x in self.b.rows(self.b.pg_off[r], ids, c) if x is not None]] = True
            for i, p in enumerate(prefix or []):
                used[[x for x in self.b.rows(self.b.pre_off[i], pre_ids, p) if x is not None]] = True
            for x in kv:
                x.view(torch.uint8 if pool == "fp8" else torch.int16)[torch.from_numpy(~used)] = \
                    0x7f if pool == "fp8" else 0x7fff if dtype == "bf16" else 0x7e00
        self.layers, self.joint = layers, joint
        self.upload()

    def upload(self):
        """The pool on the device: [layers][2][pages] blocks, or (joint) one
        [pages][layers][2] tensor of blocks."""
        es = self.kv[0].element_size()
        P, B, H, D, Q = self.num_pages, self.page, self.H, self.D, 2 * self.layers
        raw = torch.zeros(Q, P, B, H, D * es, dtype=torch.uint8)
        for j in range(2):
            raw[2 * self.layer + j] = self.kv[j].view(P, B, H, D).view(torch.uint8)
        if self.layout == "hnd":
            raw = raw.transpose(2, 3).contiguous()
        R = H * D * es
        if self.joint:
            self.store = raw.view(Q, P, -1).transpose(0, 1).contiguous().to(DEV)
            base = self.store.data_ptr()
            self.pool = kvx.Pool([base + q * B * R for q in range(Q)], P, B, slot_stride=R,
                                 page_stride=Q * B * R, keep=self.store)
        else:
            self.store = raw.to(DEV)
            self.pool = kvx.Pool(self.store, P, B, slot_stride=R)
        self.lay = kvx.Layout(self.layers, 2, H, D, self.pool_type)
        b = self.b
        self.qd = self.q.to(DEV)
        self.tok_off = ints(offsets(b.new), torch.int64)
        self.reqs = kvx.Requests(self.tok_off, sum(b.new))
        self.ctx = ints(b.ctx, torch.int32)
        self.table = kvx.Table(ints(b.pg_off, torch.int64), ints(b.ids, torch.int32))
        self.prefix = None
        if b.members is not None:
            self.prefix = kvx.Prefix(ints(b.members, torch.int64), ints(b.prefix, torch.int32),
                                     kvx.Table(ints(b.pre_off, torch.int64),
                                               ints(b.pre_ids, torch.int32)))

    def run(self, out=None, lse=None, q=None, **kw):
        q = self.qd if q is None else q
        out = torch.full_like(self.qd, float("nan")) if out is None else out
        lse = torch.full(self.q.shape[:2], float("nan"), device=DEV) if lse is None else lse
        kvx.attend(self.lay, self.layer, self.pool, self.reqs, self.ctx, self.table, q, out,
                   prefix=self.prefix, lse=lse, k_scale=self.k_scale, v_scale=self.v_scale,
                   block_layout=self.layout, **kw)
        return out, lse

    def expected(self, scale=None, causal=True):
        k, v = (x.double().numpy() * s for x, s in zip(self.kv, (self.k_scale, self.v_scale)))
        scale = self.D ** -0.5 if scale is None else scale
        return ref.attend(self.b, self.q.double().numpy(), k, v, scale, causal)

    def check(self, out, lse, scale=None, causal=True):
        eo, el, mass, size, seen = self.expected(scale, causal)
        fin = self.kv[1].double().numpy()
        vmax = np.abs(fin[np.isfinite(fin)]).max() * self.v_scale if np.isfinite(fin).any() else 1.0
        tol, tol_lse = ref.bounds(self.dtype, self.D, eo, el, mass, size, seen, vmax)
        go, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        ok = np.isfinite(eo)
        assert np.array_equal(np.isfinite(go), ok), "finite values differ"
        assert np.array_equal(go[~ok & ~np.isnan(eo)], eo[~ok & ~np.isnan(eo)])
        off = np.abs(go[ok] - eo[ok])
        bad = off > tol[ok]
        assert not bad.any(), \
            f"{bad.sum()} of {bad.size} values off, worst {off.max():.3g}, " \
            f"{(off / tol[ok]).max():.3g} times the bound"
        okl = np.isfinite(el)
        assert np.array_equal(gl[~okl & ~np.isnan(el)], el[~okl & ~np.isnan(el)])
        offl = np.abs(gl[okl] - el[okl])
        assert not (offl > tol_lse[okl]).any(), f"lse: {offl.max():.3g}"
