"""Seeded attention batches over 4-bit pools on the device."""
from __future__ import annotations

import numpy as np
import torch

import scatter_kvx_gather_amd as kvx
from tests import fp4_ref as f4
from tests.serve_util import DEV, Case, ints


def room_for_large(H, D, page):
    """Page ids whose 4-bit rows are 256 MiB: a table with so many counts as a
    large batch's, whatever its requests use."""
    return int((256 << 20) / (2 * H * D * 17 / 32 * page)) + 1


class Fp4Case(Case):
    """A Case whose pool holds 4 bits: `codes` and `scales` are [rows, H, D] and
    [rows, H, D / 32] for K and V, and kv the values that they stand for.  Rows that
    no list holds a token in are blocks of NaN.  `roomy`: the table has room for many
    more pages, as a step that is captured for larger batches has."""

    roomy = False

    def __init__(self, *args, spread=3, **kw):
        self.codes = None
        kw.setdefault("poison", True)
        super().__init__(*args, **kw)
        rng = np.random.default_rng(kw.get("seed", args[0] if args else 0) + 77)
        self.pool_type = "fp4"
        self.codes, self.scales, dead = [], [], []
        for x in self.kv:
            x = x.float().numpy()
            dead.append(np.isnan(x).any(-1).any(-1))
            # blocks of several sizes
            x = x * np.repeat(2.0 ** rng.integers(-spread, spread + 1, (*x.shape[:2], self.D // 32)), 32, -1)
            c, s = f4.quantise(x.astype(np.float32))
            self.codes.append(c)
            self.scales.append(s)
        for c, s, d in zip(self.codes, self.scales, dead):
            c[d] = rng.integers(0, 16, c[d].shape)
            s[d] = f4.NAN_SCALE
        self.decode()
        self.upload()

    def decode(self):
        self.kv = [torch.from_numpy(f4.values(c, s)) for c, s in zip(self.codes, self.scales)]

    def upload(self):
        if self.codes is None:
            self.pool = self.store = None
            return super().upload()
        P, B, H, D, Q = self.num_pages, self.page, self.H, self.D, 2 * self.layers
        R = f4.row_bytes(H, D)
        # padding and other layers' rows: scales of 255
        raw = np.full((Q, P, B * R), 255, np.uint8)
        for j in range(2):
            n, s = f4.views(raw[2 * self.layer + j], B, H, D, self.layout)
            n[:] = f4.pack(self.codes[j]).reshape(P, B, H, D // 2)
            s[:] = self.scales[j].reshape(P, B, H, D // 32)
        raw = torch.from_numpy(raw)
        if self.joint:
            self.store = raw.transpose(0, 1).contiguous().to(DEV)
            base = self.store.data_ptr()
            pool = kvx.Pool([base + q * B * R for q in range(Q)], P, B, slot_stride=R,
                            page_stride=Q * B * R, keep=self.store)
        else:
            self.store = raw.to(DEV)
            pool = kvx.Pool(self.store, P, B, slot_stride=R)
        store = self.store
        kv, self.kv = self.kv, [torch.zeros(P * B, H, D, dtype=torch.float16) for _ in range(2)]
        codes, self.codes = self.codes, None
        joint, self.joint, layout, self.layout = self.joint, False, self.layout, "nhd"
        kind, self.pool_type = self.pool_type, "f16"
        super().upload()                # tables, queries and offsets as they are there
        self.kv, self.codes, self.joint, self.layout, self.pool_type = kv, codes, joint, layout, kind
        self.store, self.pool = store, pool
        self.lay = kvx.Layout(self.layers, 2, H, D, "fp4")
        if self.roomy:
            ids = np.concatenate([self.b.ids, np.full(room_for_large(H, D, B), -1)])
            self.table = kvx.Table(ints(self.b.pg_off, torch.int64), ints(ids, torch.int32))
