"""Rows of 4-bit pools over their whole range: every scale byte read, rows that a
second pass leaves bit for bit, and head-major pages copied whole."""
import numpy as np
import pytest
import torch

import scatter_kvx_gather_amd as kvx
from tests import fp4_ref as f4
from tests.gpu_util import say
from tests.serve_util import DEV, ints, offsets
from tests.test_gpu_fp4 import BITS, TORCH

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("to", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 0.03, 2.0 ** 40, 2.0 ** -40])
def test_read_every_scale_byte(to, scale):
    """All sixteen numbers under every scale byte, whoever wrote it: the value in 32
    bits (past its range an infinity), times the scale in 32 bits, rounded once."""
    say("read every scale byte", to, scale)
    H, D, page, P = 2, 32, 16, 16
    raw = np.zeros((2, P, page * f4.row_bytes(H, D)), np.uint8)
    codes = np.tile(np.arange(16, dtype=np.uint8), (256, H, 2))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None, None], H, 1)
    for j in range(2):
        n, s = f4.views(raw[j], page, H, D, "nhd")
        n[:] = f4.pack(codes).reshape(n.shape)
        s[:] = scales.reshape(s.shape)
    store = torch.from_numpy(raw).to(DEV)
    out = torch.zeros(2, 256, H, D, dtype=TORCH[to], device=DEV)
    kvx.read(kvx.Layout(1, 2, H, D, "fp4"), 0, kvx.Pool(store, P, page, slot_stride=f4.row_bytes(H, D)),
             torch.arange(256, device=DEV), out[0], out[1], k_scale=scale, v_scale=scale)
    with np.errstate(over="ignore"):
        exp = torch.from_numpy(f4.values(codes, scales).astype(np.float32) * np.float32(scale)).to(TORCH[to])
    for got in out.cpu():
        nan = exp.isnan()
        assert torch.equal(got.isnan(), nan)
        same = got.view(BITS[to]) == exp.view(BITS[to])
        off = sorted({int(x) for x in torch.nonzero(~same & ~nan)[:, 0]})
        assert not off, f"scale bytes {off}"


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_a_second_pass_leaves_every_byte(dtype, layout):
    """A block's largest held number is 4 or 6 steps of its power of two (its largest
    value is more than 3.5 of them), unless that is the least one: what is read
    back takes the same power and the same numbers."""
    say("append, read, append, bytes", dtype, layout)
    rng = np.random.default_rng(4)
    T, H, D, page, P = 50, 4, 128, 16, 8
    lay = kvx.Layout(1, 2, H, D, "fp4")
    store = torch.zeros(2, P, page * lay.row_bytes, dtype=torch.uint8, device=DEV)
    pool = kvx.Pool(store, P, page, slot_stride=lay.row_bytes)
    x = (rng.standard_normal((2, T, H, D)) * 2.0 ** rng.integers(-30, 20, (2, T, H, 1))).astype(np.float32)
    x[0, 3, 1, 40], x[1, 4, 2, 5], x[1, 7, 0, 100] = np.inf, np.nan, -0.0
    x[0, 9], x[1, 9, 0, :32] = 0.0, 3.5
    slots = ints(rng.permutation(P * page)[:T], torch.int64)
    dev = torch.from_numpy(x).to(DEV)
    kvx.append(lay, 0, pool, slots, dev[0], dev[1], block_layout=layout)
    before = store.clone()
    back = torch.zeros(2, T, H, D, dtype=TORCH[dtype], device=DEV)
    kvx.read(lay, 0, pool, slots, back[0], back[1], block_layout=layout)
    kvx.append(lay, 0, pool, slots, back[0], back[1], block_layout=layout)
    assert before.any() and torch.equal(store, before)


def test_head_major_pages_are_copied_whole():
    """Requests that fill their pages, between pools of one page size: numbers and
    scales of head-major blocks arrive as they were."""
    say("copies of head-major 4-bit pages")
    rng = np.random.default_rng(9)
    L, H, D, page, need = 2, 3, 96, 16, [2, 0, 3]
    lay = kvx.Layout(L, 2, H, D, "fp4")
    R, Q, n = lay.row_bytes, 2 * L, sum(need)
    off = ints(offsets(need), torch.int64)
    reqs = kvx.Requests(ints(offsets([page * x for x in need]), torch.int64), page * n)

    def side(pages):
        ids = rng.permutation(pages)[:n]
        raw = rng.integers(0, 256, (Q, pages, page * R), dtype=np.uint8)
        store = torch.from_numpy(raw).to(DEV)
        return raw, ids, store, kvx.Pool(store, pages, page, slot_stride=R), kvx.Table(off, ints(ids, torch.int32))

    src, dst, third = side(9), side(12), side(7)
    kvx.gather_scatter(lay, src[3], src[4], reqs, dst[3], dst[4])
    staging = torch.zeros(page * n * Q * R, dtype=torch.uint8, device=DEV)
    kvx.gather(lay, src[3], src[4], reqs, staging)
    kvx.scatter(lay, staging, reqs, third[3], third[4])
    for raw, ids, store, *_ in (dst, third):
        raw[:, ids] = src[0][:, src[1]]
        assert np.array_equal(store.cpu().numpy(), raw)
        for layer in range(L):
            for a, b in zip(f4.views(raw[layer], page, H, D, "hnd"), f4.views(src[0][layer], page, H, D, "hnd")):
                assert np.array_equal(a[ids], b[src[1]])
