"""Dense rows of 64 MiB and more, which pass by the caches on their way into and
out of pools, byte for byte; and a few tokens less, which do not."""
import numpy as np
import pytest
import torch

import scatter_kvx_gather_amd as kvx
from tests import fp4_ref as f4
from tests.gpu_util import say
from tests.serve_util import DEV, ints
from tests.test_gpu_fp4 import BITS, TORCH, rows_of

pytestmark = pytest.mark.gpu

H, D, PAGE = 8, 128, 16
PAST = 1 << 26              # bytes of K and V rows together


def tokens(dtype, side):
    """The fewest odd number of tokens whose rows reach the bound, or the most below."""
    n = PAST // (2 * H * D * TORCH[dtype].itemsize)
    return n + 1 if side == "above" else n - 1


def a_pool(rng, T, R):
    """Random bytes [2, P, page * R] and distinct slots of T tokens, three of them out of range."""
    P = T // PAGE + 3
    store = torch.from_numpy(rng.integers(0, 256, (2, P, PAGE * R), dtype=np.uint8)).to(DEV)
    slots = torch.from_numpy(rng.permutation(P * PAGE)[:T]).to(DEV)
    for t, x in ((0, -1), (T // 2, P * PAGE), (T - 1, 1 << 40)):
        slots[t] = x
    return store, kvx.Pool(store, P, PAGE, slot_stride=R), slots


def views(plane, layout, numbers, scales):
    """[pages * page, H, numbers] and [.., scales] views of a plane [pages, page * R] on the device."""
    P = plane.shape[0]
    if layout == "nhd":
        rows = plane.view(P, PAGE, -1)
        return (rows[..., :H * numbers].unflatten(-1, (H, numbers)),
                rows[..., H * numbers:H * (numbers + scales)].unflatten(-1, (H, scales)))
    n = H * PAGE * numbers
    return (plane[:, :n].view(P, H, PAGE, numbers).transpose(1, 2),
            plane[:, n:n + H * PAGE * scales].view(P, H, PAGE, scales).transpose(1, 2))


def in_pool(slots, pages):
    return (slots >= 0) & (slots < pages * PAGE)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("side", ["below", "above"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("scale", [1.0, 0.03])
def test_append(dtype, side, layout, scale):
    say("append fp4, large", dtype, side, layout, scale)
    rng = np.random.default_rng(17)
    T, n = tokens(dtype, side), 301
    store, pool, slots = a_pool(rng, T, f4.row_bytes(H, D))
    P = store.shape[1]
    expected = store.clone()
    skipped = torch.zeros(1, dtype=torch.int64, device=DEV)
    rows, there = [], in_pool(slots, P)
    for j, c in enumerate((scale, 2 * scale)):
        few = rows_of(rng, n, H, D, dtype)          # each many times over
        which = torch.from_numpy(rng.integers(0, n, T)).to(DEV)
        rows.append(few.to(DEV)[which])
        codes, scales = f4.quantise(few.float().numpy(), c)
        at, pick = slots[there], which[there]
        numbers, bytes_ = views(expected[j], layout, D // 2, D // 32)
        numbers[at // PAGE, at % PAGE] = torch.from_numpy(f4.pack(codes)).to(DEV)[pick]
        bytes_[at // PAGE, at % PAGE] = torch.from_numpy(scales).to(DEV)[pick]
    kvx.append(kvx.Layout(1, 2, H, D, "fp4"), 0, pool, slots, *rows, k_scale=scale, v_scale=2 * scale,
               block_layout=layout, skipped=skipped)
    assert torch.equal(store, expected)
    assert skipped.item() == 3


@pytest.mark.parametrize("held,to", [("fp4", "bf16"), ("fp4", "f16"), ("fp4", "f32"), ("fp8", "bf16"),
                                     ("fp8", "f16"), ("fp8", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                     ("f32", "f32"), ("fp8", "fp8")])
@pytest.mark.parametrize("side", ["below", "above"])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_read(held, to, side, layout):
    say("read, large", held, to, side, layout)
    rng = np.random.default_rng(18)
    T = tokens(to, side)
    lay = kvx.Layout(1, 2, H, D, held)
    store, pool, slots = a_pool(rng, T, int(lay.row_bytes))
    P, there = store.shape[1], in_pool(slots, store.shape[1])
    scale = 1.0 if held == to else 0.03
    if held == "fp4":
        for j in range(2):
            _, s = views(store[j], layout, D // 2, D // 32)
            some = np.array([*range(104, 141), 255], np.uint8)
            s[:] = torch.from_numpy(rng.choice(some, s.shape)).to(DEV)
    out = torch.full((2, T, H, D), 3.0, device=DEV).to(TORCH[to])
    expected = out.clone()
    skipped = torch.zeros(1, dtype=torch.int64, device=DEV)
    kvx.read(lay, 0, pool, slots, out[0], out[1], k_scale=scale, v_scale=2 * scale if scale != 1 else 1.0,
             block_layout=layout, skipped=skipped)
    at = slots[there]
    grid = torch.from_numpy(np.concatenate([f4.GRID, -f4.GRID])).float().to(DEV)
    for j in range(2):
        c = torch.tensor(scale * (j + 1) if scale != 1 else 1.0, dtype=torch.float32, device=DEV)
        if held == "fp4":
            b, s = (x[at // PAGE, at % PAGE] for x in views(store[j], layout, D // 2, D // 32))
            numbers = grid[torch.stack([b & 15, b >> 4], -1).flatten(-2).int()]
            unit = torch.ldexp(torch.ones((), device=DEV), s.int() - 127)
            unit[s == 255] = float("nan")
            rows = (numbers * unit.repeat_interleave(32, -1) * c).to(TORCH[to])
        else:
            es = TORCH[held].itemsize
            b, _ = views(store[j], layout, D * es, 0)
            rows = b[at // PAGE, at % PAGE].contiguous().view(TORCH[held])
            if held != to:
                rows = (rows.float() * c).to(TORCH[to])
        expected[j].view(BITS[to])[there] = rows.view(BITS[to])
    if held == to:
        assert torch.equal(out.view(BITS[to]), expected.view(BITS[to]))
    else:
        nan = expected.isnan()
        assert torch.equal(out.isnan(), nan)
        assert torch.equal(out.view(BITS[to])[~nan], expected.view(BITS[to])[~nan])
    assert skipped.item() == 3
