"""Rows quantised into 4-bit pools and rows of pools read back, byte for byte
against plain host forms; copies of 4-bit rows; the serving step over a 4-bit
pool."""
import numpy as np
import pytest
import torch

import scatter_kvx_gather_amd as kvx
from tests import fp4_ref as f4
from tests import serve_ref as ref
from tests.gpu_util import say
from tests.serve_util import DEV, ints, offsets

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
         "fp8": torch.float8_e4m3fn}
BITS = {"bf16": torch.int16, "f16": torch.int16, "f32": torch.int32, "fp8": torch.uint8}


def rows_of(rng, T, H, D, dtype):
    """Rows of many sizes, with zeros of both signs, infinities, NaN, ties and values at both ends."""
    x = rng.standard_normal((T, H, D)) * 2.0 ** rng.integers(-30, 18, (T, H, 1))
    x = x.reshape(-1)
    n = max(1, x.size // 40)
    at = rng.integers(0, x.size, n)
    with np.errstate(all="ignore"):
        x[at] = rng.choice([0.0, -0.0, 1e-30, -1e-6, 2.0 ** -25, 6e4, -6e4, 1e30, 0.25, 7.0, -5.0, 2.5], n)
        at = rng.integers(0, x.size, max(1, n // 20))
        x[at] = rng.choice([np.inf, -np.inf, np.nan], at.size)
        t = torch.from_numpy(x.reshape(T, H, D).astype(np.float32)).to(TORCH[dtype])
    # whole blocks of zeros and of halves and quarters (ties)
    t[:: 5, 0, :32] = 0.0
    if T > 2:
        t[2, -1, -32:] = torch.arange(32).to(t.dtype) * 0.25
    return t


def pool_bytes(rng, P, B, H, D, joint=0):
    """A [2, P, B * R] pool of random bytes."""
    return rng.integers(0, 256, (2, P, B * f4.row_bytes(H, D)), dtype=np.uint8)


def put(raw, slots, page, H, D, layout, codes, scales, j):
    n, s = f4.views(raw[j], page, H, D, layout)
    for t, x in enumerate(slots):
        if 0 <= x < raw.shape[1] * page:
            n[x // page, x % page] = f4.pack(codes[t])
            s[x // page, x % page] = scales[t]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H,D,page,layout", [
    (8, 128, 16, "nhd"), (8, 128, 16, "hnd"), (1, 32, 1, "nhd"), (1, 64, 4, "hnd"), (2, 96, 3, "nhd"),
    (3, 96, 5, "hnd"), (5, 160, 7, "nhd"), (4, 256, 32, "hnd"), (1, 128, 64, "nhd"), (16, 64, 1, "hnd"),
    (40, 256, 2, "nhd")])
@pytest.mark.parametrize("scale", [1.0, 0.03])
def test_append(dtype, H, D, page, layout, scale):
    say("append fp4", dtype, H, D, page, layout, scale)
    rng = np.random.default_rng(H * 1000 + D + page)
    P = 400 // page + 2
    for T in (1, 3, 130):
        raw = pool_bytes(rng, P, page, H, D)
        slots = rng.permutation(P * page)[:T]
        if T > 2:
            slots[1] = -1
            slots[2] = P * page
        store = torch.from_numpy(raw).to(DEV)
        pool = kvx.Pool(store, P, page, slot_stride=f4.row_bytes(H, D))
        # rows of a fused buffer
        k, v = rows_of(rng, T, H, D, dtype), rows_of(rng, T, H, D, dtype)
        fused = torch.zeros(T, 3 * H, D, dtype=TORCH[dtype])
        fused[:, H:2 * H], fused[:, 2 * H:] = k, v
        fused = fused.to(DEV)
        skipped = torch.zeros(1, dtype=torch.int64, device=DEV)
        kvx.append(kvx.Layout(1, 2, H, D, "fp4"), 0, pool, ints(slots, torch.int64),
                   fused[:, H:2 * H], fused[:, 2 * H:], k_scale=scale, v_scale=scale * 2,
                   block_layout=layout, skipped=skipped)
        for j, (x, c) in enumerate(((k, scale), (v, scale * 2))):
            codes, scales = f4.quantise(x.float().numpy(), c)
            put(raw, slots, page, H, D, layout, codes, scales, j)
        got = store.cpu().numpy()
        assert np.array_equal(got, raw), f"{(got != raw).sum()} bytes of {raw.size} differ"
        assert skipped.item() == (2 if T > 2 else 0)


@pytest.mark.parametrize("to", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H,D,page,layout", [
    (8, 128, 16, "nhd"), (8, 128, 16, "hnd"), (1, 32, 1, "nhd"), (1, 64, 4, "hnd"), (2, 96, 3, "nhd"),
    (3, 96, 5, "hnd"), (5, 160, 7, "nhd"), (4, 256, 32, "hnd"), (40, 256, 2, "nhd")])
@pytest.mark.parametrize("scale", [1.0, 0.03])
def test_read(to, H, D, page, layout, scale):
    say("read fp4", to, H, D, page, layout, scale)
    rng = np.random.default_rng(H * 1000 + D + page + 1)
    P = 200 // page + 2
    raw = pool_bytes(rng, P, page, H, D)
    views = [f4.views(raw[j], page, H, D, layout) for j in range(2)]
    for n, s in views:                  # scales that the pool can hold, and NaN
        s[:] = rng.choice(np.array([*range(104, 141), 255], np.uint8), s.shape)
    store = torch.from_numpy(raw).to(DEV)
    pool = kvx.Pool(store, P, page, slot_stride=f4.row_bytes(H, D))
    for T in (1, 77):
        slots = rng.integers(0, P * page, T)        # some more than once
        if T > 2:
            slots[5], slots[9] = -1, P * page + 3
        out = torch.full((T, 3 * H, D), 3.0, dtype=TORCH[to], device=DEV)
        skipped = torch.zeros(1, dtype=torch.int64, device=DEV)
        kvx.read(kvx.Layout(1, 2, H, D, "fp4"), 0, pool, ints(slots, torch.int64), out[:, H:2 * H],
                 out[:, 2 * H:], k_scale=scale, v_scale=scale * 2, block_layout=layout, skipped=skipped)
        exp = torch.full((T, 3 * H, D), 3.0, dtype=TORCH[to])
        for j, c in enumerate((scale, scale * 2)):
            n, s = views[j]
            for t, x in enumerate(slots):
                if 0 <= x < P * page:
                    y = f4.values(f4.unpack(n[x // page, x % page]), s[x // page, x % page])
                    y = torch.from_numpy(y.astype(np.float32) * np.float32(c))
                    exp[t, (j + 1) * H:(j + 2) * H] = y.to(TORCH[to])
        got = out.cpu()
        assert torch.equal(got.isnan(), exp.isnan())
        got[got.isnan()] = 0
        exp[exp.isnan()] = 0
        assert torch.equal(got.view(BITS[to]), exp.view(BITS[to]))
        assert skipped.item() == (2 if T > 2 else 0)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32", "fp8"])
@pytest.mark.parametrize("H,D,page,layout", [(8, 128, 16, "nhd"), (2, 64, 16, "hnd"), (1, 16, 1, "nhd"),
                                             (3, 80, 5, "hnd"), (5, 80, 3, "nhd")])
def test_read_copies(kind, H, D, page, layout):
    """A pool's own type comes back bit by bit, and what append wrote."""
    say("read copies", kind, H, D, page, layout)
    es = TORCH[kind].itemsize
    rng = np.random.default_rng(D)
    P, T = 60 // page + 2, 40
    store = torch.zeros(2, P, page * H * D * es, dtype=torch.uint8, device=DEV)
    pool = kvx.Pool(store, P, page, slot_stride=H * D * es)
    kv = torch.from_numpy(rng.integers(0, 256, (2, T, H, D * es), dtype=np.uint8)).to(DEV).view(TORCH[kind])
    slots = ints(rng.permutation(P * page)[:T], torch.int64)
    lay = kvx.Layout(1, 2, H, D, kind)
    kvx.append(lay, 0, pool, slots, kv[0], kv[1], block_layout=layout)
    out = torch.zeros(2, T, H, D * es, dtype=torch.uint8, device=DEV).view(TORCH[kind])
    kvx.read(lay, 0, pool, slots, out[0], out[1], block_layout=layout)
    assert torch.equal(out.view(torch.uint8), kv.view(torch.uint8))


@pytest.mark.parametrize("to", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H,D,page,layout", [(8, 128, 16, "nhd"), (2, 64, 16, "hnd"), (1, 16, 1, "nhd"),
                                             (3, 80, 5, "hnd")])
@pytest.mark.parametrize("scale", [1.0, 0.03])
def test_read_fp8(to, H, D, page, layout, scale):
    say("read fp8", to, H, D, page, layout, scale)
    rng = np.random.default_rng(D + 5)
    P, T = 60 // page + 2, 40
    raw = torch.from_numpy(rng.integers(0, 256, (2, P, page, H, D), dtype=np.uint8))
    store = (raw.transpose(2, 3).contiguous() if layout == "hnd" else raw).to(DEV)
    pool = kvx.Pool(store, P, page, slot_stride=H * D)
    slots = rng.permutation(P * page)[:T]
    out = torch.zeros(2, T, H, D, dtype=TORCH[to], device=DEV)
    kvx.read(kvx.Layout(1, 2, H, D, "fp8"), 0, pool, ints(slots, torch.int64), out[0], out[1],
             k_scale=scale, v_scale=2 * scale, block_layout=layout)
    exp = raw.view(2, P * page, H, D)[:, slots].view(TORCH["fp8"]).float()
    exp = (exp * torch.tensor([scale, 2 * scale]).view(2, 1, 1, 1)).to(TORCH[to])
    got = out.cpu()
    assert torch.equal(got.isnan(), exp.isnan())
    assert torch.equal(got.nan_to_num(0), exp.nan_to_num(0))


def test_append_then_read_keeps_what_is_held():
    """Values that 4 bits hold come back as they were, and a second pass changes nothing."""
    say("append, read, append")
    rng = np.random.default_rng(4)
    T, H, D, page, P = 50, 4, 128, 16, 8
    lay = kvx.Layout(1, 2, H, D, "fp4")
    store = torch.zeros(2, P, page * lay.row_bytes, dtype=torch.uint8, device=DEV)
    pool = kvx.Pool(store, P, page, slot_stride=lay.row_bytes)
    x = torch.from_numpy(rng.standard_normal((2, T, H, D)).astype(np.float32)).to(DEV)
    slots = ints(rng.permutation(P * page)[:T], torch.int64)
    kvx.append(lay, 0, pool, slots, x[0], x[1])
    for dtype in (torch.float16, torch.bfloat16, torch.float32):
        back = torch.zeros(2, T, H, D, dtype=dtype, device=DEV)
        kvx.read(lay, 0, pool, slots, back[0], back[1])
        before = store.clone()
        kvx.append(lay, 0, pool, slots, back[0], back[1])
        again = torch.zeros_like(back)
        kvx.read(lay, 0, pool, slots, again[0], again[1])
        assert torch.equal(back, again)
        top = before.view(2, P * page, -1)
        assert top.shape == store.view(2, P * page, -1).shape
    # each value is off by at most the step between its neighbours
    off = (back.float() - x).abs().view(2, T, H, -1, 32)
    most = x.abs().view(2, T, H, -1, 32).amax(-1, keepdim=True)
    assert (off <= most / 3.5).all()


@pytest.mark.parametrize("src_page,dst_page", [(1, 16), (16, 1), (16, 32)])
def test_copies_move_rows_whole(src_page, dst_page):
    """Rows of numbers, scales and padding through gather-scatter, gather and scatter."""
    say("copies of 4-bit rows", src_page, dst_page)
    rng = np.random.default_rng(8)
    L, H, D, n = 3, 2, 96, [17, 0, 40]
    lay = kvx.Layout(L, 2, H, D, "fp4")
    R, Q, T = lay.row_bytes, 2 * L, sum(n)

    def side(page):
        need = [-(-x // page) for x in n]
        P = sum(need) + 4
        ids = rng.permutation(P)[:sum(need)]
        raw = rng.integers(0, 256, (Q, P * page, R), dtype=np.uint8)
        off = offsets(need)
        rows = [int(ids[off[r] + t // page]) * page + t % page for r, m in enumerate(n) for t in range(m)]
        store = torch.from_numpy(raw).to(DEV)
        return (raw, rows, store, kvx.Pool(store, P, page, slot_stride=R),
                kvx.Table(ints(off, torch.int64), ints(ids, torch.int32)))

    src, dst, third = side(src_page), side(dst_page), side(dst_page)
    reqs = kvx.Requests(ints(offsets(n), torch.int64), T)
    kvx.gather_scatter(lay, src[3], src[4], reqs, dst[3], dst[4])
    staging = torch.zeros(T * Q * R, dtype=torch.uint8, device=DEV)
    kvx.gather(lay, src[3], src[4], reqs, staging)
    kvx.scatter(lay, staging, reqs, third[3], third[4])
    for raw, rows, store, *_ in (dst, third):
        raw[:, rows] = src[0][:, src[1]]
        assert np.array_equal(store.cpu().numpy(), raw)


def step_inputs(rng, dtype, n, H, G, D):
    new = rng.integers(1, 6, n)
    have = rng.integers(0, 90, n)
    q = torch.from_numpy(rng.standard_normal((int(new.sum()), H * G, D)).astype(np.float32))
    return new, have, q.to(TORCH[dtype])


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("page", [4, 16])
def test_step(dtype, layout, page):
    """A prompt's step and a decode step as a server runs them: tables, rows
    appended, read back, attended; the attention sees what was read."""
    say("fp4 step", dtype, layout, page)
    rng = np.random.default_rng(page)
    H, G, D, n, P = 2, 4, 64, 5, 200
    lay = kvx.Layout(2, 2, H, D, "fp4")
    store = torch.full((4, P, page * lay.row_bytes), 255, dtype=torch.uint8, device=DEV)
    pool = kvx.Pool(store, P, page, slot_stride=lay.row_bytes)
    free = rng.permutation(P).astype(np.int32)
    tab, held, have = kvx.BatchTables(n, 600, P), None, None
    keys = [[[] for _ in range(n)] for _ in range(2)]
    used = 0
    for add in (rng.integers(1, 90, n), np.ones(n, np.int64), rng.integers(0, 4, n)):
        T = int(add.sum())
        out_tab = kvx.BatchTables(n, 600, P)
        kvx.build_tables(out_tab, page, ints(add, torch.int32), ints(free[used:], torch.int32),
                         have_len=have, held=held.table if held is not None else None)
        reqs = out_tab.requests(T)
        q = torch.from_numpy(rng.standard_normal((T, H * G, D)).astype(np.float32)).to(TORCH[dtype])
        kv = torch.from_numpy(rng.standard_normal((2, T, H, D)).astype(np.float32)).to(TORCH[dtype])
        dev = kv.to(DEV)
        slots = out_tab.slots[:T]
        kvx.append(lay, 1, pool, slots, dev[0], dev[1], k_scale=0.5, v_scale=1.5, block_layout=layout)
        back = torch.zeros_like(dev)
        kvx.read(lay, 1, pool, slots, back[0], back[1], k_scale=0.5, v_scale=1.5, block_layout=layout)
        out = torch.zeros(T, H * G, D, dtype=TORCH[dtype], device=DEV)
        lse = torch.zeros(T, H * G, device=DEV)
        kvx.attend(lay, 1, pool, reqs, out_tab.ctx_len, out_tab.table, q.to(DEV), out, lse=lse,
                   k_scale=0.5, v_scale=1.5, block_layout=layout)
        torch.cuda.synchronize()
        for j, c in enumerate((0.5, 1.5)):
            codes, scales = f4.quantise(kv[j].float().numpy(), c)
            exact = f4.values(codes, scales) * c
            assert torch.equal(back[j].cpu(), torch.from_numpy(exact).to(TORCH[dtype]))
            for r in range(n):
                a, b = int(out_tab.tok_off[r]), int(out_tab.tok_off[r + 1])
                keys[j][r] += list(exact[a:b])
        # the same batch with its rows in a row
        ctx = out_tab.ctx_len.tolist()
        assert ctx == [len(x) for x in keys[0]]
        b = ref.Batch(1, sum(ctx), add.tolist(), ctx, offsets(ctx), np.arange(sum(ctx)))
        k, v = (np.concatenate([np.stack(x) for x in keys[j] if x]) for j in range(2))
        eo, el, mass, size, seen = ref.attend(b, q.double().numpy(), k, v, D ** -0.5)
        tol, tol_lse = ref.bounds(dtype, D, eo, el, mass, size, seen, np.abs(v).max())
        assert (np.abs(out.double().cpu().numpy() - eo) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - el) <= tol_lse).all()
        used += int(out_tab.totals[2])
        held, have = out_tab, out_tab.ctx_len


def test_rows_past_4_gib():
    """Slots whose byte offsets pass 32 bits, in both block layouts."""
    say("rows past 4 GiB")
    H, D, page = 8, 256, 16
    lay = kvx.Layout(1, 2, H, D, "fp4")
    R = lay.row_bytes
    P = (9 << 29) // (page * R) + 8             # planes of 4.5 GiB
    store = torch.zeros(2, P, page * R, dtype=torch.uint8, device=DEV)
    pool = kvx.Pool(store, P, page, slot_stride=R)
    rng = np.random.default_rng(6)
    at = [0, 5, (1 << 32) // R, (1 << 32) // R + 1, (1 << 31) // R, P * page - 1, P * page - 16]
    x = torch.from_numpy(rng.standard_normal((2, len(at), H, D)).astype(np.float32)).to(torch.bfloat16)
    for layout in ("nhd", "hnd"):
        dev = x.to(DEV)
        kvx.append(lay, 0, pool, ints(at, torch.int64), dev[0], dev[1], block_layout=layout)
        back = torch.zeros_like(dev)
        kvx.read(lay, 0, pool, ints(at, torch.int64), back[0], back[1], block_layout=layout)
        for j in range(2):
            codes, scales = f4.quantise(x[j].float().numpy())
            assert torch.equal(back[j].cpu().double(), torch.from_numpy(f4.values(codes, scales)))
            for t, s in enumerate(at):
                page_bytes = store[j, s // page].cpu().numpy()[None]
                n, sc = f4.views(page_bytes, page, H, D, layout)
                assert np.array_equal(n[0, s % page], f4.pack(codes[t]))
                assert np.array_equal(sc[0, s % page], scales[t])
        # attention over pages there
        q = torch.from_numpy(rng.standard_normal((1, 2 * H, D)).astype(np.float32)).to(torch.bfloat16)
        pages = [P - 1, (1 << 32) // R // page, 0]
        out, lse = torch.zeros_like(q).to(DEV), torch.zeros(1, 2 * H, device=DEV)
        store[:] = 0
        kv = torch.from_numpy(rng.standard_normal((2, 48, H, D)).astype(np.float32)).to(DEV)
        slots = [p * page + i for p in pages for i in range(page)]
        kvx.append(lay, 0, pool, ints(slots, torch.int64), kv[0], kv[1], block_layout=layout)
        kvx.attend(lay, 0, pool, kvx.Requests(ints([0, 1], torch.int64), 1), ints([45], torch.int32),
                   kvx.Table(ints([0, 3], torch.int64), ints(pages, torch.int32)), q.to(DEV), out, lse=lse,
                   block_layout=layout)
        k, v = (f4.values(*f4.quantise(kv[j].cpu().numpy())) for j in range(2))
        b = ref.Batch(1, 48, [1], [45], np.array([0, 45]), np.arange(45))
        eo, el, mass, size, seen = ref.attend(b, q.double().numpy(), k, v, D ** -0.5)
        tol, tol_lse = ref.bounds("bf16", D, eo, el, mass, size, seen, np.abs(v).max())
        assert (np.abs(out.double().cpu().numpy() - eo) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - el) <= tol_lse).all()
