"""Tables built from lengths, and rows appended, against plain host forms; and
the serving step as a whole."""
import numpy as np
import pytest
import torch

import scatter_kvx_gather_amd as kvx
from tests import serve_ref as ref
from tests.gpu_util import say
from tests.serve_util import DEV, TORCH, ints, offsets

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ build_tables --

def build(page, have, add, free, held_lists=None, cap_tokens=None, cap_pages=None, out=None):
    have_l = have if have is not None else None
    exp = ref.build_tables(page, have_l, add, held_lists, free)
    n = len(add)
    ct = len(exp["slots"]) if cap_tokens is None else cap_tokens
    cp = len(exp["ids"]) if cap_pages is None else cap_pages
    o = out or kvx.BatchTables(n, ct, cp)
    held = None
    if have is not None:
        held = kvx.Table(ints(offsets([len(x) for x in held_lists]), torch.int64),
                         ints(np.concatenate([np.asarray(x, np.int32) for x in held_lists] +
                                             [np.zeros(0, np.int32)]), torch.int32))
    kvx.build_tables(o, page, ints(add, torch.int32), ints(free, torch.int32),
                     have_len=ints(have, torch.int32) if have is not None else None, held=held)
    torch.cuda.synchronize()
    assert o.ctx_len.tolist() == exp["ctx"]
    assert o.tok_off.tolist() == exp["tok_off"] and o.pg_off.tolist() == exp["pg_off"]
    assert o.totals.tolist() == exp["totals"]
    k = min(cp, len(exp["ids"]))
    assert o.page_ids[:k].tolist() == exp["ids"][:k]
    assert (o.page_ids[k:] == -1).all()             # rows behind the last: as they were
    k = min(ct, len(exp["slots"]))
    assert o.slots[:k].tolist() == exp["slots"][:k]
    assert (o.slots[k:] == -1).all()
    return o, exp


def lists(rng, have, page, pool):
    perm = rng.permutation(pool)
    out, at = [], 0
    for h in have:
        k = -(-max(int(h), 0) // page)
        out.append(perm[at:at + k])
        at += k
    return out, perm[at:]


@pytest.mark.parametrize("page", [1, 2, 7, 16, 64])
@pytest.mark.parametrize("n,most_have,most_add", [(1, 0, 1), (1, 5000, 1), (3, 40, 40), (64, 300, 1),
                                                  (256, 20, 3), (257, 20, 3), (40, 9000, 9000), (1023, 9, 2), (1024, 9, 2),
                                                  (1025, 9, 2), (3000, 3, 1), (2, 0, 9000)])
def test_build_tables(page, n, most_have, most_add):
    say("build", page, n, most_have, most_add)
    rng = np.random.default_rng(page * 10000 + n + most_have)
    have = rng.integers(0, most_have + 1, n)
    add = rng.integers(0, most_add + 1, n)
    held, free = lists(rng, have, page, int(sum(have)) + int(sum(add)) + 3 * n + 20)
    build(page, have, add, free, held, cap_tokens=int(sum(add)) + 37)
    build(page, have, add, free, held)


def test_build_tables_without_a_held_table():
    build(16, None, [5, 0, 16, 17, 1000], np.arange(100)[::-1])


def test_build_tables_edges():
    say("build edges")
    # no request at all; nothing but empty requests; negative lengths count as 0
    o = kvx.BatchTables(0, 0, 0)
    kvx.build_tables(o, 16, ints([], torch.int32), ints([], torch.int32))
    assert o.tok_off.tolist() == [0] and o.pg_off.tolist() == [0] and o.totals.tolist() == [0] * 4
    build(16, None, [0, 0, 0], np.arange(4))
    build(16, [-5, 3, -1], [2, -7, 0], np.arange(100, 120), [[], [9], []])
    # the free list runs short; held lists shorter than the length says
    build(4, None, [10, 10, 10], np.arange(5))
    build(4, [0, 6], [9, 9], np.arange(50, 52), [[], [3, 8]])
    build(4, [9, 9], [1, 5], np.arange(50, 60), [[1, 2, 3], [7]])
    # a held page that is out of range already stays so, and its tokens get slot -1
    build(4, [6], [5], np.arange(50, 60), [[3, -1]])


def test_build_tables_capacities():
    say("build capacities")
    rng = np.random.default_rng(3)
    add = rng.integers(0, 200, 50)
    free = rng.permutation(4000)
    for ct, cp in ((0, 0), (1, 1), (1000, 100), (10**5, 10**4)):
        build(8, None, add, free, cap_tokens=ct, cap_pages=cp)


def test_build_tables_total_stops_at_int32():
    have, add = ints([2**31 - 3, 5], torch.int32), ints([10, 1], torch.int32)
    o = kvx.BatchTables(2, 8, 8)
    held = kvx.Table(ints([0, 0], torch.int64), ints([4], torch.int32))
    kvx.build_tables(o, 1 << 20, add, ints([7, 8, 9], torch.int32), have_len=have, held=held)
    assert o.ctx_len.tolist() == [2**31 - 1, 6]
    assert o.tok_off.tolist() == [0, 2, 3]
    assert o.slots[2].item() == 4 * (1 << 20) + 5


def test_build_tables_in_buffers_side_by_side():
    """Inputs and outputs that touch, in one allocation, do not overlap; one
    that is an input's memory is refused and nothing is written."""
    say("build side by side")
    n, page, have, add = 3, 4, [5, 0, 9], [4, 1, 7]
    held_lists, free = [[3, 4], [], [7, 8, 9]], list(range(20, 30))
    exp = ref.build_tables(page, have, add, held_lists, free)
    arena = torch.full((4096,), 77, dtype=torch.uint8, device=DEV)
    at = 0

    def take(count, dtype):
        nonlocal at
        size = count * torch.empty(0, dtype=dtype).element_size()
        at += size
        return arena[at - size:at].view(dtype)

    ids = [x for h in held_lists for x in h]
    slots, pages = len(exp["slots"]), len(exp["ids"])
    free_ids, held_ids, page_ids = (take(c, torch.int32) for c in (len(free), len(ids), pages + pages % 2 + 1))
    have_len, ctx, add_len = (take(n, torch.int32) for _ in range(3))
    at += -at % 8
    held_off, tok_off, pg_off = (take(n + 1, torch.int64) for _ in range(3))
    o = kvx.BatchTables(n, slots, pages)
    o.slots, o.totals = take(slots, torch.int64), take(4, torch.int64)
    o.ctx_len, o.tok_off, o.pg_off, o.page_ids = ctx, tok_off, pg_off, page_ids[:pages]
    o._c = kvx._CBatchTables(*(x.data_ptr() for x in (ctx, tok_off, pg_off, page_ids)), pages,
                             o.slots.data_ptr(), slots, o.totals.data_ptr())
    for dst, src in ((free_ids, free), (held_ids, ids), (have_len, have), (add_len, add),
                     (held_off, offsets([len(x) for x in held_lists]))):
        dst.copy_(torch.as_tensor(np.asarray(src)))
    held = kvx.Table(held_off, held_ids)
    kvx.build_tables(o, page, add_len, free_ids, have_len=have_len, held=held)
    torch.cuda.synchronize()
    assert ctx.tolist() == exp["ctx"] and tok_off.tolist() == exp["tok_off"]
    assert pg_off.tolist() == exp["pg_off"] and o.page_ids.tolist() == exp["ids"]
    assert o.slots.tolist() == exp["slots"] and o.totals.tolist() == exp["totals"]
    assert have_len.tolist() == have and add_len.tolist() == add and held_ids.tolist() == ids
    before = arena.clone()
    for kw in (dict(have_len=ctx), dict(add_len=ctx), dict(held=kvx.Table(pg_off, held_ids)),
               dict(free_ids=page_ids)):
        args = dict(add_len=add_len, free_ids=free_ids, have_len=have_len, held=held)
        args.update(kw)
        with pytest.raises(kvx.KvxError) as e:
            kvx.build_tables(o, page, **args)
        assert e.value.status == 9, kw
    torch.cuda.synchronize()
    assert torch.equal(arena, before)


# ----------------------------------------------------------------- append --

def e4m3(x):
    """Values as e4m3 holds them: nearest even of the held values, by torch on the host."""
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def append_case(seed, T, H, D, src, pool, page, layout, joint=False, layers=2, layer=1, bad=False):
    rng = np.random.default_rng(seed)
    pages = -(-T // page) + 9
    t = {"f32": torch.float32, **TORCH}
    es = {"f32": 4, "fp8": 1}.get(pool, 2)
    R, Q = H * D * es, 2 * layers
    fill = torch.from_numpy(rng.integers(0, 256, (Q, pages, page * R), dtype=np.uint8))
    if joint:
        store = fill.transpose(0, 1).contiguous().to(DEV)
        base = store.data_ptr()
        P = kvx.Pool([base + q * page * R for q in range(Q)], pages, page, slot_stride=R,
                     page_stride=Q * page * R, keep=store)
    else:
        store = fill.to(DEV)
        P = kvx.Pool(store, pages, page, slot_stride=R)
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn(T, 3 * H, D, generator=g) * 20)
    qkv = qkv.clamp(-448, 448).to(t[src]) if src == "fp8" else qkv.to(t[src])
    k, v = qkv[:, H:2 * H], qkv[:, 2 * H:]
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    if bad:
        m = rng.random(T) < 0.3
        slots[m] = rng.choice([-1, -2**62, pages * page, 2**62], m.sum())
    scales = (0.05, 0.3) if pool == "fp8" and src != "fp8" else (1.0, 1.0)
    skipped = torch.zeros(1, dtype=torch.int64, device=DEV)
    qd = qkv.view(torch.uint8).to(DEV).view(qkv.dtype)
    kvx.append(kvx.Layout(layers, 2, H, D, pool), layer, P, ints(slots, torch.int64),
               qd[:, H:2 * H], qd[:, 2 * H:], *scales, block_layout=layout, skipped=skipped)
    torch.cuda.synchronize()
    exp = fill.clone()
    for j, (x, s) in enumerate(((k, scales[0]), (v, scales[1]))):
        if scales != (1.0, 1.0):
            x = e4m3(x.float() / torch.tensor(s, dtype=torch.float32))
        x = x.contiguous().view(torch.uint8).view(T, H, D * es)
        plane = exp[2 * layer + j]
        plane = plane.view(pages, page, H, D * es) if layout == "nhd" else \
            plane.view(pages, H, page, D * es).transpose(1, 2)
        ok = (slots >= 0) & (slots < pages * page)
        at = torch.from_numpy(slots[ok])
        plane[at // page, at % page] = x[torch.from_numpy(ok)]
    got = store.cpu()
    got = got.transpose(0, 1) if joint else got
    assert torch.equal(got, exp), (seed, T, H, D, src, pool, page, layout)
    assert skipped.item() == int((~((slots >= 0) & (slots < pages * page))).sum())


@pytest.mark.parametrize("src,pool", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("fp8", "fp8"),
                                      ("bf16", "fp8"), ("f16", "fp8"), ("f32", "fp8")])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("T", [1, 3, 64, 700])
def test_append(src, pool, layout, T):
    say("append", src, pool, layout, T)
    for i, (H, D, page, joint) in enumerate(((8, 128, 16, False), (1, 64, 1, False), (5, 80, 3, True),
                                             (2, 256, 32, True))):
        append_case(T * 10 + i, T, H, D, src, pool, page, layout, joint, bad=i == 2)


def test_append_rows_that_are_not_whole_heads():
    """NHD rows only need to be a multiple of 16 bytes."""
    append_case(1, 33, 4, 4, "bf16", "bf16", 4, "nhd")
    append_case(2, 33, 4, 12, "f16", "f16", 4, "nhd")


def test_append_rounding_and_special_values():
    """Every bf16 value as e4m3: ties to even, held at 448, NaN kept."""
    say("append every bf16")
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(512, 1, 128)
    pool = torch.zeros(2, 512, 128, dtype=torch.uint8, device=DEV)
    kvx.append(kvx.Layout(1, 2, 1, 128, "fp8"), 0, kvx.Pool(pool, 512, 1, slot_stride=128),
               torch.arange(512, device=DEV), x.to(DEV), x.to(DEV))
    got = pool.cpu().view(torch.float8_e4m3fn).float()
    f = x.view(512, 128).float()
    exp = e4m3(f).float()
    for p in range(2):
        assert torch.equal(torch.isnan(got[p]), torch.isnan(f))
        assert torch.equal(got[p][~torch.isnan(f)], exp[~torch.isnan(f)])


def test_append_nothing():
    pool = torch.zeros(2, 4, 128, dtype=torch.uint8, device=DEV)
    kv = torch.zeros(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    kvx.append(kvx.Layout(1, 2, 1, 64, "bf16"), 0, kvx.Pool(pool, 4, 1, slot_stride=128),
               torch.zeros(0, dtype=torch.int64, device=DEV), kv, kv)


# ---------------------------------------------------------- the whole step --

class Server:
    """A decoder's cache beside a plain one: lists of K and V rows per request."""

    def __init__(self, layers, H, G, D, dtype, pool, page, pages, layout, seed):
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator().manual_seed(seed)
        self.L, self.H, self.G, self.D, self.dtype, self.page, self.layout = layers, H, G, D, dtype, page, layout
        self.scales = (0.05, 0.04) if pool == "fp8" else (1.0, 1.0)
        es = 1 if pool == "fp8" else 2
        self.pool_type = pool
        self.store = torch.zeros(2 * layers, pages * page, H * D * es, dtype=torch.uint8, device=DEV)
        self.pool = kvx.Pool(self.store, pages, page, slot_stride=H * D * es)
        self.lay = kvx.Layout(layers, 2, H, D, pool)
        self.free = list(self.rng.permutation(pages))

    def rows(self, T):
        return [(torch.randn(T, n, self.D, generator=self.gen)).to(TORCH[self.dtype])
                for n in (self.H * self.G, self.H, self.H)]

    def held(self, x, j):
        if self.pool_type != "fp8":
            return x.double().numpy()
        s = torch.tensor(self.scales[j], dtype=torch.float32)
        return e4m3(x.float() / s).double().numpy() * float(s)


@pytest.mark.parametrize("pool,layout,page", [("bf16", "nhd", 16), ("fp8", "hnd", 8), ("bf16", "nhd", 1)])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_step(pool, layout, page, captured):
    """A prompt shared by all, prompts of their own, then decode steps: tables,
    append and attend of two layers in a row, the decode step eager or replayed
    from one capture.  Checked against plain caches after every step."""
    say("serve", pool, layout, page, captured)
    S = Server(2, 2, 4, 64, "bf16", pool, page, 200 if page > 1 else 900, layout, 5)
    N, P = 5, 45
    cache = [[[np.zeros((0, S.H, S.D)) for _ in range(2)] for _ in range(N + 1)] for _ in range(S.L)]

    def step(tables, add, T, data, prefix):
        outs = []
        reqs = tables.requests(T)
        for l, (q, k, v) in enumerate(data):
            kvx.append(S.lay, l, S.pool, tables.slots[:T], k, v, *S.scales, block_layout=layout)
            out = torch.empty_like(q)
            kvx.attend(S.lay, l, S.pool, reqs, tables.ctx_len, tables.table, q, out, prefix=prefix,
                       k_scale=S.scales[0], v_scale=S.scales[1], block_layout=layout)
            outs.append(out)
        return outs

    def remember(who, add, data):
        for l, (q, k, v) in enumerate(data):
            at = 0
            for r, a in zip(who, add):
                for j, x in enumerate((k, v)):
                    cache[l][r][j] = np.concatenate([cache[l][r][j], S.held(x[at:at + a], j)])
                at += a

    def check(outs, who, add, data, shared):
        for l, out in enumerate(outs):
            at = 0
            for r, a in zip(who, add):
                k, v = (np.concatenate([cache[l][N][j][:P if shared else 0], cache[l][r][j]])
                        for j in range(2))
                n = len(k)
                b = ref.Batch(n, 1, [a], [n], np.array([0, 1]), np.array([0]))
                q = data[l][0][at:at + a].double().numpy()
                eo, el, mass, size, seen = ref.attend(b, q, k, v, S.D ** -0.5)
                tol, _ = ref.bounds("bf16", S.D, eo, el, mass, size, seen, np.abs(v).max())
                assert (np.abs(out[at:at + a].double().cpu().numpy() - eo) <= tol).all(), (l, r)
                at += a

    def upload(data):
        return [tuple(x.to(DEV) for x in row) for row in data]

    # the shared prompt, as a batch of one
    sys_t = kvx.BatchTables(1, P, 64 if page > 1 else 64)
    free = ints(S.free, torch.int32)
    data = [S.rows(P) for _ in range(S.L)]
    kvx.build_tables(sys_t, page, ints([P], torch.int32), free)
    outs = step(sys_t, [P], P, upload(data), None)
    remember([N], [P], data)
    check(outs, [N], [P], data, False)
    S.free = S.free[sys_t.totals[2].item():]
    prefix = kvx.Prefix(ints([0, N], torch.int64), ints([P], torch.int32), sys_t.table)

    # their own prompts
    add = [7, 1, 30, 16, 70]
    cap = 400
    T2 = [kvx.BatchTables(N, 200, cap) for _ in range(2)]
    free = ints(S.free, torch.int32)
    data = [S.rows(sum(add)) for _ in range(S.L)]
    kvx.build_tables(T2[0], page, ints(add, torch.int32), free)
    outs = step(T2[0], add, sum(add), upload(data), prefix)
    remember(range(N), add, data)
    check(outs, range(N), add, data, True)
    S.free = S.free[T2[0].totals[2].item():]

    # decode: tables of one step feed the next
    ones = ints([1] * N, torch.int32)
    free_d = ints(S.free + [-1] * (1000 - len(S.free)), torch.int32)
    ins = upload([S.rows(N) for _ in range(S.L)])
    graph = None

    def decode():
        kvx.build_tables(T2[1], page, ones, free_d, have_len=T2[0].ctx_len, held=T2[0].table)
        outs = step(T2[1], [1] * N, N, ins, prefix)
        for a, b in ((T2[0].ctx_len, T2[1].ctx_len), (T2[0].pg_off, T2[1].pg_off),
                     (T2[0].page_ids, T2[1].page_ids)):
            a.copy_(b)
        return outs

    for i in range(4):
        data = [S.rows(N) for _ in range(S.L)]
        for dst, src in zip(ins, data):
            for a, b in zip(dst, src):
                a.copy_(b)
        free_d[:len(S.free)] = ints(S.free, torch.int32)
        torch.cuda.synchronize()
        if captured and graph is None and i == 1:
            # capture enqueues nothing, so the state is untouched by it
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs = decode()
            torch.cuda.synchronize()
        if graph is not None:
            graph.replay()
        else:
            outs = decode()
        torch.cuda.synchronize()
        remember(range(N), [1] * N, data)
        check(outs, range(N), [1] * N, data, True)
        S.free = S.free[T2[1].totals[2].item():]


def test_captured_step_of_batches_that_shrink():
    """One capture of tables, append and attend with room for 40 tokens of 4
    requests, replayed with fewer: rows and slots behind the batch are left."""
    say("padded step")
    rng = np.random.default_rng(31)
    H, G, D, page, room, N = 2, 2, 64, 16, 40, 4
    lay = kvx.Layout(1, 2, H, D, "bf16")
    store = torch.zeros(2, 64, page, H, D, dtype=torch.bfloat16, device=DEV)
    pool = kvx.Pool(store, 64, page, slot_stride=H * D * 2)
    t = kvx.BatchTables(N, room, 16)
    free = ints(rng.permutation(64), torch.int32)
    add = ints([1] * N, torch.int32)
    q, out = (torch.zeros(room, H * G, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v = (torch.zeros(room, H, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    skipped = torch.zeros(1, dtype=torch.int64, device=DEV)
    reqs = t.requests(room)
    ws = torch.empty(kvx.attend_workspace(lay, reqs, H * G), dtype=torch.uint8, device=DEV)

    def step():
        t.slots.fill_(-1)
        kvx.build_tables(t, page, add, free)
        kvx.append(lay, 0, pool, t.slots, k, v, skipped=skipped)
        kvx.attend(lay, 0, pool, reqs, t.ctx_len, t.table, q, out, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for new in ([20, 1, 3, 16], [0, 5, 0, 1], [0, 0, 0, 0], [17, 17, 2, 0]):
        T = sum(new)
        host = [torch.randn(room, h, D).to(torch.bfloat16) for h in (H * G, H, H)]
        for x, y in zip((q, k, v), host):
            x.copy_(y)
        add.copy_(ints(new, torch.int32))
        out.fill_(7)
        skipped.zero_()
        before = store.clone()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert skipped.item() == room - T and (out[T:] == 7).all()
        rows = t.slots[:T].cpu().numpy()
        left = np.setdiff1d(np.arange(64 * page), rows)
        now = store.view(2, 64 * page, H, D)
        assert torch.equal(now[:, left], before.view(now.shape)[:, left])
        off = np.concatenate([[0], np.cumsum(new)])
        for r, n in enumerate(new):
            if n == 0:
                continue
            mine = slice(off[r], off[r + 1])
            b = ref.Batch(n, 1, [n], [n], np.array([0, 1]), np.array([0]))
            a = [x[mine].double().numpy() for x in host]
            eo, el, mass, size, seen = ref.attend(b, *a, D ** -0.5)
            tol, _ = ref.bounds("bf16", D, eo, el, mass, size, seen, np.abs(a[2]).max())
            assert (np.abs(out[mine].double().cpu().numpy() - eo) <= tol).all()
