"""Attention over 4-bit pools, against a 64-bit softmax of the values that the
pool stands for, within bounds that the arithmetic gives (serve_ref.bounds: the
values are exact in the query's type, so nothing else is rounded)."""
import numpy as np
import pytest
import torch

import scatter_kvx_gather_amd as kvx
from tests import fp4_ref as f4
from tests.fp4_util import Fp4Case, room_for_large
from tests.gpu_util import say
from tests.serve_util import DEV, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[False, True], ids=["small", "roomy"], autouse=True)
def roomy(request, monkeypatch):
    """Every test with a table of its own size and with one that has room for a
    large batch, whose rows go another way."""
    monkeypatch.setattr(Fp4Case, "roomy", request.param)
    return request.param


def run(name, scale=None, causal=True, **kw):
    say("attend fp4", name)
    c = Fp4Case(**kw)
    out, lse = c.run(scale=scale, causal=causal)
    torch.cuda.synchronize()
    c.check(out, lse, scale, causal)
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("ctx", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 257, 1000])
def test_one_token_one_request(dtype, ctx):
    run(f"1 token {dtype} {ctx}", seed=ctx, new=[1], ctx=[ctx], H=2, G=4, D=128, dtype=dtype)


@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("page,layout", [(16, "nhd"), (16, "hnd"), (4, "nhd"), (4, "hnd")])
def test_head_dims(D, dtype, new, page, layout):
    run(f"dim {D} {dtype} new {new} page {page} {layout}", seed=D, new=[new, 1, new], ctx=[70, 33, 129],
        H=2, G=3, D=D, dtype=dtype, page=page, layout=layout, k_scale=0.7, v_scale=1.3,
        members=[0, 3], prefix=[37])


@pytest.mark.parametrize("H,G", [(1, 1), (1, 8), (1, 16), (1, 17), (1, 32), (1, 100), (1, 128),
                                 (2, 6), (3, 5), (4, 1), (5, 3), (6, 7), (7, 2), (8, 8), (9, 1),
                                 (12, 3), (16, 2), (20, 1), (32, 1)])
def test_head_layouts(H, G):
    run(f"heads {H} x {G}", seed=H * 200 + G, new=[1, 1, 2], ctx=[77, 5, 130], H=H, G=G, D=64,
        members=[0, 3], prefix=[50])


@pytest.mark.parametrize("H,G", [(1, 1), (2, 6), (3, 5), (1, 100), (1, 128), (4, 8)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_query_tokens(H, G, D):
    """Enough rows per kv head for the wide tiles, ragged at every end."""
    run(f"wide {H} x {G} dim {D}", seed=H * 300 + G, new=[67, 1, 130, 9], ctx=[67, 300, 200, 9], H=H, G=G,
        D=D, members=[0, 1, 4], prefix=[150, 33])


@pytest.mark.parametrize("page", [1, 2, 3, 7, 16, 32, 48, 64, 100])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("joint", [False, True])
@pytest.mark.parametrize("D", [64, 96])
def test_pages(page, layout, joint, D):
    run(f"page {page} {layout} joint={joint} dim {D}", seed=page, new=[1, 3, 1],
        ctx=[page, 3 * page + 1, 130], H=3, G=2, D=D, page=page, layout=layout, joint=joint, layers=3,
        layer=1, members=[0, 3], prefix=[2 * page + 5])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx", [([5, 64, 33], [5, 64, 33]), ([16, 100, 1], [300, 100, 1]),
                                     ([300, 7], [310, 500]), ([1, 1, 1], [0, 1, 2]),
                                     ([3, 2], [64, 130])])
def test_masks(causal, new, ctx):
    run(f"mask {causal} {new}", causal=causal, seed=sum(new), new=new, ctx=ctx, H=2, G=4, D=128)


@pytest.mark.parametrize("with_prefix", [False, True])
def test_rows_that_see_nothing(with_prefix):
    """More query tokens than context, empty contexts, empty requests and empty
    prefixes: rows without a key get zeros and -inf."""
    kw = dict(members=[0, 2, 2, 6], prefix=[0, 40, 0]) if with_prefix else {}
    c = run("empty rows", seed=5, new=[5, 0, 40, 1, 3, 0], ctx=[2, 10, 7, 0, 0, 0], H=2, G=4, D=64,
            **kw)
    out, lse = c.run()
    assert not out[:3].any() and torch.isinf(lse[:3]).all() and (lse[:3] < 0).all()


@pytest.mark.parametrize("groups", [1, 3])
@pytest.mark.parametrize("rows", ["few", "many"])
def test_prefixes(groups, rows):
    n = 5 if rows == "few" else 40
    rng = np.random.default_rng(groups)
    new = rng.integers(1, 4, n).tolist()
    ctx = [x + int(rng.integers(0, 90)) for x in new]
    members = [0, n] if groups == 1 else [0, 2, 2, n]
    prefix = [200] if groups == 1 else [100, 55, 301]
    run(f"prefix {groups} {rows}", seed=9, new=new, ctx=ctx, H=2, G=4, D=128, members=members,
        prefix=prefix)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("page", [4, 16])
def test_out_of_range_pages(new, page):
    """Bad page ids and lists that run off the id array are not seen, counted
    once each, and read nothing."""
    say("fp4 out of range", new, page)
    c = Fp4Case(77, new=[new, 1, new], ctx=[200, 90, 150], H=2, G=4, D=64, page=page, bad=0.3,
                members=[0, 3], prefix=[120])
    skipped = torch.zeros(1, dtype=torch.int64, device=DEV)
    out, lse = c.run(skipped=skipped)
    c.check(out, lse)
    assert skipped.item() == c.b.skipped() > 0
    for r, x in ((0, -3), (1, 10**12), (2, -2**62)):
        c.b.pg_off[r] = x
    c.b.pre_off[0] = len(c.b.pre_ids) - 2
    c.upload()
    skipped.zero_()
    out, lse = c.run(skipped=skipped)
    c.check(out, lse)
    assert skipped.item() == c.b.skipped()
    # nothing left to see
    c.b.ids[:] = -1
    c.b.pre_ids[:] = c.num_pages
    c.upload()
    out, lse = c.run()
    assert not out.any() and (lse == -np.inf).all()


@pytest.mark.parametrize("new", [1, 3, 60])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (128, 2), (256, 16), (96, 3)])
def test_masked_nan_blocks(new, dtype, D, page):
    """Blocks of NaN in K and V rows of the newest tokens reach exactly the
    queries that see them."""
    say("fp4 NaN blocks", new, dtype, D, page)
    c = Fp4Case(13, new=[new, 2], ctx=[new + 21, 40], H=2, G=4, D=D, dtype=dtype, page=page,
                members=[0, 2], prefix=[30])
    for which in (0, 1):
        keep = [x.copy() for x in c.scales]
        rows = c.b.rows(c.b.pg_off[0], c.b.ids, c.b.ctx[0])
        c.scales[which][rows[-1], 0, 0] = f4.NAN_SCALE
        c.scales[which][rows[-(new + 1) // 2], 1, D // 32 - 1] = f4.NAN_SCALE
        c.decode()
        c.upload()
        out, lse = c.run()
        eo, el, *_ = c.expected()
        go = out.double().cpu().numpy()
        assert np.array_equal(np.isnan(go), np.isnan(eo)) and np.isnan(eo).any()
        if which == 1:
            c.check(out, lse)
        c.scales = keep


def test_every_number_and_scale():
    """All sixteen numbers under every scale that a pool holds, in K and in V, one
    key at a time: its value is the output."""
    say("fp4 numbers and scales")
    H, D, n = 2, 64, 37
    for dtype in ("bf16", "f16"):
        c = Fp4Case(3, new=[1] * n, ctx=[1] * n, H=H, G=1, D=D, dtype=dtype)
        rows = [c.b.rows(c.b.pg_off[r], c.b.ids, 1)[0] for r in range(n)]
        for j in range(2):
            for r, x in enumerate(rows):
                c.codes[j][x] = (np.arange(H * D) % 16).reshape(H, D)
                c.scales[j][x] = 104 + r if j else min(104 + r, 127)
        c.decode()
        c.upload()
        out, lse = c.run()
        v = c.kv[1][rows].double()
        assert torch.equal(out.cpu().double(), v.expand(n, H, D))
        c.check(out, lse)


@pytest.mark.parametrize("prefix", [0, 5000])
@pytest.mark.parametrize("new", [[1], [3, 1], [40]])
@pytest.mark.parametrize("D,H,G,page", [(64, 1, 5, 32), (128, 3, 2, 32), (256, 1, 3, 8), (128, 1, 9, 1)])
def test_many_pieces(D, H, G, page, new, prefix):
    """Few rows and long contexts: items in two to a hundred pieces, thin and
    wide, whose joins share a row among waves and workgroups."""
    say("fp4 pieces", D, H, G, page, new, prefix)
    n = len(new)
    extra = dict(members=[0, n], prefix=[prefix]) if prefix else {}
    for own in (700, 6000):
        c = Fp4Case(24, new=new, ctx=[own, 333][:n], H=H, G=G, D=D, page=page, **extra)
        out, lse = c.run()
        torch.cuda.synchronize()
        c.check(out, lse)


@pytest.mark.parametrize("roomy", [True], indirect=True)
@pytest.mark.parametrize("layout,page", [("nhd", 1), ("nhd", 16), ("hnd", 16), ("hnd", 64), ("hnd", 48)])
@pytest.mark.parametrize("H,G,D", [(2, 3, 32), (3, 2, 64), (4, 4, 128), (5, 2, 96), (8, 4, 128), (8, 1, 64),
                                   (12, 2, 128), (11, 1, 96), (3, 20, 64), (4, 2, 160), (2, 4, 256)])
@pytest.mark.parametrize("prefix", [0, 75])
def test_many_requests(layout, page, H, G, D, prefix):
    """Batches that go through shared memory in both block layouts: ragged
    contexts, empty ones, pages out of range, blocks of NaN in the newest rows."""
    say("fp4 many requests", layout, page, H, G, D, prefix)
    n = 70
    rng = np.random.default_rng(H * 100 + D)
    new = rng.choice([1, 1, 1, 2, 3, 0], n).tolist()
    ctx = [max(x, int(rng.choice([0, 1, 15, 17, 31, 33, 64, 90, 150]))) for x in new]
    extra = dict(members=[0, n], prefix=[prefix]) if prefix else {}
    c = Fp4Case(8, new=new, ctx=ctx, H=H, G=G, D=D, page=page, layout=layout, bad=0.04,
                k_scale=0.5, v_scale=2.0, **extra)
    for r in range(0, n, 9):
        rows = [x for x in c.b.rows(c.b.pg_off[r], c.b.ids, ctx[r])[-2:] if x is not None]
        for x in rows:
            c.scales[1][x, r % H, 0] = f4.NAN_SCALE
    c.decode()
    c.upload()
    skipped = torch.zeros(1, dtype=torch.int64, device=DEV)
    out, lse = c.run(skipped=skipped)
    torch.cuda.synchronize()
    c.check(out, lse)
    assert skipped.item() == c.b.skipped()
    again, lse2 = c.run()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_scores_that_grow():
    """Maxima that rise along the keys (the accumulators are rescaled often)."""
    say("fp4 growing scores")
    c = Fp4Case(21, new=[1, 70], ctx=[500, 400], H=2, G=4, D=64)
    for r in range(2):
        rows = c.b.rows(c.b.pg_off[r], c.b.ids, c.b.ctx[r])
        for i, x in enumerate(rows):
            c.codes[0][x] = 2
            c.scales[0][x] = 120 + i * 10 // len(rows)
    c.q = torch.ones_like(c.q)
    c.decode()
    c.upload()
    out, lse = c.run()
    c.check(out, lse)


def test_results_repeat_and_the_workspace_is_scratch():
    say("fp4 repeat")
    c = Fp4Case(40, new=[1] * 30 + [50], ctx=[300] * 30 + [400], H=2, G=4, D=128, members=[0, 31],
                prefix=[700])
    need = kvx.attend_workspace(c.lay, c.reqs, 8, c.prefix)
    ws = torch.full((need,), 0x7f, dtype=torch.uint8, device=DEV)
    out, lse = c.run(workspace=ws)
    c.check(out, lse)
    ws.fill_(0xff)
    again, lse2 = c.run(workspace=ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)
    third, lse3 = c.run()
    assert torch.equal(out, third) and torch.equal(lse, lse3)


def test_rows_behind_the_last_request():
    """tok_off ends before total_tokens: rows from there on keep their contents."""
    say("fp4 rows behind")
    c = Fp4Case(41, new=[1, 2, 1], ctx=[90, 40, 300], H=2, G=4, D=128)
    out, lse = c.run()
    T = sum(c.b.new)
    q = torch.cat([c.qd, torch.full_like(c.qd, float("nan"))])
    o = torch.full_like(q, 5.0)
    z = torch.full((2 * T, 8), 6.0, device=DEV)
    kvx.attend(c.lay, 0, c.pool, kvx.Requests(c.tok_off, 2 * T), c.ctx, c.table, q, o, lse=z)
    assert torch.equal(o[:T], out) and torch.equal(z[:T], lse)
    assert (o[T:] == 5.0).all() and (z[T:] == 6.0).all()


def test_step_in_a_graph_and_on_another_stream(roomy):
    """append, read and attend captured once and replayed while slots, rows,
    lengths and tables change, eager work between; two graphs with a workspace
    each; and the same calls on a stream of their own."""
    say("fp4 graph")
    H, G, D, page, n, P = 2, 4, 128, 16, 6, 64
    lay = kvx.Layout(1, 2, H, D, "fp4")
    R = lay.row_bytes
    g = torch.Generator(device=DEV).manual_seed(2)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)

    def fresh():
        s = dict(store=torch.zeros(2, P, page * R, dtype=torch.uint8, device=DEV))
        s["pool"] = kvx.Pool(s["store"], P, page, slot_stride=R)
        s["slots"] = torch.zeros(n, dtype=torch.int64, device=DEV)
        s["ctx"] = torch.zeros(n, dtype=torch.int32, device=DEV)
        room = torch.full((P + roomy * room_for_large(H, D, page),), -1, dtype=torch.int32, device=DEV)
        s["ids"] = room[:P]
        s["tok"] = torch.arange(n + 1, device=DEV)
        s["off"] = torch.arange(0, 10 * n + 1, 10, device=DEV)
        s["table"], s["reqs"] = kvx.Table(s["off"], room), kvx.Requests(s["tok"], n)
        s["k"], s["v"], s["q"] = rand(n, H, D), rand(n, H, D), rand(n, H * G, D)
        s["bk"], s["bv"] = torch.zeros_like(s["k"]), torch.zeros_like(s["v"])
        s["out"] = torch.zeros_like(s["q"])
        s["ws"] = torch.zeros(kvx.attend_workspace(lay, s["reqs"], H * G), dtype=torch.uint8, device=DEV)
        return s

    def step(s, stream=None):
        kvx.append(lay, 0, s["pool"], s["slots"], s["k"], s["v"], stream=stream)
        kvx.read(lay, 0, s["pool"], s["slots"], s["bk"], s["bv"], stream=stream)
        kvx.attend(lay, 0, s["pool"], s["reqs"], s["ctx"], s["table"], s["q"], s["out"],
                   workspace=s["ws"], stream=stream)

    def change(s, i):
        perm = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
        s["ids"].copy_(perm)
        ctx = torch.randint(1, 160, (n,), generator=g, device=DEV).to(torch.int32)
        s["ctx"].copy_(ctx)
        t = ctx.long() - 1
        s["slots"].copy_(perm[s["off"][:-1] + t // page].long() * page + t % page)
        for x in ("k", "v", "q"):
            s[x].copy_(rand(*s[x].shape))

    a, b, eager = fresh(), fresh(), fresh()
    graphs = []
    for s in (a, b):
        change(s, 0)
        step(s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(s)
        graphs.append(graph)
    side = torch.cuda.Stream()
    for i in range(6):
        for s in (a, b):
            s["store"].random_(0, 256, generator=g)
            s["store"][:, :, :].bitwise_and_(0x7f)          # no block of NaN
            change(s, i)
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for s in (a, b):
            got = [s[x].clone() for x in ("bk", "bv", "out")]
            for x in ("store", "slots", "ctx", "ids", "k", "v", "q"):
                eager[x].copy_(s[x])
            eager["out"].fill_(9)
            side.wait_stream(torch.cuda.current_stream())
            step(eager, side if i % 2 else None)
            torch.cuda.synchronize()
            for x, y in zip(got, (eager["bk"], eager["bv"], eager["out"])):
                assert torch.equal(x, y) and x.isfinite().all()
