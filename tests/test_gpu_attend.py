"""Attention over paged pools with shared prefixes, against a 64-bit softmax on
the host, within bounds that the arithmetic gives (serve_ref.bounds)."""
import numpy as np
import pytest
import torch

import scatter_kvx_gather_amd as kvx
from tests.gpu_util import say
from tests.serve_util import DEV, Case, ints, offsets

pytestmark = pytest.mark.gpu


def run(name, scale=None, causal=True, **kw):
    say("attend", name)
    c = Case(**kw)
    out, lse = c.run(scale=scale, causal=causal)
    torch.cuda.synchronize()
    c.check(out, lse, scale, causal)
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("ctx", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 257, 1000])
def test_one_token_one_request(dtype, ctx):
    run(f"1 token {dtype} {ctx}", seed=ctx, new=[1], ctx=[ctx], H=2, G=4, D=128, dtype=dtype)


@pytest.mark.parametrize("D", [16, 40, 64, 72, 80, 96, 112, 128, 136, 160, 192, 256])
@pytest.mark.parametrize("new", [1, 40])
def test_head_dims(D, new):
    run(f"dim {D} new {new}", seed=D, new=[new, 1, new], ctx=[70, 33, 129], H=2, G=3, D=D)


@pytest.mark.parametrize("D", [16, 64, 96, 128, 192, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("new", [1, 50])
def test_fp8_pools(D, dtype, new):
    run(f"fp8 dim {D} {dtype}", seed=D + 1, new=[new, 2], ctx=[90, 41], H=2, G=2, D=D, dtype=dtype,
        pool="fp8", k_scale=0.03, v_scale=0.07, members=[0, 2], prefix=[37])


@pytest.mark.parametrize("H,G", [(1, 1), (1, 8), (1, 16), (1, 17), (1, 32), (1, 100), (1, 128),
                                 (2, 6), (3, 5), (4, 1), (5, 3), (6, 7), (7, 2), (8, 8), (9, 1),
                                 (12, 3), (16, 2), (20, 1), (32, 1)])
def test_head_layouts(H, G):
    run(f"heads {H} x {G}", seed=H * 200 + G, new=[1, 1, 2], ctx=[77, 5, 130], H=H, G=G, D=64,
        members=[0, 3], prefix=[50])


@pytest.mark.parametrize("H,G", [(1, 1), (2, 6), (3, 5), (1, 100), (1, 128), (4, 8)])
def test_many_query_tokens(H, G):
    """Enough rows per kv head for the wide tiles, ragged at every end."""
    run(f"wide {H} x {G}", seed=H * 300 + G, new=[67, 1, 130, 9], ctx=[67, 300, 200, 9], H=H, G=G,
        D=64, members=[0, 1, 4], prefix=[150, 33])


@pytest.mark.parametrize("page", [1, 2, 3, 7, 16, 32, 64, 100])
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
@pytest.mark.parametrize("joint", [False, True])
def test_pages(page, layout, joint):
    run(f"page {page} {layout} joint={joint}", seed=page, new=[1, 3, 1], ctx=[page, 3 * page + 1, 130],
        H=2, G=2, D=64, page=page, layout=layout, joint=joint, layers=3, layer=1,
        members=[0, 3], prefix=[2 * page + 5])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,ctx", [([5, 64, 33], [5, 64, 33]), ([16, 100, 1], [300, 100, 1]),
                                     ([300, 7], [310, 500]), ([1, 1, 1], [0, 1, 2])])
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
    """Prefixes of several lengths, a group without requests and a batch whose
    groups end inside tiles."""
    n = 5 if rows == "few" else 40
    rng = np.random.default_rng(groups)
    new = rng.integers(1, 4, n).tolist()
    ctx = [x + int(rng.integers(0, 90)) for x in new]
    members = [0, n] if groups == 1 else [0, 2, 2, n]
    prefix = [200] if groups == 1 else [100, 55, 301]
    c = run(f"prefix {groups} {rows}", seed=9, new=new, ctx=ctx, H=2, G=4, D=128, members=members,
            prefix=prefix)
    # the same keys as one context per request give the same sums
    assert c.prefix.num_groups == len(prefix)


def test_prefix_equals_own_copy():
    """A prefix written into each request's own context gives the same result
    within the bounds of both."""
    c = Case(31, new=[1, 1, 1, 1], ctx=[20, 1, 33, 64], H=2, G=4, D=128, members=[0, 4], prefix=[48])
    b = c.b
    lists, off = [], [0]
    for r, n in enumerate(b.ctx):
        lists += list(b.pre_ids) + list(b.ids[b.pg_off[r]:b.pg_off[r + 1]])
        off.append(len(lists))
    out, lse = c.run()
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    kvx.attend(c.lay, 0, c.pool, c.reqs, ints([x + 48 for x in b.ctx], torch.int32),
               kvx.Table(ints(off, torch.int64), ints(lists, torch.int32)), c.qd, out2, lse=lse2)
    c.check(out, lse)
    c.check(out2, lse2)


@pytest.mark.parametrize("new", [1, 40])
def test_out_of_range_pages(new):
    """Bad page ids and lists that run off the id array are not seen, counted
    once each, and read nothing."""
    say("out of range", new)
    c = Case(77, new=[new, 1, new], ctx=[200, 90, 150], H=2, G=4, D=64, page=4, bad=0.3,
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
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_masked_infinities(new, dtype, value):
    """Infinities and NaN in K and V rows of the newest tokens reach exactly the
    queries that see them."""
    say("infinities", new, dtype, value)
    c = Case(13, new=[new, 2], ctx=[new + 21, 40], H=2, G=4, D=64, dtype=dtype, members=[0, 2],
             prefix=[30])
    for which in (0, 1):
        kv = [x.clone() for x in c.kv]
        rows = c.b.rows(c.b.pg_off[0], c.b.ids, c.b.ctx[0])
        c.kv[which][rows[-1], 0, 3] = value
        c.kv[which][rows[-(new + 1) // 2], 1, 60] = value
        c.upload()
        out, lse = c.run()
        eo, el, *_ = c.expected()
        go, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        assert np.array_equal(np.isnan(go), np.isnan(eo))
        assert np.array_equal(np.isinf(go), np.isinf(eo))
        assert np.array_equal(go[np.isinf(eo)], eo[np.isinf(eo)])
        if which == 1:
            c.check(out, lse)
        c.kv = kv


def test_long_context_few_rows_is_split():
    """One request over many workgroups, joined."""
    run("long", seed=3, new=[1], ctx=[20000], H=2, G=4, D=128, page=16)


@pytest.mark.parametrize("prefix", [0, 5000])
@pytest.mark.parametrize("new", [[1], [3, 1], [40]])
@pytest.mark.parametrize("D,H,G,pool", [(64, 1, 5, "bf16"), (128, 3, 2, "bf16"), (256, 1, 3, "bf16"),
                                        (256, 1, 3, "fp8"), (128, 1, 9, "fp8")])
def test_many_pieces(D, H, G, pool, new, prefix):
    """Few rows and long contexts: items in two to a hundred pieces, thin and
    wide, whose joins share a row among waves and workgroups."""
    say("pieces", D, H, G, pool, new, prefix)
    n = len(new)
    extra = dict(members=[0, n], prefix=[prefix]) if prefix else {}
    for own in (700, 6000):
        c = Case(24, new=new, ctx=[own, 333][:n], H=H, G=G, D=D, pool=pool, page=32, **extra)
        out, lse = c.run()
        torch.cuda.synchronize()
        c.check(out, lse)


def test_scores_that_grow():
    """Maxima that rise along the keys (the accumulators are rescaled often)
    and scores of large size."""
    say("growing scores")
    c = Case(21, new=[1, 70], ctx=[500, 400], H=2, G=4, D=64, amp=1.0)
    for r in range(2):
        rows = c.b.rows(c.b.pg_off[r], c.b.ids, c.b.ctx[r])
        ramp = torch.linspace(-6, 6, len(rows))[:, None, None]
        c.kv[0][rows] = (c.kv[0][rows].float() * ramp.abs() + ramp).to(c.kv[0].dtype)
    c.upload()
    for scale in (0.01, 0.125, 1.0):
        out, lse = c.run(scale=scale)
        c.check(out, lse, scale)


@pytest.mark.parametrize("n", [300, 513, 1100])
def test_many_requests(n):
    """More segments than one scan holds."""
    rng = np.random.default_rng(n)
    ctx = rng.integers(0, 40, n)
    new = np.minimum(ctx, rng.integers(0, 3, n))
    cuts = sorted(rng.integers(0, n + 1, 3).tolist())
    run(f"{n} requests", seed=n, new=new.tolist(), ctx=ctx.tolist(), H=1, G=2, D=64, page=4,
        members=[0, *cuts, n], prefix=[10, 0, 33, 70])


@pytest.mark.parametrize("new", [1, 80])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_small_weights(dtype, new):
    """One key of weight 1 and value 0 before 60000 of weight 2^-22.6 and value
    1: in f16 such weights would be subnormal, and all rounded alike."""
    say("small weights", dtype, new)
    n = 60000
    c = Case(19, new=[new], ctx=[n], H=1, G=1, D=64, dtype=dtype, page=64)
    rows = np.array(c.b.rows(c.b.pg_off[0], c.b.ids, n))
    k, v = (torch.zeros(n, 1, 64) for _ in range(2))
    k[:, 0, 0] = 0.335
    k[0, 0, 0] = 16.0
    v[1:] = 1.0
    c.kv[0][rows], c.kv[1][rows] = k.to(c.kv[0].dtype), v.to(c.kv[1].dtype)
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    c.upload()
    out, lse = c.run(scale=1.0, causal=False)
    torch.cuda.synchronize()
    c.check(out, lse, 1.0, False)


def test_strided_queries_and_outputs():
    """q as a slice of a fused projection, out with padded tokens: the bytes
    between are left alone."""
    say("strides")
    c = Case(8, new=[3, 1, 50], ctx=[30, 64, 90], H=2, G=4, D=64, members=[0, 3], prefix=[20])
    T, Hq, D = c.q.shape
    wide = torch.randn(T, Hq + 4, D, device=DEV).to(c.qd.dtype)
    wide[:, 2:2 + Hq] = c.qd
    room = torch.full((T + 3, Hq + 2, D), 7.0, device=DEV, dtype=c.qd.dtype)
    out = room[:T, 1:1 + Hq]
    _, lse = c.run(q=wide[:, 2:2 + Hq], out=out)
    c.check(out, lse)
    assert (room[T:] == 7).all() and (room[:, 0] == 7).all() and (room[:, -1] == 7).all()


@pytest.mark.parametrize("new", [[1, 1, 0, 1], [3, 0, 90, 2], [1, 2, 3, 0], [0, 0, 0, 0]])
@pytest.mark.parametrize("prefix", [False, True])
def test_rows_behind_the_last_request(new, prefix):
    """total_tokens beyond tok_off[num_reqs]: those rows stay as they were, and
    NaN in their queries harms nothing."""
    say("rows behind", new, prefix)
    extra = dict(members=[0, 1, 4], prefix=[40, 33]) if prefix else {}
    c = Case(18, new=new, ctx=[50, 9, 120, 3], H=2, G=4, D=64, **extra)
    T, room = sum(new), sum(new) + 7
    q = torch.full((room, 8, 64), float("nan"), dtype=c.qd.dtype, device=DEV)
    q[:T] = c.qd
    out = torch.full_like(q, 7.0)
    lse = torch.full((room, 8), 7.0, device=DEV)
    c.reqs = kvx.Requests(c.tok_off, room)
    c.run(q=q, out=out, lse=lse)
    torch.cuda.synchronize()
    assert (out[T:] == 7).all() and (lse[T:] == 7).all()
    if T:
        c.check(out[:T], lse[:T])


@pytest.mark.parametrize("new", [1, 64])
def test_results_repeat(new):
    c = Case(4, new=[new] * 6, ctx=[900, 64, 300, 77, 1024, 500], H=4, G=4, D=128, members=[0, 6],
             prefix=[700])
    a, la = c.run()
    for _ in range(3):
        b, lb = c.run()
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_without_lse_and_with_kept_workspace():
    c = Case(6, new=[1, 2], ctx=[65, 40], H=2, G=2, D=128)
    ws = torch.full((kvx.attend_workspace(c.lay, c.reqs, 4) + 64,), 255, dtype=torch.uint8, device=DEV)
    out, lse = c.run(workspace=ws)
    c.check(out, lse)
    out2 = torch.empty_like(out)
    kvx.attend(c.lay, 0, c.pool, c.reqs, c.ctx, c.table, c.qd, out2, workspace=ws)
    assert torch.equal(out, out2)
    with pytest.raises(kvx.KvxError) as e:
        c.run(workspace=ws[:1024])
    assert e.value.status == 2


def test_graph_replays_with_new_lengths():
    """One capture; lengths, tables and values change between replays."""
    say("graph")
    c = Case(50, new=[1] * 5, ctx=[100, 3, 64, 200, 31], H=2, G=4, D=64, members=[0, 2, 5],
             prefix=[90, 40])
    out, lse = torch.empty_like(c.qd), torch.empty(c.q.shape[:2], device=DEV)
    ws = torch.empty(kvx.attend_workspace(c.lay, c.reqs, 8, c.prefix), dtype=torch.uint8, device=DEV)
    c.run(out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(out=out, lse=lse, workspace=ws)
    for rep, ctx in enumerate(([100, 3, 64, 200, 31], [1, 0, 60, 111, 5], [96, 2, 1, 199, 30])):
        c.b.ctx = list(ctx)
        c.ctx.copy_(ints(ctx, torch.int32))
        c.q = torch.randn(c.q.shape).to(c.q.dtype)
        c.qd.copy_(c.q)
        out.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse)
        eager, el = c.run()
        assert torch.equal(out, eager) and torch.equal(lse, el), rep


def test_two_streams_at_once():
    a = Case(60, new=[1] * 8, ctx=[700] * 8, H=4, G=4, D=128)
    b = Case(61, new=[30] * 4, ctx=[300] * 4, H=4, G=4, D=128, members=[0, 4], prefix=[500])
    want = [c.run() for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        got.append([c.run(stream=s) for c, s in zip((a, b), streams)])
    torch.cuda.synchronize()
    for g in got:
        for (x, lx), (y, ly) in zip(g, want):
            assert torch.equal(x, y) and torch.equal(lx, ly)


def test_offsets_past_32_bits():
    """Pages whose rows lie more than 4 GiB into a plane."""
    say("large pool")
    H, D, page = 8, 128, 16
    pages = (5 << 30) // (page * H * D * 2)
    pool = torch.zeros(2, pages, page, H, D, dtype=torch.bfloat16, device=DEV)
    c = Case(70, new=[1, 20], ctx=[100, 70], H=H, G=2, D=D, members=[0, 2], prefix=[60], poison=False)
    move = pages - 1 - 7 * np.arange(c.num_pages)
    at = torch.from_numpy(move).to(DEV)
    src = c.store.view(torch.uint8).view(2, c.num_pages, page, H, D * 2)
    pool.view(torch.uint8)[:, at] = src
    lay, P = kvx.Layout(1, 2, H, D, "bf16"), kvx.Pool(pool, pages, page)
    table = kvx.Table(ints(c.b.pg_off, torch.int64), ints(move[c.b.ids], torch.int32))
    prefix = kvx.Prefix(c.prefix.grp_off, c.prefix.lens,
                        kvx.Table(c.prefix.table.pg_off, ints(move[c.b.pre_ids], torch.int32)))
    out, lse = torch.empty_like(c.qd), torch.empty(c.q.shape[:2], device=DEV)
    kvx.attend(lay, 0, P, c.reqs, c.ctx, table, c.qd, out, prefix=prefix, lse=lse)
    c.check(out, lse)


@pytest.mark.parametrize("seed", range(24))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    n = int(rng.integers(1, 9))
    most = int(rng.choice([1, 4, 90]))
    new = rng.integers(0, most + 1, n)
    new[0] = max(new[0], 1)
    ctx = new + rng.integers(0, 200, n) * rng.integers(0, 2, n)
    if rng.random() < 0.3:
        ctx[rng.integers(n)] = int(rng.integers(0, 5))
    groups = int(rng.integers(0, 3))
    kw = {}
    if groups:
        cuts = sorted(rng.integers(0, n + 1, groups - 1).tolist())
        kw = dict(members=[0, *cuts, n], prefix=rng.integers(0, 150, groups).tolist())
    pool = str(rng.choice(["", "", "fp8"]))
    run(f"random {seed}", seed=seed, new=new.tolist(), ctx=ctx.tolist(), H=int(rng.integers(1, 6)),
        G=int(rng.integers(1, 10)), D=int(rng.choice([16, 48, 64, 96, 128, 176, 256])),
        dtype=str(rng.choice(["bf16", "f16"])), pool=pool, k_scale=0.1 if pool else 1.0,
        v_scale=0.2 if pool else 1.0, page=int(rng.choice([1, 5, 16, 32])),
        layout=str(rng.choice(["nhd", "hnd"])), bad=float(rng.choice([0, 0, 0.2])),
        causal=bool(rng.random() < 0.8), **kw)


@pytest.mark.parametrize("kind", ["wide", "thin"])
@pytest.mark.parametrize("prefix", [0, 33])
@pytest.mark.parametrize("ctx", [2, 130])
def test_skipped_where_tokens_outnumber_the_context(kind, prefix, ctx):
    """More query tokens than context, in items that are cut: the page table
    behind a request's own list is no key of it, and is not counted."""
    say("skipped", kind, prefix, ctx)
    # 2000 rows of one kv head in wide tiles; 200 among 41 requests in thin ones
    new, G = ([1000, 3], 4) if kind == "wide" else ([200] + [0] * 40, 1)
    n = len(new)
    extra = dict(members=[0, n], prefix=[prefix]) if prefix else {}
    for bad in (0.0, 0.4):
        c = Case(90, new=new, ctx=[ctx] + [0] * (n - 1), H=1, G=G, D=64, bad=bad, page=4, **extra)
        skipped = torch.zeros(1, dtype=torch.int64, device=DEV)
        out, lse = c.run(skipped=skipped)
        torch.cuda.synchronize()
        c.check(out, lse)
        assert skipped.item() == c.b.skipped(), bad


@pytest.mark.parametrize("new", [1, 40])
def test_groups_equal_contexts_of_their_own(new):
    """Several groups, one of them without requests and one without a prefix:
    the prefix's pages in front of each request's own list, as one context,
    give the same sums within the bounds of both."""
    say("groups as contexts", new)
    members, prefix = [0, 2, 2, 3, 6], [48, 16, 0, 112]
    c = Case(32, new=[new, 1, new, 1, 2, new], ctx=[new + 5, 1, new, 20, 33, new + 64], H=2, G=4, D=64,
             members=members, prefix=prefix)
    b = c.b
    lists, off, ctx = [], [0], []
    for r, n in enumerate(b.ctx):
        g = b.group_of(r)
        lists += list(b.pre_ids[b.pre_off[g]:b.pre_off[g + 1]]) + list(b.ids[b.pg_off[r]:b.pg_off[r + 1]])
        off.append(len(lists))
        ctx.append(n + prefix[g])
    out, lse = c.run()
    out2, lse2 = torch.empty_like(out), torch.empty_like(lse)
    kvx.attend(c.lay, 0, c.pool, c.reqs, ints(ctx, torch.int32),
               kvx.Table(ints(off, torch.int64), ints(lists, torch.int32)), c.qd, out2, lse=lse2)
    torch.cuda.synchronize()
    c.check(out, lse)
    c.check(out2, lse2)


@pytest.mark.parametrize("new", [[1], [3, 1, 50]])
def test_queries_and_outputs_of_one_buffer(new):
    """q and out as slices of one fused buffer do not overlap; outputs that
    share a byte with a query are refused and nothing is written."""
    say("one buffer", new)
    n, T, Hq, D = len(new), sum(new), 8, 64
    c = Case(9, new=new, ctx=[30, 64, 90][:n], H=2, G=4, D=D, members=[0, n], prefix=[20])
    for q_at, out_at in ((0, Hq), (Hq + 2, 1)):
        fused = torch.full((T, 2 * Hq + 3, D), 7.0, device=DEV, dtype=c.qd.dtype)
        q, out = fused[:, q_at:q_at + Hq], fused[:, out_at:out_at + Hq]
        q.copy_(c.qd)
        _, lse = c.run(q=q, out=out)
        torch.cuda.synchronize()
        c.check(out, lse)
        rest = [h for h in range(2 * Hq + 3) if not out_at <= h < out_at + Hq]
        before = fused[:, rest].clone()
        c.run(q=q, out=out)
        assert torch.equal(fused[:, rest], before) and torch.equal(q, c.qd)
    for out_at in (Hq - 1, Hq + 3, Hq + 2):
        before = fused.clone()
        with pytest.raises(kvx.KvxError) as e:
            c.run(q=q, out=fused[:, out_at:out_at + Hq])
        assert e.value.status == 9
        torch.cuda.synchronize()
        assert torch.equal(fused, before)


@pytest.mark.parametrize("new", [1, 40])
def test_largest_values(new):
    """bf16 values at the size that the sums' range allows for (2^119 over the
    keys seen), with scores that rise along the keys past the first maximum."""
    say("largest values", new)
    n = 96
    c = Case(33, new=[new], ctx=[n], H=2, G=4, D=64, page=16)
    rows = c.b.rows(c.b.pg_off[0], c.b.ids, n)
    c.q = torch.ones_like(c.q)
    k = torch.zeros(n, 2, 64)
    k[:, :, 0] = torch.linspace(0, 5.4, n)[:, None]
    c.kv[0][rows] = k.to(c.kv[0].dtype)
    sign = torch.where(torch.rand(n, 2, 64, generator=torch.Generator().manual_seed(1)) < 0.9, 1.0, -1.0)
    c.kv[1][rows] = (sign * 2.0 ** 119 / 128).to(c.kv[1].dtype)
    c.upload()
    out, lse = c.run(scale=1.0, causal=False)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all()
    c.check(out, lse, 1.0, False)
