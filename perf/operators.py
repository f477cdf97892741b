"""The serving operators on real work: page tables and slot maps from request lengths
(build_tables), new K/V rows written into a paged pool (append), and attention over a paged pool
for requests that share prefixes (attend).  Each case has a plain torch form; with ``own`` set the
same inputs go through the framework's calls."""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "fp8": torch.float8_e4m3fn}
FP8_MAX = 448.0


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # one decode step of a batch of 64 at about 2000 tokens each: one new token per request,
        # few new pages; what counts is latency
        {"name": "tables_decode_64", "op": "tables", "reqs": 64, "page": 16, "have_lo": 1,
         "have_hi": 4096, "add_lo": 1, "add_hi": 1, "lens": 1},
        # the prompts of 32 requests of 1024 to 2048 tokens entering a token-paged pool
        {"name": "tables_prompts_page1", "op": "tables", "reqs": 32, "page": 1, "have_lo": 0,
         "have_hi": 0, "add_lo": 1024, "add_hi": 2048, "lens": 2},
        # a large mixed step: 2048 requests, chunks of prompts beside single tokens
        {"name": "tables_mixed_2048", "op": "tables", "reqs": 2048, "page": 16, "have_lo": 0,
         "have_hi": 8191, "add_lo": 0, "add_hi": 255, "lens": 3},
        # the new rows of one layer in a decode step of 64 requests
        {"name": "append_decode_64", "op": "append", "tokens": 64, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "pool": "bf16", "page": 16, "layout": "nhd", "rows": 65536},
        # one layer of 8192 prompt tokens quantised into head-major blocks
        {"name": "append_fp8_hnd_8192", "op": "append", "tokens": 8192, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "pool": "fp8", "page": 16, "layout": "hnd", "rows": 65536},
        # one layer of the 49152 tokens of a batch of prompts, 4-head rows, token-paged
        {"name": "append_49152_page1", "op": "append", "tokens": 49152, "kv_heads": 4, "dim": 128,
         "dtype": "f16", "pool": "f16", "page": 1, "layout": "nhd", "rows": 131072},
        # four short chats behind one system prompt, 2 kv heads of 6 query heads, token-paged
        {"name": "attend_4_short", "op": "attend", "reqs": 4, "groups": 1, "kv_heads": 2,
         "group": 6, "dim": 128, "dtype": "f16", "pool": "f16", "page": 1, "layout": "nhd",
         "prefix_lo": 256, "prefix_hi": 256, "own_lo": 1, "own_hi": 64, "new_lo": 1, "new_hi": 1,
         "lens": 4},
        # the ordinary decode step: 64 requests, 2048 shared tokens, some hundreds of their own
        {"name": "attend_64_decode", "op": "attend", "reqs": 64, "groups": 1, "kv_heads": 8,
         "group": 4, "dim": 128, "dtype": "bf16", "pool": "bf16", "page": 16, "layout": "nhd",
         "prefix_lo": 2048, "prefix_hi": 2048, "own_lo": 128, "own_hi": 1024, "new_lo": 1,
         "new_hi": 1, "lens": 5},
        # a quantised cache in head-major blocks
        {"name": "attend_128_fp8_hnd", "op": "attend", "reqs": 128, "groups": 1, "kv_heads": 8,
         "group": 4, "dim": 128, "dtype": "bf16", "pool": "fp8", "page": 16, "layout": "hnd",
         "prefix_lo": 4001, "prefix_hi": 4001, "own_lo": 512, "own_hi": 2048, "new_lo": 1,
         "new_hi": 1, "lens": 6},
        # eight prompts with some requests behind each, heads of 64, one query head per kv head
        {"name": "attend_8_groups_d64", "op": "attend", "reqs": 61, "groups": 8, "kv_heads": 8,
         "group": 1, "dim": 64, "dtype": "f16", "pool": "f16", "page": 16, "layout": "nhd",
         "prefix_lo": 500, "prefix_hi": 2000, "own_lo": 1, "own_hi": 700, "new_lo": 1,
         "new_hi": 3, "lens": 7},
        # chunks of prompts behind one long shared document: many query rows, causal at the end
        {"name": "attend_8_chunks", "op": "attend", "reqs": 8, "groups": 1, "kv_heads": 8,
         "group": 4, "dim": 128, "dtype": "bf16", "pool": "bf16", "page": 16, "layout": "nhd",
         "prefix_lo": 4096, "prefix_hi": 4096, "own_lo": 200, "own_hi": 512, "new_lo": 100,
         "new_hi": 256, "lens": 8},
        # the largest batch: 256 requests behind 8192 shared tokens
        {"name": "attend_256_long", "op": "attend", "reqs": 256, "groups": 1, "kv_heads": 8,
         "group": 8, "dim": 128, "dtype": "bf16", "pool": "bf16", "page": 16, "layout": "nhd",
         "prefix_lo": 8192, "prefix_hi": 8192, "own_lo": 256, "own_hi": 2048, "new_lo": 1,
         "new_hi": 1, "lens": 9},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend"])
    lens = rng.randrange(1 << 30)
    page = rng.choice([1, 2, 16, 16, 32, 64])
    if op == "tables":
        reqs = _spread(rng, 1, 2048)
        have = rng.choice([0, _spread(rng, 1, 8191)])
        add = rng.choice([1, _spread(rng, 1, max(1, min(2048, 500000 // reqs)))])
        return {"op": op, "reqs": reqs, "page": page, "have_lo": min(have, 1), "have_hi": have,
                "add_lo": rng.choice([0, 1]), "add_hi": add, "lens": lens}
    if op == "append":
        tokens = _spread(rng, 1, 49152)
        dtype = rng.choice(["bf16", "f16"])
        rows = _spread(rng, tokens + 64, 131072) // page * page + page
        return {"op": op, "tokens": tokens, "kv_heads": rng.choice([1, 2, 4, 5, 8]),
                "dim": rng.choice([64, 128]), "dtype": dtype, "pool": rng.choice([dtype, "fp8"]),
                "page": page, "layout": rng.choice(["nhd", "hnd"]), "rows": rows}
    dtype = rng.choice(["bf16", "f16"])
    new = rng.choice([1, 1, _spread(rng, 1, 256)])
    reqs = _spread(rng, 1, 256 if new == 1 else max(1, 2048 // new))
    groups = min(reqs, rng.choice([1, 1, 2, 8]))
    prefix = rng.choice([0, _spread(rng, 1, 8192 // groups), _spread(rng, 64, 8192 // groups)])
    own_hi = max(new, _spread(rng, 1, 2048))
    return {"op": op, "reqs": reqs, "groups": groups, "kv_heads": rng.choice([1, 2, 4, 8]),
            "group": rng.choice([1, 2, 4, 5, 6, 8]), "dim": rng.choice([64, 128]),
            "dtype": dtype, "pool": rng.choice([dtype, dtype, "fp8"]), "page": page,
            "layout": rng.choice(["nhd", "nhd", "hnd"]),
            "prefix_lo": prefix // 2, "prefix_hi": prefix, "own_lo": min(new, own_hi),
            "own_hi": own_hi, "new_lo": 1, "new_hi": new, "lens": lens}


def _lengths(case):
    """The batch's lengths: of the case alone, so that every seed has the same work."""
    r = random.Random(case["lens"])
    if case["op"] == "tables":
        have = [r.randint(case["have_lo"], case["have_hi"]) for _ in range(case["reqs"])]
        add = [r.randint(case["add_lo"], case["add_hi"]) for _ in range(case["reqs"])]
        add[0] = max(add[0], 1)
        return have, add
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["reqs"])]
    ctx = [max(n, r.randint(case["own_lo"], case["own_hi"])) for n in new]
    prefix = [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case["groups"])]
    cuts = sorted(r.sample(range(1, case["reqs"]), case["groups"] - 1))
    members = [0] + cuts + [case["reqs"]]
    return new, ctx, prefix, members


def _pages(n, page):
    return -(-n // page)


def _offsets(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return off


# ----------------------------------------------------------------- inputs --

def _ints(values, dtype):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _normal(shape, dtype, gen, scale=1.0):
    x = torch.randn(shape, device=DEV, generator=gen) * scale
    return x.clamp(-FP8_MAX, FP8_MAX).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _pool_shape(case, pages):
    h, d, b = case["kv_heads"], case["dim"], case["page"]
    return (2, pages, b, h, d) if case["layout"] == "nhd" else (2, pages, h, b, d)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 1000003 + 17)
    s = {"case": dict(case)}
    page = case["page"]
    if case["op"] == "tables":
        have, add = _lengths(case)
        n = case["reqs"]
        held = [_pages(h, page) for h in have]
        total = [_pages(h + a, page) for h, a in zip(have, add)]
        # every page of a pool in a random order: the held ones first, the free list behind them
        ids = torch.randperm(sum(total) + 4096, device=DEV, generator=gen).to(torch.int32)
        s.update(have=_ints(have, torch.int32), add=_ints(add, torch.int32),
                 held_off=_ints(_offsets(held), torch.int64), held_ids=ids[:sum(held)].clone(),
                 free=ids[sum(held):].clone(), tokens=sum(add), pages=sum(total))
        if own:     # the output buffers that a serving loop keeps
            import scatter_kvx_gather_amd as kvx
            s["out"] = kvx.BatchTables(n, s["tokens"], s["pages"], device=DEV)
            s["held"] = kvx.Table(s["held_off"], s["held_ids"])
        return s
    dtype, pool_t = DTYPES[case["dtype"]], DTYPES[case["pool"]]
    h, d = case["kv_heads"], case["dim"]
    scales = (0.03, 0.05) if case["pool"] == "fp8" else (1.0, 1.0)
    s["k_scale"], s["v_scale"] = scales
    if case["op"] == "append":
        pages, t = case["rows"] // page, case["tokens"]
        s["pool"] = torch.zeros(_pool_shape(case, pages), dtype=torch.uint8, device=DEV) \
            .view(pool_t) if case["pool"] == "fp8" else \
            torch.zeros(_pool_shape(case, pages), dtype=pool_t, device=DEV)
        s["slots"] = torch.randperm(pages * page, device=DEV, generator=gen)[:t].contiguous()
        # K and V as slices of a fused projection's output rows
        qkv = _normal((t, 4 * h, d), dtype, gen)
        s["k"], s["v"] = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
    else:
        new, ctx, prefix, members = _lengths(case)
        need = sum(_pages(c, page) for c in ctx) + sum(_pages(p, page) for p in prefix)
        pages = need + need // 4 + 1
        hq = h * case["group"]
        kv = [_normal(_pool_shape(case, pages)[1:], torch.float32, gen) for _ in range(2)]
        s["pool"] = torch.stack([(x / c).clamp(-FP8_MAX, FP8_MAX).to(pool_t) if case["pool"] == "fp8"
                                 else x.to(pool_t) for x, c in zip(kv, scales)])
        del kv
        ids = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
        pre_off = _offsets([_pages(p, page) for p in prefix])
        s.update(q=_normal((sum(new), hq, d), dtype, gen), scale=d ** -0.5,
                 tok_off=_ints(_offsets(new), torch.int64), ctx=_ints(ctx, torch.int32),
                 pg_off=_ints(_offsets([_pages(c, page) for c in ctx]), torch.int64),
                 ids=ids[pre_off[-1]:].clone(), members=_ints(members, torch.int64),
                 prefix=_ints(prefix, torch.int32), pre_off=_ints(pre_off, torch.int64),
                 pre_ids=ids[:max(pre_off[-1], 1)].clone(), max_new=max(new), max_ctx=max(ctx),
                 max_prefix=max(prefix), tokens=sum(new),
                 max_rows=max(sum(new[a:b]) for a, b in zip(members, members[1:])))
    if own:         # the descriptors of pool and batch, and the workspace, that a user's program keeps
        import scatter_kvx_gather_amd as kvx
        es = s["pool"].element_size()
        s["kvx"] = {"layout": kvx.Layout(1, 2, h, d, case["pool"]),
                    "pool": kvx.Pool(s["pool"], pages, page, slot_stride=h * d * es)}
        if case["op"] == "attend":
            s["kvx"].update(
                reqs=kvx.Requests(s["tok_off"], s["tokens"]), table=kvx.Table(s["pg_off"], s["ids"]),
                prefix=kvx.Prefix(s["members"], s["prefix"], kvx.Table(s["pre_off"], s["pre_ids"])))
            s["kvx"]["workspace"] = torch.empty(
                kvx.attend_workspace(s["kvx"]["layout"], s["kvx"]["reqs"], hq,
                                     prefix=s["kvx"]["prefix"]), dtype=torch.uint8, device=DEV)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
    return s


# -------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "attend": _own_attend}[op](s)
    return {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend}[op](s)


def _own_tables(s):
    import scatter_kvx_gather_amd as kvx
    o = s["out"]
    kvx.build_tables(o, s["case"]["page"], s["add"], s["free"], have_len=s["have"], held=s["held"])
    return {"ctx": o.ctx_len, "tok_off": o.tok_off, "pg_off": o.pg_off, "ids": o.page_ids,
            "slots": o.slots, "totals": o.totals}


def _own_append(s):
    import scatter_kvx_gather_amd as kvx
    c, x = s["case"], s["kvx"]
    kvx.append(x["layout"], 0, x["pool"], s["slots"], s["k"], s["v"], k_scale=s["k_scale"],
               v_scale=s["v_scale"], block_layout=c["layout"])
    return {"pool": s["pool"]}


def _own_attend(s):
    import scatter_kvx_gather_amd as kvx
    c, x = s["case"], s["kvx"]
    kvx.attend(x["layout"], 0, x["pool"], x["reqs"], s["ctx"], x["table"], s["q"], s["out"],
               prefix=x["prefix"], lse=s["lse"], scale=s["scale"], k_scale=s["k_scale"],
               v_scale=s["v_scale"], block_layout=c["layout"], workspace=x["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _before(counts):
    """Exclusive prefix sums with the total behind them."""
    return torch.nn.functional.pad(torch.cumsum(counts, 0), (1, 0))


def _plain_tables(s):
    b, n = s["case"]["page"], s["case"]["reqs"]
    have, add = s["have"].long(), s["add"].long()
    ctx = have + add
    pages, held = (ctx + b - 1) // b, (have + b - 1) // b
    tok_off, pg_off, new_off = _before(add), _before(pages), _before(pages - held)
    at = torch.arange(n, device=DEV)
    r = torch.repeat_interleave(at, pages, output_size=s["pages"])
    k = torch.arange(s["pages"], device=DEV) - pg_off[r]
    taken = s["free"][(new_off[r] + k - held[r]).clamp(min=0)]
    if s["held_ids"].numel():
        last = s["held_ids"].numel() - 1
        ids = torch.where(k < held[r], s["held_ids"][(s["held_off"][r] + k).clamp(max=last)], taken)
    else:
        ids = taken
    r = torch.repeat_interleave(at, add, output_size=s["tokens"])
    t = have[r] + torch.arange(s["tokens"], device=DEV) - tok_off[r]
    slots = ids[pg_off[r] + t // b].long() * b + t % b
    totals = torch.stack([tok_off[-1], pg_off[-1], new_off[-1], torch.zeros_like(tok_off[-1])])
    return {"ctx": ctx.to(torch.int32), "tok_off": tok_off, "pg_off": pg_off, "ids": ids,
            "slots": slots, "totals": totals}


def _plain_append(s):
    c = s["case"]
    b = c["page"]
    for plane, x, scale in ((s["pool"][0], s["k"], s["k_scale"]), (s["pool"][1], s["v"], s["v_scale"])):
        if c["pool"] == "fp8":
            x = (x.float() / scale).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
            x, plane = x.view(torch.uint8), plane.view(torch.uint8)
        if c["layout"] == "nhd":
            plane.view(-1, c["kv_heads"], c["dim"])[s["slots"]] = x
        else:
            plane[s["slots"] // b, :, s["slots"] % b] = x
    return {"pool": s["pool"]}


def _rows(plane, ids, off, count, most, case, scale):
    """[lists, heads, most, dim] in 32 bits: the first `most` rows of every list of pages."""
    b = case["page"]
    pos = torch.arange(max(most, 1), device=DEV)
    pos = torch.minimum(pos[None], (count[:, None] - 1).clamp(min=0))
    pages = ids[(off[:-1, None] + pos // b).clamp(max=ids.numel() - 1)].long()
    fp8 = plane.dtype == torch.float8_e4m3fn
    x = plane.view(torch.uint8) if fp8 else plane
    x = x[pages, pos % b] if case["layout"] == "nhd" else x[pages, :, pos % b]
    x = x.view(torch.float8_e4m3fn).float() * scale if fp8 else x.float()
    return x.transpose(1, 2).contiguous()


def _part(q, k, v, seen):
    """max, sum and weighted values of one part's softmax; q [lists, heads, rows, dim]."""
    x = torch.matmul(q, k.transpose(2, 3).contiguous())
    x = x.masked_fill(~seen, -math.inf)
    top = x.amax(3, keepdim=True)
    p = torch.exp(x - top.clamp(min=-1e30))
    return top, p.sum(3, keepdim=True), torch.matmul(p, v)


def _plain_attend(s):
    c = s["case"]
    h, g, d, t = c["kv_heads"], c["group"], c["dim"], s["tokens"]
    q = s["q"].float().view(t, h, g, d) * s["scale"]
    at = torch.arange(t, device=DEV)
    req = torch.searchsorted(s["tok_off"], at, right=True) - 1
    grp = torch.searchsorted(s["members"], req, right=True) - 1

    def lists(first, count, most):
        """Rows of q as [lists, heads, most * group, dim]."""
        i = (first[:, None] + torch.arange(most, device=DEV)[None]).clamp(max=t - 1)
        return q[i].permute(0, 2, 1, 3, 4).reshape(first.numel(), h, most * g, d)

    def tokens(x, which, inside, most):
        """[lists, heads, most * group, n] back to [tokens, heads, group, n]."""
        return x.view(x.shape[0], h, most, g, -1)[which, :, inside]

    new, ctx = s["tok_off"].diff(), s["ctx"].long()
    k, v = (_rows(s["pool"][j], s["ids"], s["pg_off"], ctx, s["max_ctx"], c, s[w])
            for j, w in ((0, "k_scale"), (1, "v_scale")))
    row = torch.arange(s["max_new"] * g, device=DEV) // g
    last = (ctx - new)[:, None] + row[None]                       # the last key that a row sees
    seen = torch.arange(k.shape[2], device=DEV)[None, None] <= last[:, :, None]
    seen = seen & (torch.arange(k.shape[2], device=DEV) < ctx[:, None, None])
    parts = [[tokens(x, req, at - s["tok_off"][req], s["max_new"])
              for x in _part(lists(s["tok_off"][:-1], new, s["max_new"]), k, v, seen[:, None])]]
    if s["max_prefix"]:
        first = s["tok_off"][s["members"]]
        count = s["prefix"].long()
        k, v = (_rows(s["pool"][j], s["pre_ids"], s["pre_off"], count, s["max_prefix"], c, s[w])
                for j, w in ((0, "k_scale"), (1, "v_scale")))
        seen = torch.arange(k.shape[2], device=DEV)[None] < count[:, None]
        parts.append([tokens(x, grp, at - first[grp], s["max_rows"])
                      for x in _part(lists(first[:-1], first.diff(), s["max_rows"]), k, v,
                                     seen[:, None, None])])
    top = torch.stack([p[0] for p in parts]).amax(0)
    weight = [torch.exp(p[0] - top.clamp(min=-1e30)) for p in parts]
    total = sum(w * p[1] for w, p in zip(weight, parts))
    out = sum(w * p[2] for w, p in zip(weight, parts)) / total.clamp(min=1e-30)
    lse = top + torch.log(total)
    return {"out": out.reshape(t, h * g, d).to(s["q"].dtype), "lse": lse.reshape(t, h * g)}


# ------------------------------------------------------------------- work --

def work(case):
    page = case["page"]
    if case["op"] == "tables":
        have, add = _lengths(case)
        n = len(have)
        pages = sum(_pages(h + a, page) for h, a in zip(have, add))
        return {"bytes": 8 * n + 4 * pages + 4 * n + 16 * (n + 1) + 4 * pages + 8 * sum(add),
                "flops": 0}
    size = {"bf16": 2, "f16": 2, "fp8": 1}
    row = case["kv_heads"] * case["dim"]
    if case["op"] == "append":
        return {"bytes": case["tokens"] * (2 * row * (size[case["dtype"]] + size[case["pool"]]) + 8),
                "flops": 0}
    new, ctx, prefix, members = _lengths(case)
    hq = case["kv_heads"] * case["group"]
    keys = sum(ctx) + sum(prefix)
    ids = sum(_pages(x, page) for x in ctx + prefix)
    seen = 0
    for g, p in enumerate(prefix):
        for n, c in zip(new[members[g]:members[g + 1]], ctx[members[g]:members[g + 1]]):
            seen += n * (p + c) - n * (n - 1) // 2
    tokens = sum(new)
    return {"bytes": 2 * keys * row * size[case["pool"]] + 4 * ids
            + tokens * hq * (2 * case["dim"] * size[case["dtype"]] + 4),
            "flops": 4 * case["dim"] * hq * seen}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "append": _exact_append, "attend": _exact_attend}[case["op"]](case, s)


def _exact_tables(case, s):
    """Request by request with whole numbers on the host."""
    b = case["page"]
    have, add, free = s["have"].tolist(), s["add"].tolist(), s["free"].tolist()
    held, held_off = s["held_ids"].tolist(), s["held_off"].tolist()
    ids, slots, tok_off, pg_off, used = [], [], [0], [0], 0
    for r, (x, y) in enumerate(zip(have, add)):
        mine = held[held_off[r]:held_off[r + 1]]
        while len(mine) * b < x + y:
            mine.append(free[used])
            used += 1
        slots += [mine[t // b] * b + t % b for t in range(x, x + y)]
        ids += mine
        tok_off.append(len(slots))
        pg_off.append(len(ids))
    return {"ctx": torch.tensor([x + y for x, y in zip(have, add)], dtype=torch.int32),
            "tok_off": torch.tensor(tok_off), "pg_off": torch.tensor(pg_off),
            "ids": torch.tensor(ids, dtype=torch.int32), "slots": torch.tensor(slots),
            "totals": torch.tensor([len(slots), len(ids), used, 0])}


def _exact_append(case, s):
    """The pool in 64 bits, each row as it would be held without rounding."""
    rows = s["pool"].view(torch.uint8).double() if case["pool"] == "fp8" else s["pool"].double()
    page, row = s["slots"].div(case["page"], rounding_mode="floor"), s["slots"].remainder(case["page"])
    for j, (x, scale) in enumerate(((s["k"], s["k_scale"]), (s["v"], s["v_scale"]))):
        x = x.double()
        if case["pool"] == "fp8":
            x = (x / scale).clamp(-FP8_MAX, FP8_MAX)
        if case["layout"] == "hnd":
            rows[j].transpose(1, 2)[page, row] = x
        else:
            rows[j][page, row] = x
    return {"pool": rows}


def _exact_attend(case, s):
    """Request by request in 64 bits: one softmax over prefix and own keys."""
    b, g, d = case["page"], case["group"], case["dim"]
    pool = s["pool"].transpose(2, 3) if case["layout"] == "hnd" else s["pool"]

    def rows(ids, off, i, n, j, scale):
        first = int(off[i])
        pages = ids[first:first + _pages(n, b)].long()
        x = pool[j].view(torch.uint8)[pages].contiguous().view(pool.dtype) \
            if case["pool"] == "fp8" else pool[j][pages]
        return x.double().reshape(-1, case["kv_heads"], d)[:n].permute(1, 0, 2) * scale

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    members, prefix = s["members"].tolist(), s["prefix"].tolist()
    tok, ctx, off = s["tok_off"].tolist(), s["ctx"].tolist(), s["pg_off"].tolist()
    pre_off = s["pre_off"].tolist()
    for i, p in enumerate(prefix):
        shared = [rows(s["pre_ids"], pre_off, i, p, j, s[w]) for j, w in ((0, "k_scale"), (1, "v_scale"))]
        for r in range(members[i], members[i + 1]):
            n = tok[r + 1] - tok[r]
            k, v = (torch.cat([shared[j], rows(s["ids"], off, r, ctx[r], j, s[w])], 1)
                    for j, w in ((0, "k_scale"), (1, "v_scale")))
            q = s["q"][tok[r]:tok[r + 1]].double().view(n, -1, g, d).permute(1, 2, 0, 3)
            x = torch.matmul(q.reshape(-1, g * n, d), k.transpose(1, 2).contiguous()) * s["scale"]
            edge = p + ctx[r] - n + torch.arange(n, device=DEV).repeat(g)
            x[:, torch.arange(p + ctx[r], device=DEV)[None] > edge[:, None]] = -math.inf
            z = torch.logsumexp(x, 2)
            y = torch.matmul(torch.exp(x - z[..., None]), v)
            out[tok[r]:tok[r + 1]] = y.view(-1, g, n, d).permute(2, 0, 1, 3).reshape(n, -1, d)
            lse[tok[r]:tok[r + 1]] = z.view(-1, g, n).permute(2, 0, 1).reshape(n, -1)
    return {"out": out, "lse": lse}
