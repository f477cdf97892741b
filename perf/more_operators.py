"""A paged KV cache held in 4 bits, on real work: rows quantised as they are written and read back
(store: append, then read), rows of a held cache read back alone (read), and attention over it
(attend).  Each case has a plain torch form; with ``own`` set the same inputs go through the
framework's calls.

A row of a 4-bit pool holds, for each kv head, dim / 2 bytes of e2m1 numbers (dim 2 i in the low half
of byte i) and dim / 32 scale bytes s, one for each 32 dims, which stand for 2^(s - 127); all heads'
numbers come first, then all scales, and the row is padded to 16 bytes.  Head-major blocks hold a
page's numbers as [heads][rows][dim / 2] and behind them its scales as [heads][rows][dim / 32].  A
block of 32 holds the 32-bit quotients of its values by the tensor's scale: with the smallest power
of two 2^e that leaves the largest magnitude at most 7 * 2^e, -23 <= e <= 13, each is the nearest of
0, 0.5, 1, 1.5, 2, 3, 4, 6 times 2^e (ties to the number whose last bit is 0)."""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32,
          "fp8": torch.float8_e4m3fn}
FP8_MAX = 448.0
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # the new rows of one layer in a decode step of 64 requests, and the cache's values of them:
        # two small launches, latency
        {"name": "store_decode_64", "op": "store", "tokens": 64, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "page": 16, "layout": "nhd", "rows": 65536, "scale": 1.0},
        # one layer of 8192 prompt tokens, quantised into head-major blocks under a tensor's scale
        {"name": "store_8192_hnd_scaled", "op": "store", "tokens": 8192, "kv_heads": 8, "dim": 64,
         "dtype": "f16", "page": 16, "layout": "hnd", "rows": 65536, "scale": 0.75},
        # one layer of the 49152 tokens of a batch of prompts, token-paged
        {"name": "store_49152_page1", "op": "store", "tokens": 49152, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "page": 1, "layout": "nhd", "rows": 131072, "scale": 1.0},
        # one request's context of 2001 tokens read back, rows of a shard with 2 heads
        {"name": "read_2001_h2", "op": "read", "tokens": 2001, "kv_heads": 2, "dim": 128,
         "dtype": "f16", "pool": "fp4", "page": 32, "layout": "nhd", "rows": 65536, "scale": 1.0},
        # 65536 tokens of a head-major cache, to be held at 16 bits elsewhere
        {"name": "read_65536_hnd", "op": "read", "tokens": 65536, "kv_heads": 8, "dim": 128,
         "dtype": "bf16", "pool": "fp4", "page": 16, "layout": "hnd", "rows": 131072, "scale": 1.0},
        # four short chats, 2 kv heads of 6 query heads, token-paged
        {"name": "attend_4_short", "op": "attend", "reqs": 4, "groups": 0, "kv_heads": 2,
         "group": 6, "dim": 128, "dtype": "f16", "page": 1, "layout": "nhd", "prefix_lo": 0,
         "prefix_hi": 0, "own_lo": 1, "own_hi": 300, "new_lo": 1, "new_hi": 1, "lens": 4,
         "scale": 1.0},
        # the ordinary decode step: 64 requests of some thousand tokens each
        {"name": "attend_64_decode", "op": "attend", "reqs": 64, "groups": 0, "kv_heads": 8,
         "group": 4, "dim": 128, "dtype": "bf16", "page": 16, "layout": "nhd", "prefix_lo": 0,
         "prefix_hi": 0, "own_lo": 512, "own_hi": 4096, "new_lo": 1, "new_hi": 1, "lens": 5,
         "scale": 1.0},
        # one request that continues a document of 131071 tokens, in head-major blocks
        {"name": "attend_1_long_hnd", "op": "attend", "reqs": 1, "groups": 0, "kv_heads": 8,
         "group": 4, "dim": 128, "dtype": "bf16", "page": 64, "layout": "hnd", "prefix_lo": 0,
         "prefix_hi": 0, "own_lo": 131071, "own_hi": 131071, "new_lo": 1, "new_hi": 1, "lens": 6,
         "scale": 1.0},
        # eight prompts with some requests behind each, heads of 64, one query head per kv head,
        # one to three new tokens a request, under a tensor's scale
        {"name": "attend_8_groups_d64", "op": "attend", "reqs": 61, "groups": 8, "kv_heads": 8,
         "group": 1, "dim": 64, "dtype": "f16", "page": 16, "layout": "nhd", "prefix_lo": 500,
         "prefix_hi": 2000, "own_lo": 3, "own_hi": 700, "new_lo": 1, "new_hi": 3, "lens": 7,
         "scale": 0.75},
        # chunks of prompts behind one long shared document: many query rows, causal at the end
        {"name": "attend_8_chunks", "op": "attend", "reqs": 8, "groups": 1, "kv_heads": 8,
         "group": 8, "dim": 128, "dtype": "bf16", "page": 16, "layout": "nhd", "prefix_lo": 8192,
         "prefix_hi": 8192, "own_lo": 256, "own_hi": 512, "new_lo": 100, "new_hi": 256, "lens": 8,
         "scale": 1.0},
        # the largest batch: 256 requests, each with up to 8192 tokens of its own
        {"name": "attend_256_long", "op": "attend", "reqs": 256, "groups": 0, "kv_heads": 8,
         "group": 8, "dim": 128, "dtype": "bf16", "page": 16, "layout": "nhd", "prefix_lo": 0,
         "prefix_hi": 0, "own_lo": 256, "own_hi": 8192, "new_lo": 1, "new_hi": 1, "lens": 9,
         "scale": 1.0},
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(["store", "read", "attend", "attend"])
    page = rng.choice([1, 2, 16, 16, 32, 64])
    layout = rng.choice(["nhd", "nhd", "hnd"])
    dim = rng.choice([64, 96, 128, 128, 256])
    scale = rng.choice([1.0, 1.0, 0.75])
    if op != "attend":
        tokens = _spread(rng, 1, 49152 * 128 // max(dim, 128))
        rows = _spread(rng, tokens + 64, 131072) // page * page + page
        case = {"op": op, "tokens": tokens, "kv_heads": rng.choice([1, 2, 4, 5, 8]), "dim": dim,
                "dtype": rng.choice(["bf16", "f16"] if op == "read" else ["bf16", "f16", "f32"]),
                "page": page, "layout": layout, "rows": rows, "scale": scale}
        if op == "read":
            case["pool"] = rng.choice(["fp4", "fp4", "fp8", case["dtype"]])
            case["scale"] = 1.0 if case["pool"] == case["dtype"] else scale
        return case
    new = rng.choice([1, 1, _spread(rng, 2, 256)])
    reqs = _spread(rng, 1, 256 if new == 1 else max(1, 1024 // new))
    groups = min(reqs, rng.choice([0, 0, 1, 8]))
    prefix = _spread(rng, 1, 8192 // groups) if groups else 0
    own_hi = max(new, _spread(rng, 1, 8192 * 128 // max(dim, 128) if new == 1 else 1024))
    return {"op": op, "reqs": reqs, "groups": groups, "kv_heads": rng.choice([1, 2, 4, 8]),
            "group": rng.choice([1, 2, 4, 5, 6, 8]), "dim": dim,
            "dtype": rng.choice(["bf16", "f16"]), "page": page, "layout": layout,
            "prefix_lo": prefix // 2, "prefix_hi": prefix, "own_lo": min(new, own_hi),
            "own_hi": own_hi, "new_lo": 1, "new_hi": new, "lens": rng.randrange(1 << 30),
            "scale": scale}


def _lengths(case):
    """The batch's lengths: of the case alone, so that every seed has the same work."""
    r = random.Random(case["lens"])
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["reqs"])]
    ctx = [max(n, r.randint(case["own_lo"], case["own_hi"])) for n in new]
    prefix = [r.randint(case["prefix_lo"], case["prefix_hi"]) for _ in range(case["groups"])]
    cuts = sorted(r.sample(range(1, case["reqs"]), case["groups"] - 1)) if case["groups"] else []
    return new, ctx, prefix, [0] + cuts + [case["reqs"]]


def _pages(n, page):
    return -(-n // page)


def _offsets(counts):
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    return off


# ---------------------------------------------------------------- the pool --

def _row_bytes(case, pool):
    n = case["kv_heads"] * case["dim"]
    return {"fp4": _pages(n * 17 // 32, 16) * 16, "fp8": n}.get(pool, 2 * n)


def _views(pool, case):
    """Numbers and scales of a 4-bit pool [2, pages, bytes] as [2, pages, rows, heads, ..] views."""
    b, h, d = case["page"], case["kv_heads"], case["dim"]
    if case["layout"] == "nhd":
        x = pool.view(2, -1, b, pool.shape[2] // b)
        return (x[..., :h * d // 2].unflatten(-1, (h, d // 2)),
                x[..., h * d // 2:h * d // 2 + h * d // 32].unflatten(-1, (h, d // 32)))
    n = b * h * d // 2
    return (pool[..., :n].unflatten(-1, (h, b, d // 2)).transpose(2, 3),
            pool[..., n:n + b * h * d // 32].unflatten(-1, (h, b, d // 32)).transpose(2, 3))


def _quantise(x):
    """Bytes of numbers and of scales of x [.., dim] (32 bits, finite)."""
    y = x.unflatten(-1, (-1, 32))
    top = y.abs().amax(-1, keepdim=True)
    mantissa, power = torch.frexp(top)                     # top = mantissa * 2^power, 1/2 <= mantissa < 1
    e = (power - 3 + (mantissa > 0.875)).clamp(-23, 13)
    e = torch.where(top > 0, e, torch.full_like(e, -23))
    z = torch.ldexp(y, -e)
    a = z.abs()
    # how many of the borders between neighbours lie below, where ties go to the even number
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(z).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (e + 127).to(torch.uint8).squeeze(-1)


def _values(numbers, scales):
    """The values in 32 bits that numbers [.., dim / 2] and scales [.., dim / 32] stand for."""
    table = torch.tensor(GRID + [-g for g in GRID], dtype=torch.float32, device=DEV)
    code = torch.stack([numbers & 15, numbers >> 4], -1).flatten(-2)
    x = table[code.int()].unflatten(-1, (-1, 32))
    return torch.ldexp(x, scales.int()[..., None] - 127).flatten(-2)


# ----------------------------------------------------------------- inputs --

def _ints(values, dtype):
    return torch.tensor(values, dtype=dtype, device=DEV)


def _normal(shape, gen):
    return torch.randn(shape, device=DEV, generator=gen)


def _rows_of(case, gen, n):
    """n rows of keys or values in 32 bits: normal, some dims of each head larger than others."""
    x = _normal((n, case["kv_heads"], case["dim"]), gen)
    x[..., ::16] *= 4.0
    return x


def _pool_of(case, kind, pages, gen):
    """Bytes of a pool [2, pages, page * row] that holds a cache of rows."""
    b = case["page"]
    pool = torch.zeros((2, pages, b * _row_bytes(case, kind)), dtype=torch.uint8, device=DEV)
    part = max(1, (1 << 27) // (b * case["kv_heads"] * case["dim"]))
    for j in range(2):
        for p in range(0, pages, part):
            n = min(part, pages - p)
            x = _rows_of(case, gen, n * b).view(n, b, case["kv_heads"], case["dim"])
            if kind == "fp4":
                for view, bytes_ in zip(_views(pool, case), _quantise(x)):
                    view[j, p:p + n] = bytes_
                continue
            x = x.clamp(-FP8_MAX, FP8_MAX).to(DTYPES[kind])
            x = x.transpose(1, 2) if case["layout"] == "hnd" else x
            pool[j, p:p + n] = x.contiguous().view(torch.uint8).reshape(n, -1)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed) * 1000003 + 29)
    page, h, d = case["page"], case["kv_heads"], case["dim"]
    dtype, kind = DTYPES[case["dtype"]], case.get("pool", "fp4")
    s = {"case": dict(case)}
    if case["op"] != "attend":
        pages, t = case["rows"] // page, case["tokens"]
        s["slots"] = torch.randperm(pages * page, device=DEV, generator=gen)[:t].contiguous()
        if case["op"] == "store":
            s["pool"] = torch.zeros((2, pages, page * _row_bytes(case, kind)), dtype=torch.uint8,
                                    device=DEV)
            # K and V as slices of a fused projection's output rows
            qkv = _normal((t, 4 * h, d), gen)
            qkv[..., ::16] *= 4.0
            qkv = qkv.to(dtype)
            s["k"], s["v"] = qkv[:, 2 * h:3 * h], qkv[:, 3 * h:]
        else:
            s["pool"] = _pool_of(case, kind, pages, gen)
    else:
        new, ctx, prefix, members = _lengths(case)
        need = sum(_pages(c, page) for c in ctx) + sum(_pages(p, page) for p in prefix)
        pages = need + need // 4 + 1
        hq = h * case["group"]
        s["pool"] = _pool_of(case, kind, pages, gen)
        ids = torch.randperm(pages, device=DEV, generator=gen).to(torch.int32)
        pre_off = _offsets([_pages(p, page) for p in prefix])
        s.update(q=_normal((sum(new), hq, d), gen).to(dtype), softmax=d ** -0.5,
                 tok_off=_ints(_offsets(new), torch.int64), ctx=_ints(ctx, torch.int32),
                 pg_off=_ints(_offsets([_pages(c, page) for c in ctx]), torch.int64),
                 ids=ids[pre_off[-1]:].clone(), max_new=max(new), max_ctx=max(ctx), tokens=sum(new))
        if prefix:
            s.update(members=_ints(members, torch.int64), prefix=_ints(prefix, torch.int32),
                     pre_off=_ints(pre_off, torch.int64), pre_ids=ids[:max(pre_off[-1], 1)].clone(),
                     max_prefix=max(prefix),
                     max_rows=max(sum(new[a:b]) for a, b in zip(members, members[1:])))
    if own:         # the descriptors of pool and batch, buffers and workspace that a user's program keeps
        import scatter_kvx_gather_amd as kvx
        layout = kvx.Layout(1, 2, h, d, kind)
        s["layout"] = layout
        s["kvx_pool"] = kvx.Pool(s["pool"], s["pool"].shape[1], page,
                                 slot_stride=_row_bytes(case, kind))
        if case["op"] == "attend":
            s["reqs"] = kvx.Requests(s["tok_off"], s["tokens"])
            s["table"] = kvx.Table(s["pg_off"], s["ids"])
            s["kvx_prefix"] = kvx.Prefix(s["members"], s["prefix"], kvx.Table(
                s["pre_off"], s["pre_ids"])) if case["groups"] else None
            s["workspace"] = torch.empty(
                kvx.attend_workspace(layout, s["reqs"], hq, prefix=s["kvx_prefix"]),
                dtype=torch.uint8, device=DEV)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device=DEV)
        else:
            s["k_out"], s["v_out"] = (torch.empty((case["tokens"], h, d), dtype=dtype, device=DEV)
                                      for _ in range(2))
    return s


# -------------------------------------------------------------------- run --

def run(s):
    op = s["case"]["op"]
    if own:
        return {"store": _own_store, "read": _own_read, "attend": _own_attend}[op](s)
    return {"store": _plain_store, "read": _plain_read, "attend": _plain_attend}[op](s)


def _own_store(s):
    import scatter_kvx_gather_amd as kvx
    c = s["case"]
    kvx.append(s["layout"], 0, s["kvx_pool"], s["slots"], s["k"], s["v"], k_scale=c["scale"],
               v_scale=c["scale"], block_layout=c["layout"])
    return _own_read(s)


def _own_read(s):
    import scatter_kvx_gather_amd as kvx
    c = s["case"]
    kvx.read(s["layout"], 0, s["kvx_pool"], s["slots"], s["k_out"], s["v_out"], k_scale=c["scale"],
             v_scale=c["scale"], block_layout=c["layout"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_attend(s):
    import scatter_kvx_gather_amd as kvx
    c = s["case"]
    kvx.attend(s["layout"], 0, s["kvx_pool"], s["reqs"], s["ctx"], s["table"], s["q"], s["out"],
               prefix=s["kvx_prefix"], lse=s["lse"], scale=s["softmax"], k_scale=c["scale"],
               v_scale=c["scale"], block_layout=c["layout"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _plain_store(s):
    b, scale = s["case"]["page"], s["case"]["scale"]
    for j, x in enumerate((s["k"], s["v"])):
        for view, bytes_ in zip(_views(s["pool"], s["case"]), _quantise(x.float() / scale)):
            view[j, s["slots"] // b, s["slots"] % b] = bytes_
    return _plain_read(s)


def _at(pool, case, kind, j, pages, rows):
    """[.., heads, dim] in 32 bits: rows of pages of plane j."""
    if kind == "fp4":
        numbers, scales = _views(pool, case)
        return _values(numbers[j, pages, rows], scales[j, pages, rows])
    b, h, d = case["page"], case["kv_heads"], case["dim"]
    x = pool[j].view(-1, *((b, h) if case["layout"] == "nhd" else (h, b)),
                     d * (1 if kind == "fp8" else 2))
    x = (x if case["layout"] == "nhd" else x.transpose(1, 2))[pages, rows]
    return x.contiguous().view(DTYPES[kind]).float()


def _plain_read(s):
    c = s["case"]
    pages, rows = s["slots"] // c["page"], s["slots"] % c["page"]
    k, v = (_at(s["pool"], c, c.get("pool", "fp4"), j, pages, rows) * c["scale"] for j in range(2))
    return {"k": k.to(DTYPES[c["dtype"]]), "v": v.to(DTYPES[c["dtype"]])}


def _rows(s, j, ids, off, count, most):
    """[lists, heads, most, dim] in 32 bits: the first `most` rows of every list of pages."""
    b = s["case"]["page"]
    pos = torch.arange(max(most, 1), device=DEV)
    pos = torch.minimum(pos[None], (count[:, None] - 1).clamp(min=0))
    pages = ids[(off[:-1, None] + pos // b).clamp(max=ids.numel() - 1)].long()
    x = _at(s["pool"], s["case"], "fp4", j, pages, pos % b) * s["case"]["scale"]
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
    q = s["q"].float().view(t, h, g, d) * s["softmax"]
    at = torch.arange(t, device=DEV)
    req = torch.searchsorted(s["tok_off"], at, right=True) - 1

    def lists(first, most):
        """Rows of q as [lists, heads, most * group, dim]."""
        i = (first[:, None] + torch.arange(most, device=DEV)[None]).clamp(max=t - 1)
        return q[i].permute(0, 2, 1, 3, 4).reshape(first.numel(), h, most * g, d)

    def tokens(x, which, inside, most):
        """[lists, heads, most * group, n] back to [tokens, heads, group, n]."""
        return x.view(x.shape[0], h, most, g, -1)[which, :, inside]

    new, ctx = s["tok_off"].diff(), s["ctx"].long()
    k, v = (_rows(s, j, s["ids"], s["pg_off"], ctx, s["max_ctx"]) for j in range(2))
    row = torch.arange(s["max_new"] * g, device=DEV) // g
    last = (ctx - new)[:, None] + row[None]                       # the last key that a row sees
    seen = torch.arange(k.shape[2], device=DEV)[None, None] <= last[:, :, None]
    seen = seen & (torch.arange(k.shape[2], device=DEV) < ctx[:, None, None])
    parts = [[tokens(x, req, at - s["tok_off"][req], s["max_new"])
              for x in _part(lists(s["tok_off"][:-1], s["max_new"]), k, v, seen[:, None])]]
    if c["groups"] and s["max_prefix"]:
        grp = torch.searchsorted(s["members"], req, right=True) - 1
        first = s["tok_off"][s["members"]]
        count = s["prefix"].long()
        k, v = (_rows(s, j, s["pre_ids"], s["pre_off"], count, s["max_prefix"]) for j in range(2))
        seen = torch.arange(k.shape[2], device=DEV)[None] < count[:, None]
        parts.append([tokens(x, grp, at - first[grp], s["max_rows"])
                      for x in _part(lists(first[:-1], s["max_rows"]), k, v, seen[:, None, None])])
    top = torch.stack([p[0] for p in parts]).amax(0)
    weight = [torch.exp(p[0] - top.clamp(min=-1e30)) for p in parts]
    total = sum(w * p[1] for w, p in zip(weight, parts))
    out = sum(w * p[2] for w, p in zip(weight, parts)) / total.clamp(min=1e-30)
    lse = top + torch.log(total)
    return {"out": out.reshape(t, h * g, d).to(s["q"].dtype), "lse": lse.reshape(t, h * g)}


# ------------------------------------------------------------------- work --

def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    n = case["kv_heads"] * case["dim"]
    held = {"fp4": n * 17 / 32, "fp8": n}.get(case.get("pool", "fp4"), 2 * n)   # a row without its padding
    if case["op"] != "attend":
        # store: rows read, the cache's written, read again and the dense ones written
        passes = 2 if case["op"] == "store" else 1
        return {"bytes": passes * case["tokens"] * (2 * (n * size + held) + 8), "flops": 0}
    new, ctx, prefix, members = _lengths(case)
    hq = case["kv_heads"] * case["group"]
    ids = sum(_pages(x, case["page"]) for x in ctx + prefix)
    shared = [0] * case["reqs"]
    for g, p in enumerate(prefix):
        for r in range(members[g], members[g + 1]):
            shared[r] = p
    seen = sum(m * (p + c) - m * (m - 1) // 2 for m, c, p in zip(new, ctx, shared))
    return {"bytes": 2 * (sum(ctx) + sum(prefix)) * held + 4 * ids
            + sum(new) * hq * (2 * case["dim"] * size + 4),
            "flops": 4 * case["dim"] * hq * seen}


# ------------------------------------------------------------------ exact --

def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, s)


def _nearest(x):
    """What the cache holds of x [.., dim], in 64 bits: each block's step by step definition."""
    y = x.double().unflatten(-1, (-1, 32))
    top = y.abs().amax(-1, keepdim=True)
    unit = torch.full_like(top, 2.0 ** -23)
    for _ in range(36):                                    # the smallest power of two that is enough
        unit = torch.where(top > 7.0 * unit, unit * 2.0, unit)
    a = (y / unit).abs()
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    held = torch.minimum(torch.round(a / step) * step, torch.full_like(a, 6.0))    # round: half to even
    return (torch.sign(y) * held * unit).flatten(-2)


def _exact_store(case, s):
    c = case["scale"]                                      # the quotient is the 32-bit one
    return {"k": _nearest(s["k"].float() / c) * c, "v": _nearest(s["v"].float() / c) * c}


def _block(case, pool, page, j):
    """Page `page` of plane j, or pages of a list, as [.., rows, heads, dim] in 64 bits: from the bits."""
    b, h, d = case["page"], case["kv_heads"], case["dim"]
    raw = pool[j, page]
    kind = case.get("pool", "fp4")
    if kind != "fp4":
        x = raw.view(DTYPES[kind]).double().unflatten(-1, (b, h, d) if case["layout"] == "nhd" else (h, b, d))
        return x if case["layout"] == "nhd" else x.transpose(-2, -3)
    lead = raw.shape[:-1]
    if case["layout"] == "nhd":
        row = raw.reshape(*lead, b, -1)
        half = row[..., :h * d // 2].reshape(*lead, b, h, d // 2)
        scale = row[..., h * d // 2:h * d * 17 // 32].reshape(*lead, b, h, d // 32)
    else:
        half = raw[..., :h * b * d // 2].reshape(*lead, h, b, d // 2).transpose(-2, -3)
        scale = raw[..., h * b * d // 2:h * b * d * 17 // 32].reshape(*lead, h, b, d // 32).transpose(-2, -3)
    code = torch.empty(*half.shape[:-1], d, dtype=torch.float64, device=half.device)
    code[..., 0::2], code[..., 1::2] = (half % 16).double(), (half // 16).double()
    sign = 1.0 - 2.0 * (code >= 8)
    code = code % 8
    power, fraction = torch.floor(code / 2), code % 2      # two bits of exponent, one of mantissa
    x = torch.where(power == 0, fraction * 0.5, (1.0 + fraction * 0.5) * 2.0 ** (power - 1.0))
    return sign * x * (2.0 ** (scale.double() - 127.0)).repeat_interleave(32, -1)


def _exact_read(case, s):
    b, found = case["page"], {}
    for j, name in enumerate(("k", "v")):
        out = torch.empty((case["tokens"], case["kv_heads"], case["dim"]), dtype=torch.float64, device=DEV)
        for t in range(0, case["tokens"], 4096):
            slots = s["slots"][t:t + 4096]
            x = _block(case, s["pool"], slots.div(b, rounding_mode="floor"), j)
            out[t:t + 4096] = x[torch.arange(slots.numel(), device=DEV), slots.remainder(b)] * case["scale"]
        found[name] = out
    return found


def _exact_attend(case, s):
    """Request by request in 64 bits: one softmax over prefix and own keys."""
    b, g, d, h = case["page"], case["group"], case["dim"], case["kv_heads"]

    def rows(ids, off, i, n, j):
        x = _block(case, s["pool"], ids[off[i]:off[i] + _pages(n, b)].long(), j)
        return x.reshape(-1, h, d)[:n].permute(1, 0, 2) * case["scale"]

    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    tok, ctx, off = s["tok_off"].tolist(), s["ctx"].tolist(), s["pg_off"].tolist()
    groups = case["groups"]
    members = s["members"].tolist() if groups else [0, case["reqs"]]
    prefix = s["prefix"].tolist() if groups else [0]
    pre_off = s["pre_off"].tolist() if groups else [0, 0]
    for i, p in enumerate(prefix):
        shared = [rows(s["pre_ids"], pre_off, i, p, j) if p else None for j in range(2)]
        for r in range(members[i], members[i + 1]):
            n = tok[r + 1] - tok[r]
            k, v = (rows(s["ids"], off, r, ctx[r], j) for j in range(2))
            if p:
                k, v = torch.cat([shared[0], k], 1), torch.cat([shared[1], v], 1)
            q = s["q"][tok[r]:tok[r + 1]].double().view(n, h, g, d).permute(1, 2, 0, 3)
            x = torch.matmul(q.reshape(h, g * n, d), k.transpose(1, 2).contiguous()) * s["softmax"]
            edge = p + ctx[r] - n + torch.arange(n, device=DEV).repeat(g)
            x[:, torch.arange(p + ctx[r], device=DEV)[None] > edge[:, None]] = -math.inf
            z = torch.logsumexp(x, 2)
            y = torch.matmul(torch.exp(x - z[..., None]), v)
            out[tok[r]:tok[r + 1]] = y.view(h, g, n, d).permute(2, 0, 1, 3).reshape(n, -1, d)
            lse[tok[r]:tok[r + 1]] = z.view(h, g, n).permute(2, 0, 1).reshape(n, -1)
    return {"out": out, "lse": lse}
