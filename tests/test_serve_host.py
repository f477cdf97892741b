"""The serving calls on the host (no GPU): the library exports what
include/kvx_serve.h declares, and every bad argument is refused with its status
before anything reaches the GPU.  Device pointers here are fake addresses that
validation compares and never reads."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import scatter_kvx_gather_amd as kvx
from tests import serve_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, E_NULL, E_SHAPE, E_ALIGN, E_DTYPE, E_RANGE, E_UNSUPPORTED = 0, 1, 2, 3, 4, 5, 6
E_OVERLAP = 9
A = 0x7F0000000000
F16, BF16, FP8, F32 = 1, 2, 3, 4
NAN, INF = float("nan"), float("inf")


def test_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "kvx_serve.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(kvx_[a-z_]+)\s*\(", text))
    assert names == {"kvx_build_tables", "kvx_append", "kvx_attend", "kvx_attend_workspace"}
    lib = ctypes.CDLL(kvx.library_path())
    for n in names:
        assert hasattr(lib, n), n


def layout(L=2, kv=2, H=8, D=128, dtype=BF16):
    return kvx._CLayout(L, kv, H, D, dtype)


def pool(Q=4, num_pages=16, page_size=16, stride=2048, base=A, page_stride=0):
    arr = (ctypes.c_void_p * Q)(*[base + q * (1 << 20) if base else None for q in range(Q)])
    p = kvx._CPool(ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), num_pages, page_size, stride,
                   page_stride)
    p.keep = arr
    return p


# ------------------------------------------------------------ build_tables --

def build(n=3, page=16, have=A, add=A + 64, held=(A, A, 8), free=A, num_free=10, out=None, **o):
    f = dict(ctx_len=A, tok_off=A, pg_off=A, page_ids=A, cap_ids=4, slots=A, cap_tokens=4, totals=0)
    f.update(o)
    t = kvx._CBatchTables(**f) if out is None else out
    h = kvx._CTable(*held) if held is not None else None
    return kvx.load_library().kvx_build_tables(n, page, have, add, h, free, num_free,
                                               t if out != 0 else None, None)


def test_build_tables_refusals():
    assert build(out=0) == E_NULL
    assert build(n=-1) == E_SHAPE
    assert build(page=0) == E_SHAPE
    assert build(page=-16) == E_SHAPE
    assert build(num_free=-1) == E_SHAPE
    assert build(cap_ids=-1) == E_SHAPE
    assert build(cap_tokens=-1) == E_SHAPE
    assert build(free=None) == E_NULL
    assert build(add=None) == E_NULL
    for f in ("ctx_len", "tok_off", "pg_off", "page_ids", "slots"):
        assert build(**{f: None}) == E_NULL, f
    assert build(held=None) == E_NULL
    assert build(held=(0, A, 8)) == E_NULL
    assert build(held=(A, 0, 8)) == E_NULL
    assert build(held=(A, A, -1)) == E_SHAPE
    assert build(cap_tokens=1 << 62) == E_RANGE
    assert build(cap_ids=1 << 62) == E_RANGE
    assert build(n=(1 << 24) + 1) == E_RANGE
    assert build(cap_tokens=1 << 36) == E_RANGE


BUILD_SIZES = dict(have=12, add=12, held_off=24, held_ids=32, free=40, ctx_len=12, tok_off=32, pg_off=32,
                   page_ids=1024, slots=2048, totals=32)     # bytes, of 3 requests
BUILD_OUT = ("ctx_len", "tok_off", "pg_off", "page_ids", "slots", "totals")


def build_at(**at):
    """build() with each buffer a MiB from the next one, but for those at `at`."""
    a = {f: A + (i << 20) for i, f in enumerate(BUILD_SIZES)}
    a.update(at)
    return build(have=a["have"], add=a["add"], held=(a["held_off"], a["held_ids"], 8), free=a["free"],
                 cap_ids=256, cap_tokens=256, **{f: a[f] for f in BUILD_OUT})


def test_build_tables_refuses_overlaps():
    """A workgroup writes an output while others read the lengths and the held
    table, so no output may share a byte with them, nor with another output."""
    at = {f: A + (i << 20) for i, f in enumerate(BUILD_SIZES)}
    for out in BUILD_OUT:
        for f, size in BUILD_SIZES.items():
            if f == out:
                continue
            assert build_at(**{out: at[f]}) == E_OVERLAP, (out, f)
            assert build_at(**{out: at[f] + size - 4}) == E_OVERLAP, (out, f)
            assert build_at(**{out: at[f] - BUILD_SIZES[out] + 4}) == E_OVERLAP, (out, f)


# ----------------------------------------------------------------- append --

def append(lay=None, layer=0, p=None, bl=0, slots=A, skipped=None, rows=True, **r):
    f = dict(k=A, v=A, k_stride=2048, v_stride=4096, num_tokens=8, dtype=BF16, k_scale=1.0,
             v_scale=1.0)
    f.update(r)
    lay = layout() if lay is None else lay
    p = pool() if p is None else p
    return kvx.load_library().kvx_append(lay if lay != 0 else None, layer, p if p != 0 else None, bl,
                                         slots, kvx._CRows(**f) if rows else None, skipped, None)


def test_append_refusals():
    assert append(num_tokens=0) == OK                   # nothing to do, nothing enqueued
    assert append(lay=0) == E_NULL
    assert append(p=0) == E_NULL
    assert append(rows=False) == E_NULL
    assert append(lay=layout(kv=1), p=pool(2)) == E_UNSUPPORTED
    assert append(lay=layout(dtype=9)) == E_DTYPE
    assert append(layer=-1) == E_SHAPE
    assert append(layer=2) == E_SHAPE
    assert append(bl=2) == E_SHAPE
    assert append(dtype=0) == E_DTYPE
    assert append(num_tokens=-1) == E_SHAPE
    assert append(num_tokens=1 << 31) == E_RANGE
    assert append(dtype=F16) == E_UNSUPPORTED           # f16 rows into a bf16 pool
    assert append(dtype=FP8) == E_UNSUPPORTED
    assert append(k_scale=2.0) == E_UNSUPPORTED         # nothing is rounded
    f8 = dict(lay=layout(dtype=FP8), p=pool(stride=1024))
    for bad in (0.0, -1.0, NAN, INF):
        assert append(**f8, k_scale=bad) == E_SHAPE
        assert append(**f8, v_scale=bad) == E_SHAPE
    assert append(**f8, dtype=FP8, v_scale=0.5) == E_UNSUPPORTED
    for bad in (1e-38, 2.0 ** -65, 2.0 ** 65, 1e38):
        assert append(**f8, k_scale=bad) == E_RANGE
        assert append(**f8, v_scale=bad) == E_RANGE
    for f in ("k", "v"):
        assert append(**{f: None}) == E_NULL
        assert append(**{f: A + 8}) == E_ALIGN
        assert append(**{f + "_stride": 2047}) == E_SHAPE
        assert append(**{f + "_stride": 2056}) == E_ALIGN
    assert append(slots=None) == E_NULL
    assert append(k_stride=1 << 62, num_tokens=1 << 20) == E_RANGE
    assert append(num_tokens=1 << 27) == E_RANGE                # more threads than a launch counts
    assert append(p=pool(stride=1024)) == E_SHAPE
    assert append(p=pool(base=A + 8)) == E_ALIGN
    assert append(p=pool(base=0)) == E_NULL
    assert append(lay=layout(H=4, D=4), p=pool(stride=32), bl=1, k_stride=32, v_stride=32) == E_ALIGN


# ----------------------------------------------------------------- attend --

def attend(lay=None, layer=0, p=None, bl=0, reqs=(2, 4, A), ctx=A, table=(A, A, 4), prefix=None,
           att=True, skipped=None, **a):
    f = dict(q=A, out=A + (1 << 20), lse=A, q_stride=8192, out_stride=8192, q_heads=32, dtype=BF16,
             scale=0.1, k_scale=1.0, v_scale=1.0, flags=1, workspace=A, workspace_bytes=1 << 40)
    f.update(a)
    lay = layout() if lay is None else lay
    p = pool() if p is None else p
    pre = None
    if prefix is not None:
        n, off, ln, t = prefix
        pre = kvx._CPrefix(n, off, ln, kvx._CTable(*t))
    return kvx.load_library().kvx_attend(
        lay if lay != 0 else None, layer, p if p != 0 else None, bl,
        kvx._CReqs(*reqs) if reqs is not None else None, ctx,
        kvx._CTable(*table) if table is not None else None, pre,
        kvx._CAttention(**f) if att else None, skipped, None)


def test_attend_refusals():
    assert attend(reqs=(0, 0, 0)) == OK                 # nothing to do, nothing enqueued
    assert attend(reqs=(2, 0, A)) == OK
    assert attend(lay=0) == E_NULL
    assert attend(p=0) == E_NULL
    assert attend(reqs=None) == E_NULL
    assert attend(ctx=None) == E_NULL
    assert attend(table=None) == E_NULL
    assert attend(att=False) == E_NULL
    assert attend(reqs=(-1, 0, A)) == E_SHAPE
    assert attend(reqs=(0, 4, A)) == E_SHAPE
    assert attend(reqs=(2, 4, 0)) == E_NULL
    assert attend(reqs=(2, 1 << 31, A)) == E_RANGE
    assert attend(reqs=(2, 1 << 23, A)) == E_RANGE
    assert attend(reqs=((1 << 24) + 1, 4, A)) == E_RANGE
    assert attend(layer=2) == E_SHAPE
    assert attend(bl=-1) == E_SHAPE
    assert attend(lay=layout(kv=1), p=pool(2)) == E_UNSUPPORTED
    assert attend(lay=layout(dtype=F32), p=pool(stride=4096)) == E_UNSUPPORTED
    assert attend(lay=layout(D=264, H=1), p=pool(stride=528), q_heads=1) == E_UNSUPPORTED
    assert attend(lay=layout(H=2, D=4, dtype=BF16), p=pool(stride=16), q_heads=2) == E_ALIGN
    assert attend(dtype=F16) == E_UNSUPPORTED           # f16 queries over a bf16 pool
    assert attend(dtype=F32) == E_UNSUPPORTED
    assert attend(dtype=77) == E_DTYPE
    assert attend(flags=2) == E_UNSUPPORTED
    assert attend(q_heads=0) == E_SHAPE
    assert attend(q_heads=33) == E_SHAPE
    assert attend(lay=layout(H=1, D=16), p=pool(stride=32), q_heads=129) == E_RANGE
    for bad in (0.0, -0.1, NAN, INF):
        assert attend(scale=bad) == E_SHAPE
        assert attend(k_scale=bad) == E_SHAPE
        assert attend(v_scale=bad) == E_SHAPE
    assert attend(scale=1e38, k_scale=1e38) == E_RANGE
    assert attend(p=pool(num_pages=0, base=0)) == E_SHAPE       # no row to read
    for f in ("q", "out", "workspace"):
        assert attend(**{f: None}) == E_NULL
        assert attend(**{f: A + 8}) == E_ALIGN
    assert attend(lse=A + 2) == E_ALIGN
    assert attend(workspace=A + 128) == E_ALIGN
    assert attend(workspace_bytes=1 << 20) == E_SHAPE
    assert attend(out=A) == E_OVERLAP
    for f in ("q_stride", "out_stride"):
        assert attend(**{f: 8176}) == E_SHAPE
        assert attend(**{f: 8200}) == E_ALIGN
        assert attend(**{f: 1 << 62}) == E_RANGE
    assert attend(p=pool(page_stride=1024)) == E_SHAPE
    ok = (1, A, A, (A, A, 4))
    assert attend(prefix=(-1, A, A, (A, A, 4))) == E_SHAPE
    assert attend(prefix=(1, 0, A, (A, A, 4))) == E_NULL
    assert attend(prefix=(1, A, 0, (A, A, 4))) == E_NULL
    assert attend(prefix=(1, A, A, (0, A, 4))) == E_NULL
    assert attend(prefix=(1, A, A, (A, 0, 4))) == E_NULL
    assert attend(prefix=(1, A, A, (A, A, -4))) == E_SHAPE
    assert attend(prefix=ok, workspace_bytes=1 << 20) == E_SHAPE


def attend_at(T=4, q_stride=8192, out_stride=8192, **at):
    """attend() of T tokens (rows of 8192 bytes) with its buffers 1 GiB apart, but
    for those at `at`, and exactly the workspace that it needs."""
    ws = ctypes.c_int64(0)
    assert kvx.load_library().kvx_attend_workspace(layout(), 2, 0, T, 32, ctypes.byref(ws)) == OK
    a = dict(q=A, out=A + (1 << 30), lse=A + (2 << 30), workspace=A + (3 << 30))
    a.update(at)
    return attend(reqs=(2, T, A), q_stride=q_stride, out_stride=out_stride, workspace_bytes=ws.value, **a)


def test_attend_refuses_overlaps():
    """Rows of out are written while other workgroups read q's; lse and the
    workspace are no one's rows either.  (What is disjoint is run on the GPU.)"""
    for d in (0, 16, 8176, -16, -8176, 8192, 3 * 8192 + 16, -3 * 8192 - 16):
        assert attend_at(out=A + d) == E_OVERLAP, d
    for d in (0, 16, 8176, -8176):
        assert attend_at(T=1, out=A + d) == E_OVERLAP, d
    # rows of one fused buffer that share bytes, of other tokens too
    for d in (0, 8176, -8176, 12304, 20480 + 8176, -20480 + 16, 3 * 20480, -3 * 20480):
        assert attend_at(q_stride=20480, out_stride=20480, out=A + d) == E_OVERLAP, d
    # different strides: row 1 of out ends in row 2 of q
    assert attend_at(T=3, q_stride=32768, out_stride=40960, out=A + 2 * 32768 - 40960 - 16) == E_OVERLAP
    assert attend_at(T=3, q_stride=40960, out_stride=8192, out=A + 40960 - 2 * 8192 - 16) == E_OVERLAP
    for d in (0, 4, 3 * 8192 + 8188, -4 * 32 * 4 + 4):      # lse has 4 * 32 * 4 bytes
        assert attend_at(lse=A + d) == E_OVERLAP, d
        assert attend_at(lse=A + (1 << 30) + d) == E_OVERLAP, d
        assert attend_at(lse=A + (3 << 30) + d) == E_OVERLAP, d
    for f in ("q", "out", "lse"):
        assert attend_at(**{f: A + (3 << 30) + (1 << 20)}) == E_OVERLAP, f


def workspace(lay, n, g, t, hq):
    out = ctypes.c_int64(-7)
    s = kvx.load_library().kvx_attend_workspace(lay, n, g, t, hq, ctypes.byref(out))
    return out.value if s == OK else -s


def test_attend_workspace():
    lay = layout()
    assert kvx.load_library().kvx_attend_workspace(lay, 1, 0, 1, 8, None) == E_NULL
    assert workspace(lay, -1, 0, 1, 8) == -E_SHAPE
    assert workspace(lay, 1, -1, 1, 8) == -E_SHAPE
    assert workspace(lay, 1, 0, -1, 8) == -E_SHAPE
    assert workspace(lay, 1, 0, 1, 12) == -E_SHAPE
    assert workspace(lay, 1, 0, 1, 8 * 129) == -E_RANGE
    assert workspace(lay, 1, 0, 1 << 23, 8) == -E_RANGE
    assert workspace(lay, (1 << 24) + 1, 0, 1, 8) == -E_RANGE
    assert workspace(lay, 1, (1 << 24) + 1, 1, 8) == -E_RANGE
    # a smaller batch never needs more
    sizes = [0, 1, 3, 64, 1000]
    for hq in (8, 32, 64):
        for n in sizes:
            for g in sizes:
                for t in sizes:
                    w = workspace(lay, n, g, t, hq)
                    assert w > 0
                    for n2, g2, t2 in ((n // 2, g, t), (n, g // 2, t), (n, g, t // 2), (n, 0, t)):
                        assert workspace(lay, n2, g2, t2, hq) <= w


# ------------------------------------------------------------- the binding --

def test_binding_refusals():
    """What the binding itself refuses, before the library is asked."""
    lay = kvx.Layout(1, 2, 2, 64, "bf16")
    p = kvx.Pool(torch.zeros(2, 8, 16, 2, 64, dtype=torch.bfloat16), 8, 16)
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int64)
    for bad in (dict(slots=slots.int()), dict(slots=slots[:3]), dict(k=k[:, :1]), dict(v=k[:3]),
                dict(k=k.transpose(1, 2)), dict(v=k.half()), dict(k=k.double(), v=k.double()),
                dict(k=k.expand(4, 2, 64)[:, :, ::2], v=k), dict()):        # the last: not on a GPU
        args = dict(slots=slots, k=k, v=k)
        args.update(bad)
        with pytest.raises(ValueError):
            kvx.append(lay, 0, p, **args)
    reqs = kvx.Requests(torch.tensor([0, 4]), 4)
    table = kvx.Table(torch.tensor([0, 1]), torch.tensor([0], dtype=torch.int32))
    ctx = torch.tensor([4], dtype=torch.int32)
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    for bad in (dict(q=q[:3]), dict(out=q[:, :3]), dict(q=q.float(), out=q.float()), dict(out=q.half()),
                dict(lse=torch.zeros(4, 4, dtype=torch.bfloat16)), dict(lse=torch.zeros(4, 3)),
                dict(ctx_len=ctx.long()), dict(ctx_len=ctx[:0]), dict(q=q[0]), dict()):
        args = dict(ctx_len=ctx, table=table, q=q, out=torch.empty_like(q))
        args.update(bad)
        with pytest.raises(ValueError):
            kvx.attend(lay, 0, p, reqs, **args)
    with pytest.raises(ValueError):
        kvx.Prefix(torch.tensor([0, 1]), torch.zeros(0, dtype=torch.int32), table)
    with pytest.raises(ValueError):
        kvx.Prefix(torch.tensor([0, 1, 1]), torch.zeros(2, dtype=torch.int32), table)
    o = kvx.BatchTables(2, 8, 8, device="cpu")
    two = torch.ones(2, dtype=torch.int32)
    for bad in (dict(add_len=two.long()), dict(add_len=two[:1]), dict(have_len=two),
                dict(have_len=two, held=o.table), dict()):
        args = dict(add_len=two, free_ids=two)
        args.update(bad)
        with pytest.raises(ValueError):
            kvx.build_tables(o, 16, **args)


def test_binding_refuses_a_stream_of_another_gpu(monkeypatch):
    """A launch goes to the tensors' GPU, whose stream it has to be."""
    class Stream:
        def __init__(self, index):
            self.device_index, self.cuda_stream = index, 5

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    calls = []
    for dev, index in ((0, 1), (1, 0)):
        with pytest.raises(ValueError, match="stream"):
            kvx._launch(dev, Stream(index), lambda *a: calls.append(a), 1, 2)
    assert not calls
    kvx._launch(0, Stream(0), lambda *a: calls.append(a), 1, 2)
    assert calls == [(1, 2, 5)]


# ------------------------------------------------------- the plain reference --

def test_reference_tables():
    t = ref.build_tables(4, [5, 0], [4, 3], [[7, 9], []], [1, 2, 3])
    assert t["ids"] == [7, 9, 1, 2] and t["pg_off"] == [0, 3, 4] and t["tok_off"] == [0, 4, 7]
    assert t["slots"] == [37, 38, 39, 4, 8, 9, 10] and t["totals"] == [7, 4, 2, 0]


def test_reference_attention():
    """The host form against torch's softmax in 64 bits."""
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(24, 2, 8, generator=g, dtype=torch.float64) for _ in range(2))
    q = torch.randn(3, 4, 8, generator=g, dtype=torch.float64)
    import numpy as np
    b = ref.Batch(4, 6, [3], [7], np.array([0, 2]), np.array([5, 1]), [0, 1], [6], np.array([0, 2]),
                  np.array([2, 0]))
    out, lse, *_ = ref.attend(b, q.numpy(), k.numpy(), v.numpy(), 0.3)
    rows = [8, 9, 10, 11, 0, 1] + [20, 21, 22, 23, 4, 5, 6]
    kk, vv = (x[rows].repeat_interleave(2, 1).transpose(0, 1) for x in (k, v))
    s = q.transpose(0, 1) @ kk.transpose(1, 2) * 0.3
    for i in range(3):
        s[:, i, 6 + 7 - 3 + i + 1:] = -INF
    exp = (torch.softmax(s, -1) @ vv).transpose(0, 1)
    assert np.allclose(out, exp.numpy(), rtol=1e-12)
    assert np.allclose(lse, torch.logsumexp(s, -1).T.numpy(), rtol=1e-12)


def test_header_compiles_as_c99(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#define __HIP_PLATFORM_AMD__ 1\n#include "kvx_serve.h"\n'
                   "int main(void) { kvx_rows r; kvx_attention a; kvx_prefix p; kvx_batch_tables t;\n"
                   "(void)r; (void)a; (void)p; (void)t;\n"
                   "return kvx_attend_workspace(0, 0, 0, 0, 1, 0) == KVX_OK; }\n")
    inc = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", inc,
                    "-I", os.path.join(ROOT, "include"), str(src)], check=True)
