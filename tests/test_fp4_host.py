"""4-bit pools on the host (no GPU): the plain reference against the format's
definition, exports, and every bad argument refused with its status before
anything reaches the GPU.  Device pointers here are fake addresses that
validation compares and never reads."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import scatter_kvx_gather_amd as kvx
from tests import fp4_ref as f4

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, E_NULL, E_SHAPE, E_ALIGN, E_DTYPE, E_RANGE, E_UNSUPPORTED = 0, 1, 2, 3, 4, 5, 6
E_OVERLAP = 9
A = 0x7F0000000000
F16, BF16, FP8, F32, FP4 = 1, 2, 3, 4, 5
NAN, INF = float("nan"), float("inf")


def layout(L=2, kv=2, H=8, D=128, dtype=FP4):
    return kvx._CLayout(L, kv, H, D, dtype)


def pool(Q=4, num_pages=16, page_size=16, stride=544, base=A + (8 << 30), page_stride=0):
    arr = (ctypes.c_void_p * Q)(*[base + q * (1 << 20) if base else None for q in range(Q)])
    p = kvx._CPool(ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), num_pages, page_size, stride,
                   page_stride)
    p.keep = arr
    return p


def rows_call(name, lay=None, layer=0, p=None, bl=0, slots=A, skipped=None, rows=True, **r):
    f = dict(k=A, v=A + (1 << 42), k_stride=2048, v_stride=4096, num_tokens=8, dtype=BF16,
             k_scale=1.0, v_scale=1.0)
    f.update(r)
    lay = layout() if lay is None else lay
    p = pool() if p is None else p
    return getattr(kvx.load_library(), name)(
        lay if lay != 0 else None, layer, p if p != 0 else None, bl, slots,
        kvx._CRows(**f) if rows else None, skipped, None)


# ------------------------------------------------------------ the reference --

def test_reference_against_the_definition():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 64)) * 2.0 ** rng.integers(-40, 30, (40, 1))).astype(np.float32)
    x[3, :32] = 0.0
    x[4, 5] = -0.0
    x[5, 7] = NAN
    x[6, 40] = -INF
    codes, scales = f4.quantise(x)
    assert (scales[5, 0], scales[3, 0], scales[6, 1]) == (255, 104, 140)
    v = f4.values(codes, scales)
    assert np.isnan(v[5, :32]).all() and not np.isnan(v[5, 32:]).any()
    assert v[6, 40] == -49152 and codes[4, 5] == 8
    for i in range(40):
        for b in range(2):
            s = int(scales[i, b])
            y = x[i, 32 * b:32 * b + 32].astype(np.float64)
            if s == 255:
                continue
            top, u = np.abs(y).max(), 2.0 ** (s - 127)
            assert s == 140 or top <= 7 * u
            assert s == 104 or top > 3.5 * u
            grid = np.concatenate([-f4.GRID[::-1], f4.GRID]) * u
            best = np.abs(np.clip(y, -6 * u, 6 * u)[:, None] - grid).min(1)
            held = v[i, 32 * b:32 * b + 32]
            assert np.array_equal(np.abs(np.clip(y, -6 * u, 6 * u) - held), best)
    # ties go to the even code
    t = np.array([[0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 4], np.float32)
    assert f4.quantise(t)[0][0, :8].tolist() == [0, 2, 2, 4, 4, 6, 6, 7] and f4.quantise(t)[1][0, 0] == 127
    assert np.array_equal(f4.unpack(f4.pack(codes)), codes)


def test_reference_values_are_exact_in_16_bits():
    codes = np.tile(np.arange(16, dtype=np.uint8), 2)[None]
    for s in range(104, 141):
        v = torch.from_numpy(f4.values(codes, np.array([[s]], np.uint8)))
        for t in (torch.float16, torch.bfloat16, torch.float32):
            assert torch.equal(v.to(t).double(), v)


def test_page_views_cover_distinct_bytes():
    for lay in ("nhd", "hnd"):
        for H, D, B in ((1, 32, 1), (2, 96, 5), (8, 128, 16), (3, 256, 2)):
            raw = np.zeros((2, B * f4.row_bytes(H, D)), np.uint8)
            for v in f4.views(raw, B, H, D, lay):
                v += 1
            assert raw.max() == 1 and raw.sum() == 2 * B * H * D * 17 // 32


# ------------------------------------------------------------------ exports --

def test_exports_every_declared_function():
    text = open(os.path.join(ROOT, "include", "kvx_read.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(kvx_[a-z_]+)\s*\(", text))
    assert names == {"kvx_read"}
    assert hasattr(ctypes.CDLL(kvx.library_path()), "kvx_read")


def test_header_compiles_as_c99(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#define __HIP_PLATFORM_AMD__ 1\n#include "kvx_read.h"\n'
                   "int main(void) { kvx_rows_out r; (void)r;\n"
                   "return kvx_read(0, 0, 0, KVX_NHD, 0, 0, 0, 0) == KVX_OK || KVX_FP4 != 5; }\n")
    inc = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-fsyntax-only", "-I", inc,
                    "-I", os.path.join(ROOT, "include"), str(src)], check=True)


# ------------------------------------------------------------------ layouts --

@pytest.mark.parametrize("H,D", [(1, 32), (1, 64), (1, 128), (2, 96), (5, 160), (8, 128), (8, 256)])
def test_row_bytes(H, D):
    """The binding and the library agree on a row: a smaller slot stride is refused."""
    R = kvx.Layout(1, 2, H, D, "fp4").row_bytes
    assert R == f4.row_bytes(H, D) and R % 16 == 0
    wide = dict(k_stride=1 << 16, v_stride=1 << 16, num_tokens=0)
    assert rows_call("kvx_append", lay=layout(H=H, D=D), p=pool(stride=R), **wide) == OK
    assert rows_call("kvx_append", lay=layout(H=H, D=D), p=pool(stride=R - 16), **wide) == E_SHAPE


@pytest.mark.parametrize("name", ["kvx_append", "kvx_read"])
def test_layout_refusals(name):
    for D in (16, 33, 48, 100):
        assert rows_call(name, lay=layout(D=D)) == E_ALIGN
    assert rows_call(name, lay=layout(H=8, D=1 << 20), p=pool(stride=1 << 24)) == E_RANGE
    assert rows_call(name, lay=layout(H=1 << 30, D=1 << 30)) == E_RANGE
    assert rows_call(name, lay=layout(D=0)) == E_SHAPE
    assert rows_call(name, lay=layout(kv=1), p=pool(2)) == E_UNSUPPORTED
    assert rows_call(name, lay=layout(dtype=6)) == E_DTYPE


# ----------------------------------------------------------- append and read --

@pytest.mark.parametrize("name", ["kvx_append", "kvx_read"])
def test_rows_refusals(name):
    def call(**kw):
        return rows_call(name, **kw)
    assert call(num_tokens=0) == OK                     # nothing to do, nothing enqueued
    assert call(lay=0) == E_NULL
    assert call(p=0) == E_NULL
    assert call(rows=False) == E_NULL
    assert call(layer=-1) == E_SHAPE
    assert call(layer=2) == E_SHAPE
    assert call(bl=2) == E_SHAPE
    assert call(dtype=0) == E_DTYPE
    assert call(dtype=9) == E_DTYPE
    assert call(dtype=FP8) == E_UNSUPPORTED
    assert call(dtype=FP4) == E_UNSUPPORTED
    assert call(num_tokens=-1) == E_SHAPE
    assert call(num_tokens=1 << 31) == E_RANGE
    assert call(num_tokens=1 << 27) == E_RANGE          # more threads than a launch counts
    for bad in (0.0, -1.0, NAN, INF):
        assert call(k_scale=bad) == E_SHAPE
        assert call(v_scale=bad) == E_SHAPE
    for bad in (1e-38, 2.0 ** -65, 2.0 ** 65, 1e38):
        assert call(k_scale=bad) == E_RANGE
        assert call(v_scale=bad) == E_RANGE
    for f in ("k", "v"):
        assert call(**{f: None}) == E_NULL
        assert call(**{f: A + 8}) == E_ALIGN
        assert call(**{f + "_stride": 2032}) == E_SHAPE
        assert call(**{f + "_stride": 2056}) == E_ALIGN
    assert call(slots=None) == E_NULL
    assert call(k_stride=1 << 62, num_tokens=1 << 20) == E_RANGE
    assert call(p=pool(stride=528)) == E_SHAPE
    assert call(p=pool(base=A + 8)) == E_ALIGN
    assert call(p=pool(base=0)) == E_NULL
    assert call(p=pool(page_stride=544)) == E_SHAPE


def test_read_refusals_of_other_pools():
    for dt, stride in ((F16, 2048), (BF16, 2048), (F32, 4096)):
        lay, p = layout(dtype=dt), pool(stride=stride)
        for to in (F16, BF16, FP8, F32):
            if to != dt:
                assert rows_call("kvx_read", lay=lay, p=p, dtype=to, k_stride=4096) == E_UNSUPPORTED
        assert rows_call("kvx_read", lay=lay, p=p, dtype=dt, k_stride=4096, k_scale=2.0) == E_UNSUPPORTED
        assert rows_call("kvx_read", lay=lay, p=p, dtype=dt, k_stride=4096, num_tokens=0) == OK
    lay, p = layout(dtype=FP8), pool(stride=1024)
    assert rows_call("kvx_read", lay=lay, p=p, dtype=FP8, v_scale=0.5) == E_UNSUPPORTED
    assert rows_call("kvx_read", lay=lay, p=p, dtype=F16, v_scale=0.5, num_tokens=0) == OK
    assert rows_call("kvx_read", lay=layout(H=4, D=4, dtype=BF16), p=pool(stride=32), bl=1,
                     k_stride=32, v_stride=32) == E_ALIGN


def test_read_refuses_rows_that_meet():
    """Rows of k and v are both written: none may share a byte (what is disjoint
    is run on the GPU)."""
    def at(d, **kw):
        return rows_call("kvx_read", v=A + d, **kw)
    for d in (0, 16, 2032, -2032, 2048, 3 * 2048 + 16):
        assert at(d, v_stride=2048) == E_OVERLAP, d
    for d in (0, 2032, -2032):
        assert at(d, num_tokens=1) == E_OVERLAP, d
    for d in (0, 2032, -2032, 8192, 8192 * 7 + 2032):
        assert at(d, k_stride=8192, v_stride=8192) == E_OVERLAP, d


# ----------------------------------------------------------------- attention --

def attend(lay=None, p=None, bl=0, reqs=(2, 4, A), **a):
    f = dict(q=A, out=A + (1 << 20), lse=A + (1 << 21), q_stride=8192, out_stride=8192, q_heads=32,
             dtype=BF16, scale=0.1, k_scale=1.0, v_scale=1.0, flags=1, workspace=A + (1 << 30),
             workspace_bytes=1 << 40)
    f.update(a)
    lay = layout() if lay is None else lay
    p = pool() if p is None else p
    return kvx.load_library().kvx_attend(lay, 0, p, bl, kvx._CReqs(*reqs), A, kvx._CTable(A, A, 4),
                                         None, kvx._CAttention(**f), None, None)


def test_attend_refusals():
    assert attend(reqs=(2, 0, A)) == OK                 # nothing to do, nothing enqueued
    assert attend(reqs=(2, 0, A), dtype=F16) == OK
    assert attend(dtype=F32) == E_UNSUPPORTED
    assert attend(dtype=FP8) == E_UNSUPPORTED
    assert attend(dtype=FP4) == E_UNSUPPORTED or attend(dtype=FP4) == E_DTYPE
    assert attend(lay=layout(D=288), p=pool(stride=1232)) == E_UNSUPPORTED
    assert attend(lay=layout(D=48)) == E_ALIGN
    assert attend(lay=layout(kv=1), p=pool(2)) == E_UNSUPPORTED
    assert attend(p=pool(stride=528)) == E_SHAPE
    assert attend(p=pool(num_pages=0, base=0)) == E_SHAPE
    assert attend(q_heads=33) == E_SHAPE
    assert attend(bl=2) == E_SHAPE
    assert attend(workspace_bytes=1 << 20) == E_SHAPE
    assert attend(out=A) == E_OVERLAP
    assert attend(scale=1e38, k_scale=1e38) == E_RANGE


def test_copies_take_rows_and_refuse_heads():
    lib, lay, p = kvx.load_library(), layout(L=1), pool(Q=2)
    reqs, tab = kvx._CReqs(1, 4, A), kvx._CTable(A, A, 4)
    assert lib.kvx_gather(lay, p, tab, reqs, A, 4 * 2 * 544 - 1, None, 0, None) == E_SHAPE
    assert lib.kvx_gather(lay, p, tab, kvx._CReqs(0, 0, None), None, 0, None, 0, None) == OK
    heads = kvx._CHeads(8, 0, 0)
    assert lib.kvx_gather_scatter_heads(lay, p, tab, heads, reqs, p, tab, heads, None,
                                        None) == E_UNSUPPORTED
    arr = (ctypes.c_void_p * 2)(A, A + (1 << 24))
    assert lib.kvx_extract_permute(lay, arr, 8, 4, A, 1 << 30, 0, None) == E_UNSUPPORTED
    assert lib.kvx_rebuild_permute(lay, A, 1 << 30, 4, arr, 8, 0, None) == E_UNSUPPORTED


# ------------------------------------------------------------- the binding --

def test_binding_refusals():
    """What the binding itself refuses, before the library is asked."""
    lay = kvx.Layout(1, 2, 2, 64, "fp4")
    p = kvx.Pool(torch.zeros(2, 8, 16 * 80, dtype=torch.uint8), 8, 16, slot_stride=80)
    k = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int64)
    for fn in (kvx.append, kvx.read):
        for bad in (dict(slots=slots.int()), dict(slots=slots[:3]), dict(k=k[:, :1]), dict(v=k[:3]),
                    dict(k=k.transpose(1, 2)), dict(v=k.half()), dict(k=k.double(), v=k.double()),
                    dict(k=k.to(torch.uint8), v=k.to(torch.uint8)),
                    dict(k=k.expand(4, 2, 64)[:, :, ::2], v=k),
                    dict(pool=kvx.Pool(torch.zeros(2, 8, 16 * 64, dtype=torch.uint8), 8, 16,
                                       slot_stride=80)),                # too short a plane
                    dict(pool=kvx.Pool(torch.zeros(4, 8, 16 * 80, dtype=torch.uint8), 8, 16,
                                       slot_stride=80)),                # two layers' planes
                    dict()):                                            # the last: not on a GPU
            args = dict(pool=p, slots=slots, k=k, v=k.clone())
            args.update(bad)
            with pytest.raises(ValueError):
                fn(lay, 0, args.pop("pool"), **args)
