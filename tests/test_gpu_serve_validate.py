"""KVX_VALIDATE=1 (debug mode) for the serving calls on the GPU, in a child
process (the flag is read once per process): a step with good tables runs as
without it, and broken lengths, offsets, capacities and slots written twice are
refused with their status, with nothing written."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
sys.path.insert(0, {root!r})
import torch
import scatter_kvx_gather_amd as kvx

dev = torch.device("cuda:0")
i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
i64 = lambda *x: torch.tensor(x, dtype=torch.int64, device=dev)
SHAPE, DUPLICATE = 2, 8
lay = kvx.Layout(1, 2, 2, 64, "bf16")
store = torch.zeros(2, 16, 16, 2, 64, dtype=torch.bfloat16, device=dev)
pool = kvx.Pool(store, 16, 16, slot_stride=256)

def refused(status, fn, *unchanged):
    before = [x.clone() for x in unchanged]
    try:
        fn()
    except kvx.KvxError as e:
        assert e.status == status, (e.status, status)
    else:
        raise AssertionError("not refused")
    torch.cuda.synchronize()
    for x, y in zip(unchanged, before):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))

t = kvx.BatchTables(2, 40, 8)
kvx.build_tables(t, 16, i32(20, 5), i32(3, 4, 5, 6))
torch.cuda.synchronize()
assert t.totals.tolist() == [25, 3, 3, 0] and t.slots[:25].tolist() == list(range(48, 68)) + list(range(80, 85))
same = t.slots, t.page_ids, t.ctx_len
refused(SHAPE, lambda: kvx.build_tables(t, 16, i32(20, -1), i32(3, 4, 5, 6)), *same)
refused(SHAPE, lambda: kvx.build_tables(t, 16, i32(20, 21), i32(3, 4, 5, 6)), *same)       # 41 slots
refused(SHAPE, lambda: kvx.build_tables(t, 1, i32(5, 5), i32(3, 4, 5, 6)), *same)          # 10 ids
u = kvx.BatchTables(2, 40, 8)
kvx.build_tables(u, 16, i32(1, 1), i32(7), have_len=i32(20, 5), held=t.table)
refused(SHAPE, lambda: kvx.build_tables(u, 16, i32(1, 1), i32(7), have_len=i32(20, 5),
                                        held=kvx.Table(i64(0, 8, 9), t.page_ids)), u.slots)

k = torch.randn(25, 2, 64, device=dev).to(torch.bfloat16)
kvx.append(lay, 0, pool, t.slots, k, k)
torch.cuda.synchronize()
assert torch.equal(store.view(2, 256, 2, 64)[1, 80:85], k[20:])
twice = t.slots[:25].clone()
twice[7] = twice[3]
refused(DUPLICATE, lambda: kvx.append(lay, 0, pool, twice, k, k), store)
out_of_pool = t.slots[:25].clone()
out_of_pool[7] = out_of_pool[3] = -1
kvx.append(lay, 0, pool, out_of_pool, k, k)                     # skipped rows are no duplicates

q = torch.randn(25, 4, 64, device=dev).to(torch.bfloat16)
plain = [torch.full_like(q, 7.0) for _ in range(2)]
def attend(out, reqs=None, ctx=None, prefix=None):
    kvx.attend(lay, 0, pool, reqs or t.requests(25), ctx if ctx is not None else t.ctx_len, t.table,
               q, out, prefix=prefix)
attend(plain[0])
pre = lambda off, n: kvx.Prefix(i64(*off), i32(n), t.table)
attend(plain[1], prefix=pre((0, 2), 16))
torch.cuda.synchronize()
assert not (plain[0] == 7.0).all() and not torch.equal(plain[0], plain[1])
bad = lambda *x: kvx.Requests(i64(*x), 25)
refused(SHAPE, lambda: attend(plain[0], bad(0, 20, 26)), plain[0])
refused(SHAPE, lambda: attend(plain[0], bad(0, 26, 25)), plain[0])
refused(SHAPE, lambda: attend(plain[0], bad(1, 20, 25)), plain[0])
refused(SHAPE, lambda: attend(plain[0], ctx=i32(20, -5)), plain[0])
refused(SHAPE, lambda: attend(plain[0], ctx=i32(20, 2 ** 30 + 1)), plain[0])
refused(SHAPE, lambda: attend(plain[0], prefix=pre((0, 1), 16)), plain[0])
refused(SHAPE, lambda: attend(plain[0], prefix=pre((0, 2), -1)), plain[0])
print("validate ok", flush=True)
"""


def test_validate_mode_refuses_broken_tables():
    p = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], capture_output=True,
                       text=True, timeout=120, env=dict(os.environ, KVX_VALIDATE="1"), cwd=ROOT)
    assert p.returncode == 0, p.stdout + p.stderr
    assert "validate ok" in p.stdout
    for call in ("request 1's lengths", "append: slot", "attend: KVX_E_SHAPE"):
        assert call in p.stderr, call


CHILD_OVERLAP = r"""
import sys
sys.path.insert(0, {root!r})
import torch
import scatter_kvx_gather_amd as kvx

dev = torch.device("cuda:0")
for bl in ("nhd", "hnd"):
    for dtype in ("bf16", "fp8"):
        t = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
        lay = kvx.Layout(2, 2, 2, 64, dtype)
        store = (torch.arange(4 * 8 * 4 * 128, device=dev) % 200).view(4, 8, 4, 2, 64).to(torch.bfloat16).to(t)
        pool = kvx.Pool(store, 8, 4)
        slots = torch.tensor([8, -1, 10, 11], device=dev)           # in page 2
        page = lambda plane, p: store[plane, p].view(torch.uint8).view(4, 2, -1).view(t)
        before = store.clone()
        # page 2 of another layer, and page 3 of this one, are not written: a page is copied
        for k, v in ((page(0, 2), page(1, 2)), (page(2, 3), page(3, 3)), (page(3, 1), page(2, 1))):
            kvx.append(lay, 1, pool, slots, k, v, block_layout=bl)
        torch.cuda.synchronize()
        assert not torch.equal(store.view(torch.uint8), before.view(torch.uint8))
        store.copy_(before)
        for k, v in ((page(2, 2), page(0, 0)), (page(0, 0), page(2, 2)), (page(3, 2), page(0, 0)),
                     (store[2].view(t).reshape(32, 2, 64)[5:9], page(0, 0))):
            torch.cuda.synchronize()
            try:
                kvx.append(lay, 1, pool, slots, k, v, block_layout=bl)
            except kvx.KvxError as e:
                assert e.status == 9, e.status
            else:
                raise AssertionError("not refused")
            torch.cuda.synchronize()
            assert torch.equal(store.view(torch.uint8), before.view(torch.uint8))
print("overlap ok", flush=True)
"""


def test_validate_mode_refuses_appended_rows_that_are_written():
    """Rows of k and v that lie in the slots that the call writes; others of the
    same pool may be appended (a page copied to another)."""
    p = subprocess.run([sys.executable, "-c", CHILD_OVERLAP.format(root=ROOT)], capture_output=True,
                       text=True, timeout=120, env=dict(os.environ, KVX_VALIDATE="1"), cwd=ROOT)
    assert p.returncode == 0, p.stdout + p.stderr
    assert "overlap ok" in p.stdout
    assert "append: a row is read and written" in p.stderr
