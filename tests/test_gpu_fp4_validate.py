"""KVX_VALIDATE=1 (debug mode) for 4-bit pools and kvx_read on the GPU, in a
child process (the flag is read once per process): good calls run as without it,
and slots written twice and rows that are read and written are refused with their
status, with nothing written."""
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
DUPLICATE, OVERLAP = 8, 9

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
        assert torch.equal(x, y)

for layout in ("nhd", "hnd"):
    H, D, page, P = 2, 64, 16, 8
    lay = kvx.Layout(1, 2, H, D, "fp4")
    R = lay.row_bytes
    store = torch.zeros(2, P, page * R, dtype=torch.uint8, device=dev)
    pool = kvx.Pool(store, P, page, slot_stride=R)
    k = torch.randn(6, H, D, device=dev).to(torch.bfloat16)
    slots = torch.tensor([5, 100, -1, 17, P * page, 16], device=dev)
    kvx.append(lay, 0, pool, slots, k, k, block_layout=layout)
    out = [torch.zeros_like(k) for _ in range(2)]
    kvx.read(lay, 0, pool, slots, out[0], out[1], block_layout=layout)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and out[0][0].any() and not out[0][2].any()
    twice = slots.clone()
    twice[3] = 5
    refused(DUPLICATE, lambda: kvx.append(lay, 0, pool, twice, k, k, block_layout=layout), store)
    kvx.read(lay, 0, pool, twice, out[0], out[1], block_layout=layout)      # read twice is fine
    torch.cuda.synchronize()
    assert torch.equal(out[0][3], out[0][0])

    # rows that lie in the pool: dense rows as views of its own bytes
    flat = store.view(-1).view(torch.bfloat16)
    rows = flat[:6 * H * D].view(6, H, D)       # over slots 0 .. of the K plane
    far = torch.tensor([120, 121, 122, 123, 124, 125], device=dev)
    near = torch.tensor([0, 1, 122, 123, 124, 125], device=dev)
    refused(OVERLAP, lambda: kvx.append(lay, 0, pool, near, rows, k, block_layout=layout), store)
    kvx.append(lay, 0, pool, far, rows, k, block_layout=layout)
    refused(OVERLAP, lambda: kvx.read(lay, 0, pool, near, rows, out[1], block_layout=layout), store)
    kvx.read(lay, 0, pool, far, rows, out[1], block_layout=layout)
    torch.cuda.synchronize()
print("child ok", flush=True)
"""


def test_validate_mode():
    env = dict(os.environ, KVX_VALIDATE="1")
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], env=env, cwd=ROOT,
                       capture_output=True, text=True, timeout=110)
    assert r.returncode == 0 and "child ok" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
