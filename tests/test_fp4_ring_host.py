"""The ring of 4-bit attention on the host (no GPU): for every shape that the
host sends through it, what a stage's loads bring and what its flags tell is
worked out index by index.  The library says in its log which shapes those are;
it is asked without a GPU, and its launches fail."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

ASK = r"""
import ctypes, itertools, sys
import torch
import scatter_kvx_gather_amd as kvx
from tests import fp4_ref as f4
assert not torch.cuda.is_available()
A = 0x7F0000000000
lib = kvx.load_library()
arr = (ctypes.c_void_p * 2)(A + (8 << 30), A + (16 << 30))
for hnd, D, H, G in itertools.product((0, 1), range(32, 257, 32), HEADS, QUERIES):
    R = f4.row_bytes(H, D)
    if G * H > 256:
        continue
    p = kvx._CPool(ctypes.cast(arr, ctypes.POINTER(ctypes.c_void_p)), 1 << 20, 16, R, 0)
    a = kvx._CAttention(q=A, out=A + (1 << 32), lse=None, q_stride=G * H * D * 2, out_stride=G * H * D * 2,
                        q_heads=G * H, dtype=2, scale=0.1, k_scale=1.0, v_scale=1.0, flags=1,
                        workspace=A + (1 << 40), workspace_bytes=1 << 40)
    print("ask", hnd, D, H, G, file=sys.stderr, flush=True)
    st = lib.kvx_attend(kvx._CLayout(1, 2, H, D, 5), 0, p, hnd, kvx._CReqs(4, 4, A), A,
                        kvx._CTable(A, A, 1 << 30), None, a, None, None)
    assert st not in (0, 1, 2, 3, 4, 5, 6, 9), (hnd, D, H, G, st)
"""


def asked(heads, queries):
    """(hnd, D, H, G) -> how thin tiles get their keys, pieces of a row, waves that share a head's keys."""
    env = dict(os.environ, KVX_LOG="1", HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1",
               PYTHONPATH=ROOT)
    env.pop("KVX_VALIDATE", None)
    r = subprocess.run([sys.executable, "-c", f"HEADS = {heads}\nQUERIES = {queries}\n" + ASK], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    got, at = {}, None
    for line in r.stderr.splitlines():
        if line.startswith("ask "):
            at = tuple(int(x) for x in line.split()[1:])
        m = re.search(r"kvx: attend .* own=(\w+) thin_keys=(\w+) pieces=(\d+) waves_a_head=(\d+)", line)
        if m:
            got[at] = (m[1], m[2], int(m[3]), int(m[4]))
    return got


def stage(D, pieces, kp):
    """Rows that an NHD stage's loads bring for another key's, and keys of which no wave
    tells whether they are there.  A stage is 64 kp rows of `pieces` 16-byte pieces, K's
    and then V's; waves take its loads of 64 pieces in runs; a lane looks up one key, and a
    load takes the offset of lane (row - first row) % 64."""
    NJ = 2 if D <= 64 else (4 if D <= 128 else 8)
    keys, loads = 32 * kp, kp * pieces
    extra = max(0, loads - 8 * NJ)
    wrong, told = set(), set()
    for wave in range(8):
        load0 = wave * NJ + min(wave, extra)
        row0 = load0 * 64 // pieces
        told |= {(row0 + lane) % keys for lane in range(64) if row0 + lane < keys}
        for load in range(load0, min(loads, load0 + NJ + (wave < extra))):
            for r in {p // pieces for p in range(load * 64, load * 64 + 64)}:
                if r < 2 * keys and (row0 + (r - row0) % 64) % keys != r % keys:
                    wrong.add(r)
    return wrong, set(range(keys)) - told


def test_stage_model():
    """The model itself, where one look-up a lane is enough and where it is not."""
    assert stage(128, 34, 1) == (set(), set())
    assert stage(256, 9, 4) == (set(), set())
    wrong, untold = stage(160, 6, 4)
    assert len(wrong) == 66 and untold == set(range(64, 85))
    wrong, untold = stage(192, 7, 4)
    assert len(wrong) == 30 and untold == set(range(64, 73))


@pytest.mark.parametrize("heads", ["(1, 2, 3)", "range(4, 33)"])
def test_every_staged_key_is_its_own(heads):
    got = asked(heads, "range(1, 64)" if heads == "(1, 2, 3)" else "(1, 2, 3, 8, 16, 17, 20, 32, 33, 40)")
    ring = {k: v for k, v in got.items() if v[1] == "ring"}
    assert len(ring) > 100
    for (hnd, D, H, G), (own, _, pieces, kp) in ring.items():
        # head-major stages address tiles, whose first keys are all of one look-up
        assert kp <= 2 if hnd else stage(D, pieces, kp) == (set(), set()), (hnd, D, H, G, pieces, kp)
