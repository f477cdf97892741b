"""Attention over 4-bit pools whose tables have room for a large batch, over head
layouts and dims together: decode batches with contexts of several stages of the
ring, ragged, with pages out of range and prefixes, against the 64-bit softmax."""
import numpy as np
import pytest
import torch

from tests import fp4_ref as f4
from tests.fp4_util import Fp4Case
from tests.gpu_util import say
from tests.serve_util import DEV

pytestmark = pytest.mark.gpu

DIMS = [32, 64, 96, 128, 160, 192, 224, 256]


def batch(monkeypatch, H, G, D, page, layout, prefix=0):
    monkeypatch.setattr(Fp4Case, "roomy", True)
    rng = np.random.default_rng(H * 10000 + G * 300 + D)
    ctx = [1, 64, 65, 85, 127, 128, 129, 200, 300, 0, 517]
    n = len(ctx)
    extra = dict(members=[0, n], prefix=[prefix]) if prefix else {}
    c = Fp4Case(G, new=[1] * n, ctx=ctx, H=H, G=G, D=D, page=page, layout=layout, bad=0.03, **extra)
    # blocks of NaN in the newest rows of one request
    rows = [x for x in c.b.rows(c.b.pg_off[6], c.b.ids, ctx[6])[-2:] if x is not None]
    for x in rows:
        c.scales[1][x, rng.integers(0, H), D // 32 - 1] = f4.NAN_SCALE
    c.decode()
    c.upload()
    skipped = torch.zeros(1, dtype=torch.int64, device=DEV)
    out, lse = c.run(skipped=skipped)
    torch.cuda.synchronize()
    c.check(out, lse)
    assert skipped.item() == c.b.skipped()
    again, lse2 = c.run()
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


@pytest.mark.parametrize("G", [17, 20, 32])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("page", [1, 16])
def test_one_kv_head_in_two_parts(monkeypatch, G, D, page):
    """Four waves share a part's keys, and a stage is 128 of them."""
    say("fp4 ring, one kv head", G, D, page)
    batch(monkeypatch, 1, G, D, page, "nhd", prefix=0 if G == 20 else 140)


@pytest.mark.parametrize("H,G", [(1, 40), (2, 1), (2, 16), (2, 17), (3, 5), (4, 4), (5, 2), (8, 1), (9, 3)])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_heads_and_dims(monkeypatch, H, G, D, layout):
    say("fp4 ring, heads and dims", H, G, D, layout)
    batch(monkeypatch, H, G, D, 16 if layout == "hnd" else 4, layout)
