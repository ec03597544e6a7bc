"""Draft trees (pkv_paged_attention_tree) in batches that give every SM several items: what is kept per item, and what the two
query tiles of an item tell each other."""
import random

import pytest
import torch

from attention_ref import check, gather
from test_gpu_tree import Batch
from tree_ref import attend_masked, seen_keys

pytestmark = pytest.mark.gpu


def _verify_odd(b, odd, what):
    """odd: {sequence: (token, KV head, first dim, value)}: dims from there on of that token's value."""
    torch.cuda.synchronize()
    assert int(b.err) == 0
    G = b.Hq // b.k.shape[2]
    for s in range(b.n):
        a, e, L = b.cu[s], b.cu[s + 1], b.lens[s]
        if a == e:
            continue
        k, v = gather(b.k, b.tables[s], L), gather(b.v, b.tables[s], L)
        ref, bound = attend_masked(b.q[a:e], k, v, seen_keys(e - a, L, b.runs[s]), b.scale, b.kv, b.ks, b.vs)
        got = b.out[a:e].cpu().float()
        if s in odd:
            j, h, d, x = odd[s]
            hit = torch.zeros(got.shape, dtype=torch.bool)
            hit[j, h * G:(h + 1) * G, d:] = True
            assert (torch.isnan(got[hit]) if x != x else got[hit] == x).all(), f"{what}, sequence {s}: the row that sees it"
            got, ref = (torch.where(hit, torch.zeros_like(t), t) for t in (got, ref))
        check(got, ref, bound, f"{what}, sequence {s}")


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_odd_values_among_several_items_of_two_tiles(kv):
    """300 runs of 33 tokens of four heads a KV head (132 rows) that see themselves alone: 1200 items, eight on every SM.  In every
    third sequence one KV head's values of one token are infinite or no numbers from some dim on.  The same bits in every call."""
    r = random.Random(21)
    b = Batch([[1 << i for i in range(33)]] * 300, [r.randrange(1, 130) for _ in range(300)], 4, 4, 16, kv, seed=21)
    odd = {}
    for s in range(0, 300, 3):
        j, h, d = r.randrange(33), r.randrange(4), r.randrange(128)
        x = float("nan") if kv == "fp8" else r.choice((float("inf"), float("-inf"), float("nan")))
        blk, off = b.place(s, b.lens[s] - 33 + j)
        if kv == "fp8":
            b.v.view(torch.uint8)[blk, off, h, d:] = 0x7f
        else:
            b.v[blk, off, h, d:] = x
        odd[s] = j, h, d, x
    b.device().run()
    _verify_odd(b, odd, kv)
    first = b.out.view(torch.int16).clone()
    for call in range(30):
        b.out.fill_(7.0)
        assert torch.equal(b.run().out.view(torch.int16), first), call
