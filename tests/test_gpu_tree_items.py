"""Draft trees (pkv_paged_attention_tree) in batches that give every SM several items, or more of them than it lists at a time:
what is kept per listed item, and what the two query tiles of an item tell each other."""
import random

import pytest
import torch

from attention_ref import check, gather
from test_gpu_tree import Batch
from tree_ref import attend_masked, seen_keys

pytestmark = pytest.mark.gpu
KV = ["bf16", "fp8", "int8"]


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


@pytest.mark.parametrize("kv", KV)
def test_more_items_than_an_sm_lists(kv):
    """1024 runs of none to three tokens over 32 KV heads: more than 128 items for every SM, whose list is filled again."""
    r = random.Random(22)
    sizes = [r.choice((1, 2, 3, 3, 3)) if i % 11 else 0 for i in range(1024)]
    items = 32 * sum(n > 0 for n in sizes)
    assert items > 128 * torch.cuda.get_device_properties(0).multi_processor_count
    b = Batch([[r.getrandbits(n) | 1 for _ in range(n)] for n in sizes], [r.randrange(14) for _ in sizes], 32, 1, 8, kv, seed=22)
    odd = {}
    for s in range(0, 1024, 7):
        if kv == "int8" or sizes[s] == 0:
            continue
        j, h = sizes[s] - 1, r.randrange(32)
        if any(b.runs[s][i] >> j & 1 for i in range(sizes[s]) if i != j) or not b.runs[s][j] >> j & 1:
            continue  # seen by itself alone
        blk, off = b.place(s, b.lens[s] - 1)
        b.v.view(torch.uint8 if kv == "fp8" else torch.int16)[blk, off, h, 100:] = 0x7f if kv == "fp8" else 0x7fc0
        odd[s] = j, h, 100, float("nan")
    b.device().run()
    _verify_odd(b, odd, f"{kv}, refilled lists")


# (tokens, keys before) of each run: items whose lengths differ so much that a quarter of the SMs take nothing of the rest; two
# rounds of items of about one length, cut where it falls
ROUNDS = {"uneven": ([406, 558, 342, 446, 523, 324, 302, 370, 495, 504, 417, 370],
                     [2100, 1900, 1900, 2100, 6212, 2100, 1900, 2100, 1900, 2100, 1900, 2100]),
          "two": ([500, 449, 512, 513, 470, 555, 481, 460, 560, 490, 511, 449, 530, 502, 466, 497],
                  [1900 + 77 * i for i in range(16)])}


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("lengths", ROUNDS)
def test_whole_items_in_rounds(kv, lengths):
    """Runs of five query-tile pairs and more over the same keys: whole items in rounds, then a stream of the rest.  What makes the
    plan take rounds is asserted in its own units (a key tile of two query tiles 10, an item 30 and more)."""
    tokens, past = ROUNDS[lengths]
    Hkv, G, sms = 4, 4, torch.cuda.get_device_properties(0).multi_processor_count
    units = [10 * -(-(p + n) // 64) + 30 for n, p in zip(tokens, past) for _ in range(-(-n // 64) * Hkv)]
    assert len(units) >= 2 * len(tokens) * Hkv and len(units) >= 2 * sms and sum(units) >= 320 * len(units)
    share = -(-sum(units) // sms)
    if lengths == "uneven":
        assert sum(u >= share for u in units[:sms]) >= 10  # one round; these SMs have no part of the rest
    else:
        assert len(units) // sms == 3  # two rounds
    r = random.Random(23)
    words = -(-max(tokens) // 64) * 64
    b = Batch([[r.getrandbits(words) & (1 << n) - 1 for _ in range(n)] for n in tokens], past, Hkv, G, 16, kv, seed=23).device().run()
    torch.cuda.synchronize()
    assert int(b.err) == 0
    for s in range(b.n):  # in 64 bits on the GPU
        a, e, L = b.cu[s], b.cu[s + 1], b.lens[s]
        k, v = gather(b.k, b.tables[s], L).cuda(), gather(b.v, b.tables[s], L).cuda()
        ks, vs = (torch.full((Hkv,), x, dtype=torch.float64, device="cuda") for x in (b.ks, b.vs))
        j = torch.arange(e - a)
        seen = torch.ones(e - a, L, dtype=torch.bool)
        seen[:, L - (e - a):] = b.mask[a:e][:, j // 64] >> j % 64 & 1 != 0
        rows = slice(s % 3, None, 3)  # every third token, of every tile
        ref, bound = attend_masked(b.dq[a:e][rows], k, v, seen[rows].cuda(), b.scale, kv, ks, vs)
        check(b.out[a:e][rows], ref.cpu(), bound.cpu(), f"{kv} {lengths}, sequence {s}")
