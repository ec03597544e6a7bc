"""Keys that hold infinities (bf16 caches): scores of -inf have weight zero, however many of them come first.  Against
attention in 64 bits over the other keys; a row of which no key is left is zero.  Bounds in attention_ref.py."""
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv

from attention_ref import attend, check, gather
from test_gpu_cross import Batch as Cross
from test_gpu_prefix import Batch as Prefix

pytestmark = pytest.mark.gpu


def _blind(b, table, positions):
    """-inf in the first dim of these positions' keys; every query's first dim is positive, so their scores are -inf."""
    for p in positions:
        b.k[int(table[p // b.S]) - getattr(b, "far", 0), p % b.S, :, 0] = float("-inf")


def _reference(b, q, table, length, blind, tile):
    keep = torch.tensor([p for p in range(length) if p not in blind], dtype=torch.int64)
    k, v = (gather(c, table, length)[keep] for c in (b.k, b.v))
    return attend(q, k, v, b.scale, "bf16", 1.0, 1.0, tile)


CROSS = [(5, 200, range(64)), (70, 200, range(130)), (1, 9999, range(5000)), (3, 300, range(64, 128)), (2, 80, range(80)),
         (300, 129, range(128))]


@pytest.mark.parametrize("G", [1, 4])
def test_cross_attention(G):
    """The first key tile, the first two, whole pieces of a cut item, every second tile of a single query tile, all."""
    b = Cross([t for t, _, _ in CROSS], [n for _, n, _ in CROSS], 2, G, 16, "bf16", seed=40 + G)
    b.q[..., 0] = b.q[..., 0].abs() + 1
    for s, (_, _, blind) in enumerate(CROSS):
        _blind(b, b.tables[s], blind)
    b.device().run()
    torch.cuda.synchronize()
    assert int(b.err) == 0
    for s, (_, n, blind) in enumerate(CROSS):
        rows = slice(b.cu[s], b.cu[s + 1])
        check(b.out[rows], *_reference(b, b.q[rows], b.tables[s], n, blind, True), f"sequence {s}")
    assert (b.out[b.cu[4]:b.cu[5]] == 0).all()


@pytest.mark.parametrize("G", [1, 4, 8])
def test_single_tokens(G):
    """The decode on CUDA cores (G = 1, 4) and tensor cores (8): first blocks, whole shares, all."""
    cases = [(200, range(64)), (40, range(16)), (9000, range(5000)), (33, range(33)), (65, range(64))]
    b = Cross([1] * len(cases), [n for n, _ in cases], 2, G, 16, "bf16", seed=50 + G)
    b.q[..., 0] = b.q[..., 0].abs() + 1
    for s, (_, blind) in enumerate(cases):
        _blind(b, b.tables[s], blind)
    b.device().run(single=True)
    torch.cuda.synchronize()
    assert int(b.err) == 0
    for s, (n, blind) in enumerate(cases):
        check(b.out[s:s + 1], *_reference(b, b.q[s:s + 1], b.tables[s], n, blind, False), f"sequence {s}")
    assert (b.out[3] == 0).all()


@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("what", ["first tile", "prefix", "own", "all"])
def test_shared_prefixes(what, G):
    """-inf in the prefix's first key tile, in all of it, in the sequences' own keys, everywhere."""
    own = [70, 1, 20, 200]
    b = Prefix([(192, own), (64, [3, 90])], 2, G, 16, "bf16", seed=60 + G)
    b.q[..., 0] = b.q[..., 0].abs() + 1
    blind = {"first tile": range(64), "prefix": range(192), "own": range(192, 392), "all": range(392)}[what]
    for s in range(4):
        row = b.tables[s].clone()
        row[:12] = b.heads[0]
        _blind(b, row, [p for p in blind if p < b.lens[s]])
    out = b.device().run()
    torch.cuda.synchronize()
    assert int(b.err) == 0
    for s in range(6):
        g = 0 if s < 4 else 1
        row = b.tables[s].clone()
        row[: len(b.heads[g])] = b.heads[g]
        ref, bound = _reference(b, b.q[s:s + 1], row, b.lens[s], blind if g == 0 else (), True)
        check(out[s:s + 1], ref, bound, f"{what}, sequence {s}")
    if what == "all":
        assert (out[:4] == 0).all()


@pytest.mark.parametrize("blind,start", [(range(64), 100), (range(64), 20), (range(130), 100)])
def test_prefill_chunk(blind, start):
    b = Cross([100], [start + 100], 2, 4, 16, "bf16", seed=70)
    b.q[..., 0] = b.q[..., 0].abs() + 1
    _blind(b, b.tables[0], blind)
    b.device()
    pkv.pkv_paged_prefill_chunk(b.out, b.dq, start, b.dk, b.dv, b.desc, b.dt[0], start + 100, b.scale, b.err)
    torch.cuda.synchronize()
    assert int(b.err) == 0
    for i in range(0, 100, 9):
        check(b.out[i:i + 1], *_reference(b, b.q[i:i + 1], b.tables[0], start + i + 1, blind, True), f"token {i}")
    none = len(blind) - start
    assert none <= 0 or (b.out[:none] == 0).all()
