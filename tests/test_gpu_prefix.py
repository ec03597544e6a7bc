"""Decode attention over groups of sequences that share prefixes (pkv_paged_attention_decode_prefix) against attention in
64 bits over each whole sequence; bounds in attention_ref.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B
from paged_kv_cache_71_gb300 import workload as wl
from paged_kv_cache_71_gb300.runner import DeviceStep

from attention_ref import SCALE, attend, check, gather, make_cache
from parity import assert_close, oracle_step, to_host

pytestmark = pytest.mark.gpu
D = 128


class Batch:
    """groups: [(prefix tokens, [own tokens of each sequence])]."""

    def __init__(self, groups, Hkv, G, S, kv, seed, head_scales=False, far=0):
        gen = torch.Generator().manual_seed(seed)
        self.kv, self.S, self.Hkv, self.Hq = kv, S, Hkv, Hkv * G
        rows, lens, cu, pre, at = [], [], [0], [], 0
        for p, own in groups:
            head = list(range(at, at + p // S))
            at += p // S
            for i, x in enumerate(own):
                b = -(-x // S)
                # only the group's first row names the prefix: the others' entries there are not read
                rows.append((head if i == 0 else [-1] * len(head)) + list(range(at, at + b)))
                lens.append(p + x)
                at += b
            cu.append(len(rows))
            pre.append(p)
        nb = at + 3
        self.B = len(rows)
        perm = torch.randperm(nb, generator=gen) + far
        self.tables = torch.full((self.B, max(len(r) for r in rows) + 2), -1, dtype=torch.int32)
        for i, r in enumerate(rows):
            self.tables[i, : len(r)] = torch.tensor([int(perm[b]) if b >= 0 else -1 for b in r], dtype=torch.int32)
        self.heads = [self.tables[cu[g], : p // S].clone() for g, p in enumerate(pre)]
        self.k, self.v = make_cache(gen, (nb, S, Hkv, D), kv), make_cache(gen, (nb, S, Hkv, D), kv)
        self.far = far
        used = torch.zeros(nb, S, dtype=torch.bool)  # slots that hold a token
        for g, p in enumerate(pre):
            used[(self.heads[g] - far).long()] = True
            for s in range(cu[g], cu[g + 1]):
                for pos in range(p, lens[s]):
                    used[int(self.tables[s, pos // S]) - far, pos % S] = True
        if kv != "int8":  # everything else is not a number
            nan = 0x7f if kv == "fp8" else 0x7fc0
            for c in (self.k, self.v):
                c.view(torch.uint8 if kv == "fp8" else torch.int16)[~used] = nan
        self.q = torch.randn(self.B, self.Hq, D, generator=gen).to(torch.bfloat16)
        self.lens, self.cu, self.pre = lens, cu, pre
        self.scale = 1 / np.sqrt(D)
        self.ks = self.vs = SCALE[kv]
        if head_scales:
            self.ks = (torch.rand(Hkv, generator=gen) + 0.5) * SCALE[kv]
            self.vs = (torch.rand(Hkv, generator=gen) + 0.5) * SCALE[kv]

    def reference(self, seqs=None):
        outs, bounds = [], []
        for s in range(self.B) if seqs is None else seqs:
            g = int(np.searchsorted(self.cu, s, side="right")) - 1
            p = self.pre[g] // self.S
            row = self.tables[s].clone()
            row[:p] = self.heads[g]
            row = row - self.far
            k, v = gather(self.k, row, self.lens[s]), gather(self.v, row, self.lens[s])
            # the prefix and the rest round their weights differently: the looser of the two bounds
            o, b = attend(self.q[s:s + 1], k, v, self.scale, self.kv, self.ks, self.vs, True)
            b2 = attend(self.q[s:s + 1], k, v, self.scale, self.kv, self.ks, self.vs, False)[1]
            outs.append(o)
            bounds.append(torch.maximum(b, b2))
        return torch.cat(outs), torch.cat(bounds)

    def device(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        if self.far:
            self.dk = torch.zeros((self.far + self.k.shape[0], *self.k.shape[1:]), dtype=self.k.dtype, device="cuda")
            self.dv = torch.zeros_like(self.dk)
            self.dk[self.far:].copy_(self.k)
            self.dv[self.far:].copy_(self.v)
        else:
            self.dk, self.dv = self.k.cuda(), self.v.cuda()
        heads = {}
        if torch.is_tensor(self.ks):
            self.dks, self.dvs = self.ks.cuda(), self.vs.cuda()
            heads = dict(k_head_scales=self.dks, v_head_scales=self.dvs)
        sc = 1.0 if heads else SCALE[self.kv]
        self.desc = pkv.CacheDesc.for_cache(self.dk, sc, sc, **heads)
        self.dq, self.dt = self.q.cuda(), self.tables.cuda()
        self.dl, self.dcu, self.dp = (torch.tensor(x, **i32) for x in (self.lens, self.cu, self.pre))
        self.out = torch.full_like(self.dq, float("nan"))
        self.ws = torch.full((pkv.pkv_paged_attention_decode_prefix_workspace_size(self.desc, self.B, self.Hq),), 0xff,
                             dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, **i32)
        return self

    def run(self, stream=None):
        pkv.pkv_paged_attention_decode_prefix(self.out, self.dq, self.dk, self.dv, self.desc, self.dt, self.dl, self.dcu,
                                              self.dp, self.scale, self.ws, self.err, stream)
        return self.out


def _check(b, what, seqs=None):
    out = b.device().run()
    torch.cuda.synchronize()
    assert int(b.err) == 0
    ref, bound = b.reference(seqs)
    check(out if seqs is None else out[list(seqs)], ref, bound, what)
    return out


RAGGED = [(64, [1, 17, 0, 300, 33]), (0, [1, 0, 70]), (32, [5]), (1312, [64, 2, 129]), (96, [0])]


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_ragged_groups_every_head_group(kv, G):
    """Five groups: prefixes of none to 1312 tokens (key tiles that end inside), sequences without own tokens, without
    any token, of one token, and long enough to be split."""
    _check(Batch(RAGGED, 2, G, 16, kv, seed=G), f"{kv} G={G}")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("S", [8, 32])
def test_block_sizes_and_an_odd_head_count(kv, S):
    _check(Batch([(32, [1, 40, 9]), (800, [3, 0, 64, 65])], 3, 4, S, kv, seed=S), f"{kv} S={S}")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_a_long_prefix_cut_into_many_pieces(kv):
    """One KV head and few rows: the whole GPU shares one prefix, whose pieces every sequence joins."""
    _check(Batch([(9008, [1, 77, 0])], 1, 8, 16, kv, seed=3), f"{kv} cut prefix")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_groups_of_many_query_tiles(kv):
    """A group of 150 sequences (600 rows a KV head: three pairs of query tiles, the last one partly filled) beside one of
    65 (one full tile and one row group in the second)."""
    b = Batch([(208, [1 + i % 40 for i in range(150)]), (80, [i % 3 for i in range(65)])], 2, 4, 16, kv, seed=4)
    _check(b, f"{kv} many tiles")


@pytest.mark.parametrize("kv", ["fp8", "int8"])
def test_per_head_scales(kv):
    _check(Batch(RAGGED, 2, 4, 16, kv, seed=5, head_scales=True), f"{kv} per-head scales")


def test_more_items_than_a_block_lists_at_a_time():
    """160 groups of 128 KV heads: 20480 prefixes of one key tile, so that a share has more items than are listed at once."""
    _check(Batch([(16, [1, i % 3]) for i in range(160)], 128, 1, 16, "bf16", seed=16), "many items", range(0, 320, 23))


def test_groups_without_sequences():
    _check(Batch([(48, []), (64, [1, 20]), (32, []), (0, []), (160, [33])], 2, 4, 16, "bf16", seed=17), "empty groups")


def test_single_sequence_and_no_prefix_at_all():
    _check(Batch([(0, [1])], 8, 4, 16, "bf16", seed=6), "one token")
    _check(Batch([(16, [0])], 8, 4, 16, "bf16", seed=6), "one block, no own tokens")
    _check(Batch([(0, [500, 3, 0, 40])], 4, 4, 16, "bf16", seed=7), "no prefix")


def test_large_scores_and_a_dominating_part():
    """Keys 30 times larger: softmax rows that one key decides, from either part."""
    b = Batch([(320, [40, 300, 1])], 2, 4, 16, "bf16", seed=8)
    b.k = (b.k.float() * 30).to(torch.bfloat16)
    _check(b, "large scores")


def test_blocks_past_four_gigabytes():
    """A pool of 5.4 GB per tensor (8 heads, 16-token blocks of 32 KB), the batch's blocks at its end."""
    _check(Batch([(160, [20, 1]), (0, [33])], 8, 4, 16, "bf16", seed=9, far=165000), "far blocks")


def test_the_prefix_sharing_batch_against_the_oracle():
    w = wl.prefix_shared()
    st = DeviceStep(w)
    st.write()
    cu = torch.tensor([0, w.num_seqs], dtype=torch.int32, device="cuda")
    pre = torch.tensor([800], dtype=torch.int32, device="cuda")
    ws = torch.empty(pkv.pkv_paged_attention_decode_prefix_workspace_size(st.cache, w.num_seqs, w.num_q_heads),
                     dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_attention_decode_prefix(st.out, st.q, st.k_cache, st.v_cache, st.cache, st.block_tables,
                                          st.context_lens, cu, pre, w.scale, ws, st.err)
    torch.cuda.synchronize()
    assert st.device_error() == 0
    assert_close("bf16", to_host(st.out), oracle_step(w)[2], "prefix-sharing batch")


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_calls_repeat_bit_for_bit_and_replay_from_a_graph(kv):
    """The same inputs give the same bits, eagerly and from a captured graph on another stream; new lengths and values
    reach the replay."""
    b = Batch(RAGGED, 2, 4, 16, kv, seed=10).device()
    first = b.run().clone()
    for _ in range(3):
        b.out.fill_(float("nan"))
        assert torch.equal(b.run(), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            b.run()
        b.out.fill_(float("nan"))
        graph.replay()
        side.synchronize()
        assert torch.equal(b.out, first)
        b.lens[3], b.lens[1] = b.lens[3] - 150, 64
        b.q = b.q.flip(0)
        b.dl.copy_(torch.tensor(b.lens, dtype=torch.int32))
        b.dq.copy_(b.q)
        graph.replay()
        side.synchronize()
    assert int(b.err) == 0
    ref, bound = b.reference()
    check(b.out, ref, bound, "replayed with other lengths")


def test_two_batches_on_two_streams():
    """Two calls at once, each with its own workspace."""
    bs = [Batch(RAGGED, 2, 4, 16, "bf16", seed=11 + i).device() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, st in zip(bs, streams):
            b.run(st)
    torch.cuda.synchronize()
    for b in bs:
        assert int(b.err) == 0
        check(b.out, *b.reference(), "concurrent calls")


@pytest.mark.parametrize("what", ["length", "prefix", "unaligned", "short", "uncovered"])
def test_bad_lengths_are_reported_and_the_other_groups_hold(what):
    """A bad group or length: BAD_LENGTH, zero rows for its sequences, the rest as ever."""
    b = Batch([(64, [3, 20]), (32, [5, 6]), (48, [70, 1])], 2, 4, 16, "bf16", seed=13).device()
    bad = [2, 3]
    if what == "length":
        b.dl[2], bad = -1, [2]
    elif what == "prefix":
        b.dp[1] = -16
    elif what == "unaligned":
        b.dp[1] = 31
    elif what == "short":
        b.dl[3], bad = 31, [3]
    else:
        b.dcu[3], bad = 4, [4, 5]  # the last group ends before the batch does
    out = b.run()
    torch.cuda.synchronize()
    assert int(b.err) == B.DEVERR_BAD_LENGTH
    ref, bound = b.reference()
    good = [s for s in range(6) if s not in bad]
    assert (out[bad] == 0).all()
    check(out[good], ref[good], bound[good], what)


def test_a_bad_block_is_reported():
    b = Batch([(64, [3, 20]), (32, [5, 6])], 2, 4, 16, "bf16", seed=14).device()
    b.dt[0, 1] = 10 ** 6  # in the first group's prefix
    out = b.run()
    torch.cuda.synchronize()
    assert int(b.err) & B.DEVERR_BAD_BLOCK
    ref, bound = b.reference()
    check(out[2:], ref[2:], bound[2:], "the other group")


def test_a_query_beyond_f16_is_reported_for_int8():
    b = Batch([(64, [3, 20])], 2, 4, 16, "int8", seed=15).device()
    b.dq[0, 0, 0] = 70000.0
    b.run()
    torch.cuda.synchronize()
    assert int(b.err) & B.DEVERR_Q_RANGE


def test_groups_that_overlap_beyond_what_can_be_counted_are_reported():
    """Every other group claims the whole batch: 1024 times 32 heads, 64 tiles and 512 key tiles are more units than 32 bits
    hold.  The prefixes are left out, reported, and nothing is read or written out of place."""
    n, Hkv, G, S, width = 2048, 32, 8, 8, 4096
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.zeros(2, S, Hkv, D, dtype=torch.bfloat16, device="cuda")
    desc = pkv.CacheDesc.for_cache(k)
    tables = torch.zeros(n, width, **i32)
    lens = torch.full((n,), width * S, **i32)
    cu = torch.tensor([0, n] * 1024 + [0], **i32)
    pre = torch.full((2048,), width * S, **i32)
    q = torch.zeros(n, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.zeros(pkv.pkv_paged_attention_decode_prefix_workspace_size(desc, n, Hkv * G), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, **i32)
    pkv.pkv_paged_attention_decode_prefix(out, q, k, k, desc, tables, lens, cu, pre, 0.1, ws, err)
    assert int(err) & B.DEVERR_BAD_LENGTH


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_a_workspace_aligned_to_16_bytes_only(kv):
    """Exactly as many bytes as asked for, at 16 bytes past a 512-byte boundary; what lies around stays as it is."""
    b = Batch(RAGGED, 2, 4, 16, kv, seed=18).device()
    call, verify = b.run, lambda: check(b.out, *b.reference(), f"{kv} workspace at an odd 16 bytes")
    need = b.ws.numel()
    room = torch.full((need + 1024,), 0xab, dtype=torch.uint8, device="cuda")
    at = -room.data_ptr() % 512 + 16
    b.ws = room[at:at + need]
    call()
    torch.cuda.synchronize()
    verify()
    assert (room[:at] == 0xab).all() and (room[at + need:] == 0xab).all()


@pytest.mark.parametrize("kv,S,G", [("bf16", 16, 1), ("int8", 32, 1), ("bf16", 32, 8), ("fp8", 8, 2)])
def test_the_largest_batch(kv, S, G):
    """8192 sequences in three groups, one of them without a prefix."""
    b = Batch([(64, [1 + i % 3 for i in range(5000)]), (0, [i % 40 for i in range(3000)]), (32, [2] * 192)], 2, G, S, kv, seed=19)
    _check(b, f"{kv} S={S} G={G}", [*range(0, 8192, 431), 4999, 5000, 5001, 7999, 8000, 8191])
