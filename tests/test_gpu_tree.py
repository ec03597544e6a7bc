"""Attention of drafted tokens (pkv_paged_attention_tree) against attention in 64 bits; bounds in attention_ref.py."""
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B

from attention_ref import SCALE, check, gather, make_cache
from tree_ref import ancestors, attend_masked, mask_words, random_tree, seen_keys

pytestmark = pytest.mark.gpu
D = 128


class Batch:
    """runs: per sequence a list of whole numbers (what each token sees of the run) or a number of tokens (a chain; then every
    run is one); past: keys before each run.  lead, tail: query rows that no sequence owns."""

    def __init__(self, runs, past, Hkv, G, S, kv, seed, lead=0, tail=0, head_scales=False, extra_words=0):
        gen = torch.Generator().manual_seed(seed)
        self.kv, self.S, self.Hq, self.n = kv, S, Hkv * G, len(runs)
        self.chain = not any(isinstance(r, list) for r in runs)
        self.runs = [None if self.chain else r for r in runs]
        self.tokens = [r if self.chain else len(r) for r in runs]
        self.lens = [p + t for p, t in zip(past, self.tokens)]
        self.cu = (lead + np.concatenate([[0], np.cumsum(self.tokens)])).astype(int).tolist()
        nb = sum(-(-L // S) for L in self.lens) + 2
        perm, at = torch.randperm(nb, generator=gen).to(torch.int32), 0
        self.tables = torch.full((self.n, max(1, max(-(-L // S) for L in self.lens))), -1, dtype=torch.int32)
        self.k, self.v = make_cache(gen, (nb, S, Hkv, D), kv), make_cache(gen, (nb, S, Hkv, D), kv)
        used = torch.zeros(nb, S, dtype=torch.bool)
        for s, L in enumerate(self.lens):
            b = -(-L // S)
            self.tables[s, :b] = perm[at:at + b]
            at += b
            pos = torch.arange(L)
            used[self.tables[s, pos // S].long(), pos % S] = True
        if kv != "int8":  # slots without a token are not numbers
            for c in (self.k, self.v):
                c.view(torch.uint8 if kv == "fp8" else torch.int16)[~used] = 0x7f if kv == "fp8" else 0x7fc0
        self.q = torch.randn(self.cu[-1] + tail, self.Hq, D, generator=gen).to(torch.bfloat16)
        self.q[:lead] = self.q[self.cu[-1]:] = float("nan")
        self.mask = None
        if not self.chain:
            W = max(1, -(-max(self.tokens) // 64)) + extra_words
            rows = mask_words(runs, W)
            self.mask = torch.full((self.q.shape[0], W), -1, dtype=torch.int64)
            self.mask[lead:self.cu[-1]] = rows
        self.scale = 1 / np.sqrt(D)
        self.ks = self.vs = SCALE[kv]
        if head_scales:
            self.ks = (torch.rand(Hkv, generator=gen) + 0.5) * SCALE[kv]
            self.vs = (torch.rand(Hkv, generator=gen) + 0.5) * SCALE[kv]

    def place(self, s, pos):
        return int(self.tables[s, pos // self.S]), pos % self.S

    def device(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        heads = {}
        if torch.is_tensor(self.ks):
            self.dks, self.dvs = self.ks.cuda(), self.vs.cuda()
            heads = dict(k_head_scales=self.dks, v_head_scales=self.dvs)
        sc = 1.0 if heads else SCALE[self.kv]
        self.dk, self.dv, self.dq, self.dt = self.k.cuda(), self.v.cuda(), self.q.cuda(), self.tables.cuda()
        self.desc = pkv.CacheDesc.for_cache(self.dk, sc, sc, **heads)
        self.dl, self.dcu = torch.tensor(self.lens, **i32), torch.tensor(self.cu, **i32)
        self.dm = None if self.mask is None else self.mask.cuda()
        self.out = torch.full_like(self.dq, 7.0)
        need = pkv.pkv_paged_attention_tree_workspace_size(self.desc, self.q.shape[0], self.n, self.Hq)
        self.ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, **i32)
        return self

    def run(self, stream=None):
        pkv.pkv_paged_attention_tree(self.out, self.dq, self.dcu, self.dl, self.dm, self.dk, self.dv, self.desc, self.dt,
                                     self.scale, self.ws, self.err, stream)
        return self

    def verify(self, what, skip=()):
        torch.cuda.synchronize()
        for s in range(self.n):
            a, b, L = self.cu[s], self.cu[s + 1], self.lens[s]
            if s in skip or a == b:
                continue
            k, v = gather(self.k, self.tables[s], L), gather(self.v, self.tables[s], L)
            ref, bound = attend_masked(self.q[a:b], k, v, seen_keys(b - a, L, self.runs[s]), self.scale, self.kv, self.ks, self.vs)
            check(self.out[a:b], ref, bound, f"{what}, sequence {s}")
        return self


def trees(seed, sizes):
    r = random.Random(seed)
    return [ancestors(random_tree(r, n)) for n in sizes]


SIZES = [1, 8, 0, 64, 65, 3, 130, 16]
PAST = [0, 1, 40, 63, 64, 700, 0, 1025]
KV = ["bf16", "fp8", "int8"]


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_ragged_trees(kv, G):
    """Runs of none to 130 tokens behind none to 1025 keys; rows that no sequence owns stay."""
    b = Batch(trees(G, SIZES), PAST, 2, G, 16, kv, seed=G, lead=3, tail=2).device().run()
    b.verify(f"{kv} G={G}")
    assert int(b.err) == 0
    assert (b.out[:3] == 7).all() and (b.out[-2:] == 7).all()


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("S", [8, 32])
def test_block_sizes_odd_head_counts_and_masks_wider_than_the_runs(kv, S):
    Batch(trees(S, [7, 40, 1]), [33, 500, 5], 3, 4, S, kv, seed=S, extra_words=1).device().run().verify(f"{kv} S={S}")


@pytest.mark.parametrize("kv", KV)
def test_chains_without_a_mask(kv):
    b = Batch([5, 1, 70, 0, 200], [1000, 0, 63, 9, 130], 2, 4, 16, kv, seed=3, lead=1).device().run().verify(f"{kv} chains")
    assert int(b.err) == 0


@pytest.mark.parametrize("kv", KV)
@pytest.mark.parametrize("past", [0, 62, 63, 64, 65])
def test_any_set_of_the_runs_tokens(kv, past):
    """Masks that are no tree: tokens that see later ones, not themselves, or nothing at all (zero rows where nothing is before
    the run), over runs that cross the borders of words and key tiles at different places."""
    r = random.Random(past)
    runs = [[0 if r.random() < 0.2 else r.getrandbits(n) for _ in range(n)] for n in (1, 2, 63, 64, 65, 128, 129)]
    runs.append([0, 1 << 1, 1 << 0])
    b = Batch(runs, [past] * len(runs), 1, 4, 16, kv, seed=past).device().run().verify(f"{kv} past {past}")
    if past == 0:
        a = b.cu[-2]
        assert (b.out[a] == 0).all() and (b.out[a + 1] != 0).any()


def test_bits_behind_the_run_are_ignored():
    runs = trees(5, [5, 17])
    b = Batch(runs, [100, 30], 2, 4, 16, "bf16", seed=5, extra_words=1).device()
    before = b.run().out.clone()
    high = torch.tensor([-1 << 5, -1], device="cuda")
    b.dm[:5] |= high
    b.dm[5:] |= torch.tensor([-1 << 17, -1], device="cuda")
    b.out.fill_(7.0)
    b.run()
    assert torch.equal(b.out, before)


@pytest.mark.parametrize("G", [16, 128])
def test_large_head_groups(G):
    Batch(trees(G, [3, 1, 9]), [100, 64, 333], 1, G, 16, "bf16", seed=G).device().run().verify(f"G={G}")


@pytest.mark.parametrize("kv", KV)
def test_one_item_over_the_whole_gpu(kv):
    """A few tokens against many keys: one item cut into a piece for every SM, the run's own keys in the last."""
    Batch(trees(1, [4]), [9999], 1, 4, 16, kv, seed=1).device().run().verify(f"{kv} cut item")


@pytest.mark.parametrize("kv", KV)
def test_own_keys_over_several_pieces(kv):
    """Runs longer than a share: the pieces of cut items each hold masked tiles, some rows see nothing in a piece."""
    r = random.Random(7)
    runs = [ancestors(random_tree(r, 700)), [1 << i for i in range(600)], [0] * 300]
    Batch(runs, [50, 0, 0], 1, 2, 16, kv, seed=7).device().run().verify(f"{kv} long runs")


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_several_long_items_for_every_sm(kv):
    """352 items: whole items in rounds, then a stream of the rest."""
    b = Batch(trees(9, [260, 40, 129, 5, 200, 250, 128, 257]), [3000, 4100, 0, 8000, 4500, 3333, 4096, 5000], 32, 1, 16, kv,
              seed=9).device().run()
    b.verify(f"{kv} rounds")


@pytest.mark.parametrize("kv", KV)
def test_scales_per_head(kv):
    if kv == "bf16":
        pytest.skip("one-byte caches only")
    Batch(trees(2, [9, 33]), [200, 31], 4, 2, 16, kv, seed=2, head_scales=True).device().run().verify(f"{kv} head scales")


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("G,past", [(4, 100), (8, 3000), (4, 0)])
def test_what_a_token_does_not_see_does_not_reach_it(kv, G, past):
    """Infinities and NaN in keys and values of tokens on one branch: the other branches' rows are as without them, the rows
    that see them show them."""
    n = 40
    parents = [-1] + [0 if i < 3 else (i - 2) for i in range(1, n)]  # two chains from token 0: odd and even tokens
    runs = [ancestors(parents), ancestors(parents)]
    b = Batch(runs, [past, past + 37], 2, G, 16, kv, seed=G)
    odd = [(5, "nan"), (9, "inf"), (21, "nan")]  # of odd tokens
    for s in range(2):
        for j, what in odd:
            blk, off = b.place(s, b.lens[s] - n + j)
            if kv == "fp8":
                b.k.view(torch.uint8)[blk, off] = 0x7f
                b.v.view(torch.uint8)[blk, off, :, 3::7] = 0xff
            else:
                b.k[blk, off] = float("nan")
                b.v[blk, off, :, 3::7] = float(what)
    b.device().run()
    torch.cuda.synchronize()
    for s in range(2):
        a, L = b.cu[s], b.lens[s]
        even = [i for i in range(n) if i % 2 == 0 or i < 5]
        k, v = gather(b.k, b.tables[s], L), gather(b.v, b.tables[s], L)
        ref, bound = attend_masked(b.q[a:a + n], k, v, seen_keys(n, L, runs[s]), b.scale, kv, b.ks, b.vs)
        check(b.out[a:a + n][even], ref[even], bound[even], f"{kv} unseen, sequence {s}")
        rows = [i for i in range(n) if i % 2 == 1 and i >= 5]
        assert torch.isnan(b.out[a:a + n][rows].float()).all(), "a NaN key reaches every row that sees it"


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("past", [20, 9000])
def test_values_that_are_no_numbers_reach_the_rows_that_see_them(kv, past):
    """Finite keys, values infinite in one head dim of token 2, no numbers in another of token 7 (a chain)."""
    n = 12
    b = Batch([n], [past], 1, 8, 16, kv, seed=past)
    for j, dim, val in ((2, 5, float("-inf")), (7, 90, float("nan"))):
        blk, off = b.place(0, past + j)
        if kv == "fp8":
            b.v.view(torch.uint8)[blk, off, :, dim] = 0xff
        else:
            b.v[blk, off, :, dim] = val
    b.device().run()
    torch.cuda.synchronize()
    k, v = gather(b.k, b.tables[0], b.lens[0]), gather(b.v, b.tables[0], b.lens[0])
    ref, bound = attend_masked(b.q, k, v, seen_keys(n, b.lens[0], None), b.scale, kv, b.ks, b.vs)
    got = b.out.cpu().float()
    hit = torch.zeros(n, 8, D, dtype=torch.bool)
    hit[2:, :, 5] = True
    hit[7:, :, 90] = True
    check(torch.where(hit, torch.zeros_like(got), got), torch.where(hit, torch.zeros_like(ref), ref), bound, f"{kv} other dims")
    if kv == "bf16":
        assert (got[2:, :, 5] == float("-inf")).all() and torch.isnan(got[7:, :, 90]).all()
    else:
        assert torch.isnan(got[hit]).all()


@pytest.mark.parametrize("kv", KV)
def test_finished_sequences_and_malformed_ones(kv):
    """Length 0: zero rows and no error.  A length below the run, past the table, a bad block: flagged, the rest is right."""
    b = Batch(trees(4, [4, 6, 5, 3, 2]), [90, 10, 70, 33, 200], 2, 4, 16, kv, seed=4).device()
    b.dl[1] = 0
    b.run().verify(f"{kv} finished", skip=(1,))
    assert int(b.err) == 0 and (b.out[b.cu[1]:b.cu[2]] == 0).all()
    b.dl[1] = b.lens[1]
    b.dl[2] = 4  # a run of 5
    b.dl[3] = b.tables.shape[1] * 16 + 1
    b.out.fill_(7.0)
    b.run().verify(f"{kv} malformed", skip=(2, 3))
    assert int(b.err) == B.DEVERR_BAD_LENGTH
    assert (b.out[b.cu[2]:b.cu[4]] == 7).all()
    b.err.zero_()
    b.dl.copy_(torch.tensor(b.lens, dtype=torch.int32))
    b.dt[0, 2] = b.dk.shape[0]
    b.run().verify(f"{kv} bad block", skip=(0,))
    assert int(b.err) == B.DEVERR_BAD_BLOCK


def test_a_run_longer_than_its_mask():
    b = Batch(trees(6, [70, 20]), [30, 40], 1, 4, 16, "bf16", seed=6).device()
    b.dm = b.dm[:, :1].contiguous()
    b.run().verify("narrow mask", skip=(0,))
    assert int(b.err) == B.DEVERR_BAD_LENGTH and (b.out[:70] == 7).all()


@pytest.mark.parametrize("kv", KV)
def test_the_same_as_a_prefill_chunk(kv):
    """A chain is what a causal chunk computes (other order of sums): both within their bounds of each other."""
    b = Batch([33, 5], [500, 77], 2, 4, 16, kv, seed=8).device().run()
    other = torch.zeros_like(b.out)
    starts = torch.tensor([500, 77], dtype=torch.int32, device="cuda")
    pkv.pkv_paged_prefill_varlen(other, b.dq, b.dcu, starts, b.dl, b.dk, b.dv, b.desc, b.dt, b.scale)
    torch.cuda.synchronize()
    for s in range(2):
        a, e, L = b.cu[s], b.cu[s + 1], b.lens[s]
        k, v = gather(b.k, b.tables[s], L), gather(b.v, b.tables[s], L)
        _, bound = attend_masked(b.q[a:e], k, v, seen_keys(e - a, L, None), b.scale, kv, b.ks, b.vs)
        assert ((b.out[a:e].double().cpu() - other[a:e].double().cpu()).abs() <= 2 * bound).all()


def test_repeated_calls_streams_and_graphs():
    """The same bits in every call, on another stream, and from a captured graph whose inputs change."""
    b = Batch(trees(10, [16, 40, 8, 1]), [600, 30, 2000, 64], 2, 4, 16, "fp8", seed=10).device().run()
    first = b.out.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.out.fill_(7.0)
    torch.cuda.synchronize()
    b.run(stream=s)
    s.synchronize()
    assert torch.equal(b.out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    b.out.fill_(7.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, first)
    b.q = b.q.flip(0).contiguous()
    b.dq.copy_(b.q)
    g.replay()
    b.verify("replayed with other queries")


@pytest.mark.parametrize("masked", [True, False])
def test_no_tokens_at_all(masked):
    """A step in which no sequence drafts: nothing is written, nothing refused."""
    b = Batch([[], []] if masked else [0, 0], [40, 3], 2, 4, 16, "bf16", seed=15).device()
    assert b.dq.shape[0] == 0 and (b.dm is not None) == masked
    b.run()
    torch.cuda.synchronize()
    assert int(b.err) == 0


def test_two_calls_at_once():
    """Other batches, caches and sizes on two streams, each with its own workspace; masks as uint64."""
    a = Batch(trees(11, [16, 40, 8, 1]), [600, 30, 2000, 64], 2, 4, 16, "bf16", seed=11).device()
    b = Batch(trees(12, [3] * 40), [900] * 40, 1, 8, 8, "int8", seed=12).device()
    a.dm = a.dm.view(torch.uint64)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.run(stream=s)
        b.run(stream=t)
    a.verify("first stream")
    b.verify("second stream")
    assert int(a.err) == 0 and int(b.err) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_queries_and_values_that_are_no_numbers_in_pairs_of_tiles(kv):
    """Runs of more than 128 rows: both groups of a tile pair meet the same values; a NaN query stays in its row."""
    n = 60
    b = Batch([[1 << i for i in range(n)], [1 << i for i in range(n)]], [64, 500], 1, 4, 16, kv, seed=13)
    for s in range(2):
        blk, off = b.place(s, b.lens[s] - n + 17)
        if kv == "fp8":
            b.v.view(torch.uint8)[blk, off] = 0x7f
        else:
            b.v[blk, off] = float("inf")
    if kv == "bf16":
        b.q[3] = float("nan")
    b.device().run()
    torch.cuda.synchronize()
    for s in range(2):
        a, L = b.cu[s], b.lens[s]
        rest = [i for i in range(n) if i != 17 and a + i != 3]
        k, v = gather(b.k, b.tables[s], L), gather(b.v, b.tables[s], L)
        q = b.q[a:a + n].nan_to_num(0.0)
        ref, bound = attend_masked(q, k, v, seen_keys(n, L, b.runs[s]), b.scale, kv, b.ks, b.vs)
        check(b.out[a:a + n][rest], ref[rest], bound[rest], f"{kv}, sequence {s}")
        got = b.out[a + 17].float()
        assert torch.isnan(got).all() if kv == "fp8" else (got == float("inf")).all()
    if kv == "bf16":
        assert torch.isnan(b.out[3].float()).all()


def test_far_tables_and_pools():
    """Blocks whose elements lie past 2^31."""
    b = Batch(trees(14, [8, 5]), [300, 40], 8, 4, 32, "bf16", seed=14).device()
    nb = (1 << 31) // (32 * 8 * 128) + 200
    big_k = torch.zeros(nb, 32, 8, 128, dtype=torch.bfloat16, device="cuda")
    big_v = torch.zeros_like(big_k)
    shift = nb - b.dk.shape[0]
    big_k[shift:], big_v[shift:] = b.dk, b.dv
    b.dk, b.dv, b.dt = big_k, big_v, torch.where(b.dt >= 0, b.dt + shift, b.dt)
    b.desc = pkv.CacheDesc.for_cache(b.dk)
    b.run().verify("far")


def test_many_sequences():
    """2048 runs of none to three tokens."""
    r = random.Random(3)
    sizes = [r.randrange(4) for _ in range(2048)]
    b = Batch(trees(3, sizes), [r.randrange(40) for _ in sizes], 1, 8, 8, "bf16", seed=3).device().run()
    torch.cuda.synchronize()
    assert int(b.err) == 0
    b.verify("many", skip=[s for s in range(2048) if s % 16])
