"""Commit of accepted drafts (pkv_commit_tree) against a plain walk and moves one after another: equal bit for bit."""
import random

import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B

from tree_ref import random_tree

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


class Batch:
    def __init__(self, trees, past, seed, layers=3, S=16, Hkv=2, D=128, kv="bf16", go_on=0.8, lead=0, tail=0, ids=50):
        """trees: parents of each run; target ids follow a child's draft with probability go_on."""
        r, g = random.Random(seed), torch.Generator().manual_seed(seed)
        self.S, self.past, self.n = S, list(past), len(trees)
        self.sizes = [len(t) for t in trees]
        self.cu = [lead]
        for n in self.sizes:
            self.cu.append(self.cu[-1] + n)
        T = self.cu[-1] + tail
        self.parents, self.draft, self.target = [7] * T, [r.randrange(ids) for _ in range(T)], [r.randrange(ids) for _ in range(T)]
        for a, t in zip(self.cu, trees):
            for i, p in enumerate(t):
                self.parents[a + i] = p
            for i in range(len(t)):
                kids = [j for j, p in enumerate(t) if p == i and j > i]
                if kids and r.random() < go_on:
                    self.target[a + i] = self.draft[a + r.choice(kids)]
        blocks = [-(-(p + n) // S) for p, n in zip(self.past, self.sizes)]
        nb = sum(blocks) + 2
        perm, at = torch.randperm(nb, generator=g).to(torch.int32), 0
        self.tables = torch.full((self.n, max(1, max(blocks))), -1, dtype=torch.int32)
        for s, b in enumerate(blocks):
            self.tables[s, :b] = perm[at:at + b]
            at += b
        raw = (nb, S, Hkv, D * torch.empty(0, dtype=TYPES[kv]).element_size())
        self.caches = [[torch.randint(0, 256, raw, generator=g, dtype=torch.uint8).view(TYPES[kv]) for _ in range(layers)] for _ in "kv"]

    def device(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.dev = [[c.cuda() for c in cs] for cs in self.caches]
        self.layers = pkv.LayerCaches(*self.dev)
        self.dt, self.dcu, self.dpast = self.tables.cuda(), torch.tensor(self.cu, **i32), torch.tensor(self.past, **i32)
        self.ids = [torch.tensor(x, **i32) for x in (self.parents, self.draft, self.target)]
        self.accepted = torch.full((len(self.parents),), 99, **i32)
        self.outs = [torch.full((self.n,), 99, **i32) for _ in range(4)]  # count, lengths, next, blocks to keep
        self.err = torch.zeros(1, **i32)
        return self

    def run(self, stream=None):
        pkv.pkv_commit_tree(self.layers, self.dt, self.dcu, self.dpast, *self.ids, self.accepted, *self.outs, self.err, stream)
        return self

    def expected(self, skip=()):
        accepted = [99] * len(self.parents)
        outs = [[], [], [], []]
        caches = [[c.view(torch.uint8).clone() for c in cs] for cs in self.caches]
        S = self.S
        for s, (a, n, past) in enumerate(zip(self.cu, self.sizes, self.past)):
            if s in skip or n == 0:
                accepted[a:a + n] = [-1] * n
                for o, x in zip(outs, (0, past, -1, max(0, -(-past // S)))):
                    o.append(x)
                continue
            path = [0]
            while True:
                fits = [i for i in range(path[-1] + 1, n) if self.parents[a + i] == path[-1]
                        and self.draft[a + i] == self.target[a + path[-1]]]
                if not fits:
                    break
                path.append(fits[0])
            accepted[a:a + n] = path + [-1] * (n - len(path))
            m = len(path)
            for o, x in zip(outs, (m, past + m, self.target[a + path[-1]], -(-(past + m) // S))):
                o.append(x)
            for j, i in enumerate(path):
                sb, db = int(self.tables[s, (past + i) // S]), int(self.tables[s, (past + j) // S])
                for cs in caches:
                    for c in cs:
                        c[db, (past + j) % S] = c[sb, (past + i) % S].clone()
        return accepted, outs, caches

    def verify(self, what, skip=()):
        torch.cuda.synchronize()
        accepted, outs, caches = self.expected(skip)
        assert self.accepted.tolist() == accepted, what
        for name, got, want in zip(("accepted tokens", "lengths", "next tokens", "blocks to keep"), self.outs, outs):
            assert got.tolist() == want, f"{what}: {name}"
        for got, want in zip(self.dev, caches):
            for l, (x, y) in enumerate(zip(got, want)):
                assert torch.equal(x.view(torch.uint8).cpu(), y), f"{what}: caches of layer {l}"
        return self


def trees(seed, sizes):
    r = random.Random(seed)
    return [random_tree(r, n) for n in sizes]


@pytest.mark.parametrize("kv", ["f32", "bf16", "fp8", "int8"])
@pytest.mark.parametrize("S", [4, 8, 16, 32])
def test_ragged_trees(kv, S):
    b = Batch(trees(S, [1, 8, 0, 64, 65, 3, 130, 33, 16]), [0, 5, 7, 31, 0, 100, 64, 15, 1], S, S=S, kv=kv, lead=2, tail=3).device()
    b.run().verify(f"{kv} S={S}")
    assert int(b.err) == 0


@pytest.mark.parametrize("D,Hkv", [(64, 1), (64, 5), (128, 1), (128, 32)])
def test_head_layouts(D, Hkv):
    Batch(trees(D, [20, 40]), [3, 90], Hkv, D=D, Hkv=Hkv, kv="fp8").device().run().verify(f"{Hkv} heads of {D}")


def test_moves_that_chain():
    """Every second token of a long chain: what one move leaves the next takes, over several batches of moves."""
    n = 200
    parents = [-1] + [max(0, i - 2) if i % 2 == 0 else 0 for i in range(1, n)]
    b = Batch([parents, parents[:37]], [13, 0], 1, ids=1, layers=2).device()
    b.run()
    _, outs, _ = b.expected()
    assert outs[0][0] > 1
    b.verify("ids all alike: the lowest child")
    b = Batch([parents], [13], 2, layers=2, ids=100000)
    for i in range(0, n - 2, 2):
        b.target[i] = b.draft[i + 2]
    b.device().run().verify("every second token")
    assert int(b.outs[0][0]) >= 99


def test_skipped_tokens_anywhere():
    """Chains of increasing gaps: tokens 0, 1, 3, 6, 10, ... of runs of up to 1024."""
    for n in (1024, 300, 12):
        picks = [i * (i + 1) // 2 for i in range(60) if i * (i + 1) // 2 < n]
        parents = [-1] * n
        for a, c in zip(picks, picks[1:]):
            parents[c] = a
        b = Batch([parents], [9], n, layers=2, ids=10 ** 6)
        for a, c in zip(picks, picks[1:]):
            b.target[a] = b.draft[c]
        b.device().run().verify(f"{n} tokens")
        assert int(b.outs[0][0]) == len(picks)


def test_chains_are_left_where_they_are():
    b = Batch([list(range(-1, 19))] * 3, [4, 30, 0], 3, go_on=1.0).device()
    b.run().verify("chains")
    for got, was in zip(b.dev, b.caches):
        for x, y in zip(got, was):
            assert torch.equal(x.view(torch.uint8).cpu(), y.view(torch.uint8))


def test_parents_that_are_no_tree():
    """Parents at or behind the token, below -1 or beyond the run are never followed."""
    odd = [0, 1, 5, 2, 99, -7, 3, 2 ** 31 - 1, -2 ** 31, 0]
    Batch([odd, [-1, 0, 0]], [6, 6], 4, ids=1).device().run().verify("no tree")


@pytest.mark.parametrize("n,layers", [(1, 128), (300, 5), (2000, 1)])
def test_many_sequences_and_layers(n, layers):
    r = random.Random(n)
    b = Batch(trees(n, [r.randrange(20) for _ in range(n)]), [r.randrange(30) for _ in range(n)], n, layers=layers, S=8, Hkv=1, D=64)
    b.device().run().verify(f"{n} sequences, {layers} layers")


def test_malformed_sequences():
    b = Batch(trees(5, [6, 9, 4, 7]), [10, 20, 30, 40], 5, lead=1).device()
    b.dpast[1] = -1
    b.past[1] = -1
    b.dpast[2] = b.past[2] = b.tables.shape[1] * 16 - 3
    b.run()
    b.verify("malformed", skip=(1, 2))
    assert int(b.err) == B.DEVERR_BAD_LENGTH
    b = Batch(trees(6, [6, 9]), [10, 20], 6).device()
    b.dcu[1] = 900
    b.run()
    torch.cuda.synchronize()
    assert int(b.err) == B.DEVERR_BAD_LENGTH and b.outs[0].tolist() == [0, 0] and (b.accepted == 99).all()
    b = Batch([[-1] + [0] * 1024, [-1, 0]], [0, 3], 7, layers=1).device()  # 1025 tokens
    b.run().verify("too long", skip=(0,))
    assert int(b.err) == B.DEVERR_BAD_LENGTH


def test_bad_blocks():
    """A move whose place lies outside the pool is left out, the others happen."""
    b = Batch([[-1, 0, 0, 0, 3, 3, 3]], [14], 8, layers=2, go_on=0.0, ids=10 ** 6)
    b.target[0], b.target[3] = b.draft[3], b.draft[6]  # path 0, 3, 6: 17 -> 15, 20 -> 16
    b.device()
    for bad in (-1, b.dev[0][0].shape[0]):
        b.dt[0, 1] = bad  # tokens from position 16 on
        b.run()
        torch.cuda.synchronize()
        assert int(b.err) == B.DEVERR_BAD_BLOCK and b.accepted.tolist()[:3] == [0, 3, 6]
        for got, was in zip(b.dev, b.caches):
            for x, y in zip(got, was):
                assert torch.equal(x.view(torch.uint8).cpu(), y.view(torch.uint8))
        b.err.zero_()


def test_no_tokens_at_all():
    b = Batch([[], [], []], [0, 16, 37], 10).device()
    b.run().verify("no runs")
    assert int(b.err) == 0


def test_without_blocks_to_keep_on_a_stream_and_from_a_graph():
    b = Batch(trees(9, [12, 30]), [5, 17], 9).device()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pkv.pkv_commit_tree(b.layers, b.dt, b.dcu, b.dpast, *b.ids, b.accepted, *b.outs[:3], None, b.err, s)
    s.synchronize()
    assert (b.outs[3] == 99).all()
    b = Batch(trees(9, [12, 30]), [5, 17], 9).device()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.run()
    for got, was in zip(b.dev, b.caches):  # (a capture runs nothing)
        for x, y in zip(got, was):
            assert torch.equal(x.view(torch.uint8).cpu(), y.view(torch.uint8))
    g.replay()
    b.verify("replayed")


def test_pools_past_two_to_the_31_bytes():
    """Slots whose byte offset passes 32 bits."""
    nb, S, Hkv, D = 70000, 32, 8, 128
    k = torch.zeros(nb, S, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[nb - 1, 5], v[nb - 1, 5] = 3.0, 4.0
    i32 = dict(dtype=torch.int32, device="cuda")
    outs = [torch.zeros(1, **i32) for _ in range(4)]
    acc = torch.zeros(6, **i32)
    t = lambda *x: torch.tensor(x, **i32)
    pkv.pkv_commit_tree(pkv.LayerCaches([k], [v]), t(nb - 1).reshape(1, 1), t(0, 6), t(0), t(-1, 0, 0, 0, 0, 0), t(0, 1, 2, 3, 4, 5),
                        t(5, 9, 9, 9, 9, 9), acc, *outs)
    assert acc.tolist() == [0, 5, -1, -1, -1, -1] and (k[nb - 1, 1] == 3).all() and (v[nb - 1, 1] == 4).all()
