"""A speculative decoding step as a program runs it, replayed from one captured graph: step planning for the drafted tokens,
rotary append and tree attention in every layer, commit of the accepted paths, surplus blocks handed back.  Every step is
checked: attention in 64 bits over what the caches should hold, the caches after the commit bit for bit, tables and blocks."""
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv

from attention_ref import DTYPE, SCALE, check, gather
from tree_ref import attend_masked, random_tree, seen_keys

pytestmark = pytest.mark.gpu
D, S, HKV, G, LAYERS, NB = 128, 16, 2, 4, 2, 96
HQ = HKV * G
SIZES = [8, 1, 17, 40, 0, 5]       # drafted tokens of each row (0: an idle row)
START = [30, 0, 7, 64, 0, 300]     # tokens that the rows hold before the first step
T, MAX_TOKENS = sum(SIZES), 80


class Step:
    def __init__(self, kv):
        self.kv, self.n = kv, len(SIZES)
        self.gen, self.r = torch.Generator().manual_seed(5), random.Random(5)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.tables = torch.full((self.n, 32), -1, **i32)
        self.free = torch.randperm(NB, generator=self.gen).to(torch.int32).cuda()
        self.count = torch.tensor([NB], **i32)
        self.past = torch.zeros(self.n, **i32)
        self.new = torch.tensor(START, **i32)
        self.lens, self.starts, self.cu = torch.zeros(self.n, **i32), torch.zeros(self.n, **i32), torch.zeros(self.n + 1, **i32)
        self.scratch, self.err = torch.zeros(self.n, **i32), torch.zeros(1, **i32)
        self.k = [torch.zeros(NB, S, HKV, D, device="cuda").to(DTYPE[kv]) for _ in range(LAYERS)]
        self.v = [torch.zeros_like(c) for c in self.k]
        self.desc = pkv.CacheDesc.for_cache(self.k[0], SCALE[kv], SCALE[kv])
        self.layers = pkv.LayerCaches(self.k, self.v)
        inv, self.factor = pkv.rotary_frequencies(96, 10000.0, "yarn", 4.0, 64)
        self.inv = torch.from_numpy(inv).cuda()
        self.scale = 1 / np.sqrt(D)
        self.qkv = torch.zeros(LAYERS, T, HQ + 2 * HKV, D, dtype=torch.bfloat16, device="cuda")
        self.q = torch.zeros(LAYERS, MAX_TOKENS, HQ, D, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.slots = torch.zeros(MAX_TOKENS, dtype=torch.int64, device="cuda")
        self.row_of = torch.tensor([s for s, n in enumerate(SIZES) for _ in range(n)], device="cuda")
        self.depth, self.positions = torch.zeros(T, **i32), torch.zeros(T, **i32)
        self.mask = torch.zeros(MAX_TOKENS, 1, dtype=torch.int64, device="cuda")
        self.parents, self.draft, self.target, self.accepted = (torch.zeros(MAX_TOKENS, **i32) for _ in range(4))
        self.m, self.next, self.keep = (torch.zeros(self.n, **i32) for _ in range(3))
        self.all = torch.ones(self.n, dtype=torch.bool, device="cuda")
        need = pkv.pkv_paged_attention_tree_workspace_size(self.desc, MAX_TOKENS, self.n, HQ)
        self.ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
        # the tokens that are there: values as a prompt would leave them
        self.hist = [[[] for _ in range(self.n)] for _ in range(LAYERS)]
        slots = torch.zeros(sum(START), dtype=torch.int64, device="cuda")
        pkv.pkv_extend_sequences(self.tables, self.past, self.new, S, self.free, self.count, self.past, self.count, slots,
                                 device_error=self.err)
        for l in range(LAYERS):
            x = torch.randn(2, sum(START), HKV, D, generator=self.gen).to(torch.bfloat16).cuda()
            pkv.pkv_reshape_and_cache(x[0], x[1], slots, self.k[l], self.v[l], self.desc, self.err)
            for s in range(self.n):
                self.hist[l][s] = [gather(c.cpu(), self.tables[s].cpu(), START[s]) for c in (self.k[l], self.v[l])]
        self.new.copy_(torch.tensor(SIZES))

    def program(self):
        pkv.pkv_extend_sequences(self.tables, self.past, self.new, S, self.free, self.count, self.lens, self.count, self.slots,
                                 self.cu, self.starts, self.err)
        torch.add(self.starts[self.row_of], self.depth, out=self.positions)
        for l in range(LAYERS):
            x = self.qkv[l]
            pkv.pkv_rope_and_cache(self.q[l, :T], x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.positions, self.slots[:T],
                                   self.inv, self.k[l], self.v[l], self.desc, True, self.factor, self.err)
            pkv.pkv_paged_attention_tree(self.out[l], self.q[l], self.cu, self.lens, self.mask, self.k[l], self.v[l], self.desc,
                                         self.tables, self.scale, self.ws, self.err)
        pkv.pkv_commit_tree(self.layers, self.tables, self.cu, self.starts, self.parents, self.draft, self.target, self.accepted,
                            self.m, self.past, self.next, self.keep, self.err)
        pkv.pkv_release_sequences(self.tables, self.lens, self.all, S, self.free, self.count, self.scratch, self.count, self.keep,
                                  self.err)

    def inputs(self):
        """New trees, projections and choices of the model."""
        self.trees = [random_tree(self.r, n) for n in SIZES]
        self.bits, depth, words, parents = [], [], [], []
        for t in self.trees:
            masks, d = pkv.draft_tree_masks(t)
            self.bits.append([int(x) for x in masks[:, 0]])
            depth += d.tolist()
            words += masks[:, 0].tolist()
            parents += t
        self.depth.copy_(torch.tensor(depth))
        self.mask[:T, 0] = torch.tensor(words, dtype=torch.int64)
        self.parents[:T] = torch.tensor(parents, dtype=torch.int32)
        draft = [self.r.randrange(1000) for _ in range(T)]
        target, a, self.paths = [2000] * T, 0, []
        for t in self.trees:
            path = [0] if t else []
            while path:
                kids = [i for i, p in enumerate(t) if p == path[-1] and i > path[-1]]
                if not kids or self.r.random() < 0.2:
                    break
                kid = self.r.choice(kids)
                target[a + path[-1]] = draft[a + kid]
                kid = next(i for i in kids if draft[a + i] == draft[a + kid])
                path.append(kid)
            self.paths.append(path)
            a += len(t)
        self.draft[:T], self.target[:T] = torch.tensor(draft, dtype=torch.int32), torch.tensor(target, dtype=torch.int32)
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=self.gen))
        self.out.fill_(7.0)

    def check(self, before, what):
        torch.cuda.synchronize()
        assert int(self.err) == 0
        cu = np.concatenate([[0], np.cumsum(SIZES)]).tolist()
        assert self.cu.tolist() == cu and self.starts.tolist() == before
        assert self.past.tolist() == [b + len(p) for b, p in zip(before, self.paths)]
        assert self.next.tolist() == [2000 if p else -1 for p in self.paths]
        tables = self.tables.cpu()
        live = [b for s, L in enumerate(self.past.tolist()) for b in tables[s, :-(-L // S)].tolist()]
        free = self.free[: int(self.count)].tolist()
        assert sorted(live + free) == list(range(NB)), f"{what}: every block is a sequence's or free"
        for l in range(LAYERS):
            # this step's keys and values as the caches get them, from the same call into a pool of their own
            k1 = torch.zeros(-(-T // S), S, HKV, D, device="cuda").to(DTYPE[self.kv])
            v1, q1 = torch.zeros_like(k1), torch.zeros(T, HQ, D, dtype=torch.bfloat16, device="cuda")
            x = self.qkv[l]
            d1 = pkv.CacheDesc.for_cache(k1, SCALE[self.kv], SCALE[self.kv])
            pkv.pkv_rope_and_cache(q1, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.positions, torch.arange(T, device="cuda"),
                                   self.inv, k1, v1, d1, True, self.factor)
            assert torch.equal(q1, self.q[l, :T])
            step = [gather(c.cpu(), torch.arange(len(c)), T) for c in (k1, v1)]
            for s, n in enumerate(SIZES):
                a, path = cu[s], self.paths[s]
                k, v = (torch.cat([h, c[a:a + n]]) for h, c in zip(self.hist[l][s], step))
                if n:
                    ref, bound = attend_masked(q1[a:a + n].cpu(), k, v, seen_keys(n, before[s] + n, self.bits[s]), self.scale, self.kv,
                                               SCALE[self.kv], SCALE[self.kv])
                    check(self.out[l, a:a + n], ref, bound, f"{what}, layer {l}, row {s}")
                self.hist[l][s] = [torch.cat([h, c[[a + i for i in path]]]) for h, c in zip(self.hist[l][s], step)]
                for c, h in zip((self.k[l], self.v[l]), self.hist[l][s]):
                    assert torch.equal(gather(c.cpu(), tables[s], len(h)), h), f"{what}: cache of layer {l}, row {s}"
            assert (self.out[l, T:] == 7).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_steps_from_one_graph(kv):
    st = Step(kv)
    before = st.past.tolist()
    st.inputs()
    st.program()
    st.check(before, "first step")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.program()
    for step in range(5):
        before = st.past.tolist()
        st.inputs()
        graph.replay()
        st.check(before, f"replay {step}")
