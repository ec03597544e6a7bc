"""The INT8 attention stream (cross attention, draft trees, shared prefixes) where every key tile shows in the output, exactly.

Queries are ones, a key's codes all 0 or all -127: its score is 0 or -127 * 128 / 32 = -508, its weight 1 or exp(-508) = 0 in fp32.
With 1024 keys of weight 1 per KV head the output is the sum of their codes over 1024 * 32: whole numbers below 2^24 and a
power of two, so its only rounding is the last one, to bf16, and a key tile whose codes were read before they had landed,
or written over before they were used, changes it.  Caches are new in every call, so that what an earlier one left is wrong.
"""
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv

pytestmark = pytest.mark.gpu
D, S, CHOSEN = 128, 16, 1024


class Keys:
    """Per sequence a range of `lens` keys, the last of which (own[s]) are never chosen."""

    def __init__(self, lens, own, Hkv, seed):
        self.gen = torch.Generator("cuda").manual_seed(seed)
        self.lens, self.own, self.Hkv = lens, own, Hkv
        nb, at = sum(-(-L // S) for L in lens) + 1, 0
        perm = torch.randperm(nb, generator=self.gen, device="cuda").to(torch.int32)
        self.tables = torch.full((len(lens), max(-(-L // S) for L in lens)), -1, dtype=torch.int32, device="cuda")
        for s, L in enumerate(lens):
            self.tables[s, :-(-L // S)] = perm[at:at - (-L // S)]
            at += -(-L // S)
        self.k = torch.zeros(nb, S, Hkv, D, dtype=torch.int8, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.desc = pkv.CacheDesc.for_cache(self.k, 1 / 32, 1 / 32)

    def fill(self):
        """New codes; returns what every row of each sequence is, [sequences][Hkv][D] bf16."""
        self.v.random_(-127, 128, generator=self.gen)
        self.k.fill_(-127)
        ref = []
        for s, L in enumerate(self.lens):
            n = L - self.own[s]
            rank = torch.rand(self.Hkv, n, generator=self.gen, device="cuda").argsort(1)[:, :CHOSEN]  # chosen keys of each head
            block, off = self.tables[s, rank // S].long(), rank % S
            heads = torch.arange(self.Hkv, device="cuda")[:, None]
            self.k[block, off, heads] = 0
            ref.append(self.v[block, off, heads].double().sum(1) / (32 * CHOSEN))
        return torch.stack(ref).to(torch.bfloat16)


def _check(out, ref, G, what):
    """out: the rows of one sequence, [tokens][Hq][D]; ref [Hkv][D]"""
    assert torch.equal(out, ref.repeat_interleave(G, 0).expand_as(out)), what


@pytest.mark.parametrize("tokens", [[3, 1, 5, 2], [100, 7, 64, 40]])
def test_cross_attention(tokens):
    Hkv, G = 4, 4
    c = Keys([3001, 1024, 7777, 2050], [0] * 4, Hkv, seed=len(tokens) + tokens[0])
    cu = torch.tensor([0, *torch.tensor(tokens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    q = torch.ones(int(cu[-1]), Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.pkv_paged_cross_attention_workspace_size(c.desc, q.shape[0], 4, Hkv * G), dtype=torch.uint8, device="cuda")
    for call in range(20):
        ref = c.fill()
        pkv.pkv_paged_cross_attention(out, q, cu, lens, c.k, c.v, c.desc, c.tables, 1.0, ws)
        for s in range(4):
            _check(out[cu[s]:cu[s + 1]], ref[s], G, f"call {call}, sequence {s}")


@pytest.mark.parametrize("tokens", [[3, 1, 5, 2], [100, 7, 64, 40]])
def test_draft_trees(tokens):
    Hkv, G = 4, 4
    c = Keys([3001, 1200, 7777, 2050], tokens, Hkv, seed=tokens[0])
    cu = torch.tensor([0, *torch.tensor(tokens).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    q = torch.ones(int(cu[-1]), Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.pkv_paged_attention_tree_workspace_size(c.desc, q.shape[0], 4, Hkv * G), dtype=torch.uint8, device="cuda")
    for call in range(20):
        ref = c.fill()
        pkv.pkv_paged_attention_tree(out, q, cu, lens, None, c.k, c.v, c.desc, c.tables, 1.0, ws)
        for s in range(4):
            _check(out[cu[s]:cu[s + 1]], ref[s], G, f"call {call}, sequence {s}")


def test_shared_prefixes():
    """Groups of 90 and 3 sequences; their own tokens, in blocks behind the prefix, are never chosen."""
    Hkv, G, sizes, prefix, own = 4, 4, [90, 3], [4000, 1600], 21
    c = Keys([prefix[0] + 32, prefix[1] + 32], [32, 32], Hkv, seed=5)
    rows = torch.cat([c.tables[g:g + 1].expand(n, -1) for g, n in enumerate(sizes)]).contiguous()
    lens = torch.tensor([prefix[0] + own] * 90 + [prefix[1] + own] * 3, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 90, 93], dtype=torch.int32, device="cuda")
    pre = torch.tensor(prefix, dtype=torch.int32, device="cuda")
    q = torch.ones(93, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(pkv.pkv_paged_attention_decode_prefix_workspace_size(c.desc, 93, Hkv * G), dtype=torch.uint8, device="cuda")
    for call in range(20):
        ref = c.fill()
        pkv.pkv_paged_attention_decode_prefix(out, q, c.k, c.v, c.desc, rows, lens, cu, pre, 1.0, ws)
        _check(out[:90], ref[0], G, f"call {call}, group 0")
        _check(out[90:], ref[1], G, f"call {call}, group 1")
