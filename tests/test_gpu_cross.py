"""Cross attention over paged encoder states (pkv_paged_cross_attention) against attention in 64 bits; bounds in
attention_ref.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B
from paged_kv_cache_71_gb300 import workload as wl

from attention_ref import SCALE, attend, check, gather, make_cache
from parity import TOL

pytestmark = pytest.mark.gpu
D = 128


class Batch:
    """tokens, states: per sequence; lead, tail: query rows before and behind that no sequence owns."""

    def __init__(self, tokens, states, Hkv, G, S, kv, seed, lead=0, tail=0, head_scales=False):
        gen = torch.Generator().manual_seed(seed)
        self.kv, self.S, self.Hq, self.n = kv, S, Hkv * G, len(tokens)
        self.cu = (lead + np.concatenate([[0], np.cumsum(tokens)])).tolist()
        self.lens = list(states)
        nb = sum(-(-L // S) for L in states) + 2
        perm, at = torch.randperm(nb, generator=gen).to(torch.int32), 0
        self.tables = torch.full((self.n, max(1, max(-(-L // S) for L in states))), -1, dtype=torch.int32)
        self.k, self.v = make_cache(gen, (nb, S, Hkv, D), kv), make_cache(gen, (nb, S, Hkv, D), kv)
        used = torch.zeros(nb, S, dtype=torch.bool)
        for s, L in enumerate(states):
            b = -(-L // S)
            self.tables[s, :b] = perm[at:at + b]
            at += b
            for pos in range(L):
                used[int(self.tables[s, pos // S]), pos % S] = True
        if kv != "int8":  # slots without a token are not numbers
            for c in (self.k, self.v):
                c.view(torch.uint8 if kv == "fp8" else torch.int16)[~used] = 0x7f if kv == "fp8" else 0x7fc0
        self.q = torch.randn(self.cu[-1] + tail, self.Hq, D, generator=gen).to(torch.bfloat16)
        self.q[:lead] = self.q[self.cu[-1]:] = float("nan")
        self.scale = 1 / np.sqrt(D)
        self.ks = self.vs = SCALE[kv]
        if head_scales:
            self.ks = (torch.rand(Hkv, generator=gen) + 0.5) * SCALE[kv]
            self.vs = (torch.rand(Hkv, generator=gen) + 0.5) * SCALE[kv]

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
        self.out = torch.full_like(self.dq, 7.0)
        need = pkv.pkv_paged_cross_attention_workspace_size(self.desc, self.q.shape[0], self.n, self.Hq)
        self.ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
        self.err = torch.zeros(1, **i32)
        return self

    def run(self, single=False, stream=None):
        pkv.pkv_paged_cross_attention(self.out, self.dq, None if single else self.dcu, self.dl, self.dk, self.dv,
                                      self.desc, self.dt, self.scale, self.ws, self.err, stream)
        return self.out

    def verify(self, what, skip=(), tile=True):
        torch.cuda.synchronize()
        for s in range(self.n):
            if s in skip:
                continue
            a, b = self.cu[s], self.cu[s + 1]
            k, v = gather(self.k, self.tables[s], self.lens[s]), gather(self.v, self.tables[s], self.lens[s])
            ref, bound = attend(self.q[a:b], k, v, self.scale, self.kv, self.ks, self.vs, tile)
            check(self.out[a:b], ref, bound, f"{what}, sequence {s}")


TOKENS = [1, 5, 0, 64, 130, 1, 3, 2]
STATES = [1, 63, 40, 64, 65, 0, 700, 1025]


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_ragged_tokens_and_states(kv, G):
    """Query runs of none to several tiles, states of none to 1025 positions; rows that no sequence owns stay."""
    b = Batch(TOKENS, STATES, 2, G, 16, kv, seed=G, lead=3, tail=2).device()
    b.run()
    b.verify(f"{kv} G={G}")
    assert int(b.err) == 0
    assert (b.out[:3] == 7).all() and (b.out[-2:] == 7).all()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("S", [8, 32])
def test_block_sizes_and_an_odd_head_count(kv, S):
    b = Batch([7, 40], [33, 500], 3, 4, S, kv, seed=S).device()
    b.run()
    b.verify(f"{kv} S={S}")
    assert int(b.err) == 0


@pytest.mark.parametrize("G", [16, 128])
def test_large_head_groups(G):
    b = Batch([3, 1, 9], [100, 64, 333], 1, G, 16, "bf16", seed=G).device()
    b.run()
    b.verify(f"G={G}")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_one_item_over_the_whole_gpu(kv):
    """A few tokens against many states: one item cut into a piece for every SM."""
    b = Batch([3], [9999], 1, 4, 16, kv, seed=1).device()
    b.run()
    b.verify(f"{kv} cut item")
    assert int(b.err) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_items_longer_and_shorter_than_a_share(kv):
    """Many query tiles over different lengths: items that are whole, cut once and cut more than once."""
    b = Batch([600, 40, 300, 1], [900, 2100, 70, 4000], 2, 4, 16, kv, seed=2).device()
    b.run()
    b.verify(f"{kv} shares")
    assert int(b.err) == 0


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_several_long_items_for_every_sm(kv):
    """352 items of 47 to 125 key tiles, one or two query tiles each: whole items in rounds, then a stream of the rest."""
    b = Batch([300, 40, 129, 5, 260, 500, 128, 257], [3000, 4100, 0, 8000, 4500, 3333, 4096, 5000], 32, 1, 16, kv, seed=9).device()
    b.run()
    b.verify(f"{kv} rounds")
    assert int(b.err) == 0


def test_many_sequences_without_states():
    """More of them than an SM lists, and one of many tokens."""
    tokens, states = [1, 2] * 300 + [300, 5], [0] * 601 + [70]
    b = Batch(tokens, states, 2, 4, 16, "bf16", seed=10).device()
    b.run()
    torch.cuda.synchronize()
    assert (b.out[:b.cu[601]] == 0).all() and int(b.err) == 0
    b.verify("many without states", skip=range(601))


@pytest.mark.parametrize("kv", ["fp8", "int8"])
def test_per_head_scales(kv):
    b = Batch(TOKENS, STATES, 2, 4, 16, kv, seed=3, head_scales=True).device()
    b.run()
    b.verify(f"{kv} per-head scales")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("G", [1, 4, 8])
def test_single_tokens(kv, G):
    """One token a sequence (no cu_q): the decode over the states; the run form gives the same up to rounding."""
    b = Batch([1] * 8, STATES, 2, G, 16, kv, seed=G + 20).device()
    b.run(single=True)
    b.verify(f"{kv} single G={G}", tile=False)
    b.run()
    b.verify(f"{kv} runs of one G={G}")
    assert int(b.err) == 0


def test_single_tokens_fp32_and_64_dim_heads():
    """The single-token form has the decode's types: fp32 caches and 64-dim heads."""
    rng = np.random.default_rng(5)
    lens, S, Hkv, G, d = [5, 0, 130], 4, 2, 2, 64
    nb = sum(-(-L // S) for L in lens)
    k, v = (torch.from_numpy(wl.random_values(rng, (nb, S, Hkv, d), "f32")) for _ in range(2))
    q = torch.from_numpy(wl.random_values(rng, (3, Hkv * G, d), "f32"))
    t, at = torch.full((3, 40), -1, dtype=torch.int32), 0
    for s, L in enumerate(lens):
        t[s, : -(-L // S)] = torch.arange(at, at + -(-L // S))
        at += -(-L // S)
    desc = pkv.CacheDesc.for_cache(k)
    out = torch.full_like(q, 7.0).cuda()
    ws = torch.empty(max(16, pkv.pkv_paged_cross_attention_workspace_size(desc, 3, 3, Hkv * G)), dtype=torch.uint8,
                     device="cuda")
    pkv.pkv_paged_cross_attention(out, q.cuda(), None, torch.tensor(lens, dtype=torch.int32, device="cuda"), k.cuda(),
                                  v.cuda(), desc, t.cuda(), 0.125, ws)
    for s, L in enumerate(lens):
        ref, _ = attend(q[s:s + 1], gather(k, t[s], L), gather(v, t[s], L), 0.125, "f32", 1.0, 1.0, False)
        assert (out[s:s + 1].double().cpu() - ref).abs().max() <= TOL["f32"][0]


def test_calls_repeat_bit_for_bit_and_replay_from_a_graph():
    b = Batch([600, 40, 300, 1], [900, 2100, 70, 4000], 2, 4, 16, "bf16", seed=6).device()
    first = b.run().clone()
    b.out.fill_(7.0)
    assert torch.equal(b.run(), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            b.run()
        b.lens[3], b.lens[0] = 1111, 0
        b.dl.copy_(torch.tensor(b.lens, dtype=torch.int32))
        for _ in range(2):
            graph.replay()
        side.synchronize()
    assert int(b.err) == 0
    b.verify("replayed with other lengths")


def test_two_calls_on_two_streams():
    bs = [Batch(TOKENS, STATES, 2, 4, 16, "bf16", seed=30 + i).device() for i in range(2)]
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, st in zip(bs, streams):
            b.run(stream=st)
    for b in bs:
        b.verify("concurrent calls")
        assert int(b.err) == 0


@pytest.mark.parametrize("what", ["length", "negative", "past the rows", "decreasing"])
def test_bad_lengths_are_reported_and_the_other_sequences_hold(what):
    b = Batch([5, 6, 7], [30, 40, 50], 2, 4, 16, "bf16", seed=7).device()
    skip = [1]
    if what == "length":
        b.dl[1] = b.tables.shape[1] * 16 + 1
    elif what == "negative":
        b.dl[1] = -1
    elif what == "past the rows":
        b.dcu[3], skip = 19, [2]
    else:
        b.dcu[1], skip = -1, [0, 1]  # sequence 0 owns less than nothing, sequence 1 starts before the rows
    b.run()
    b.verify(what, skip=skip)
    assert int(b.err) == B.DEVERR_BAD_LENGTH
    a, e = b.cu[skip[0]], b.cu[skip[-1] + 1]
    assert (b.out[a:e] == 7).all()


def test_a_bad_block_is_reported():
    b = Batch([5, 6], [30, 40], 2, 4, 16, "bf16", seed=8).device()
    b.dt[0, 1] = -3
    b.run()
    b.verify("the other sequence", skip=[0])
    assert int(b.err) & B.DEVERR_BAD_BLOCK


def test_a_workspace_or_error_word_in_host_memory_is_refused():
    b = Batch([5, 6], [30, 40], 2, 4, 16, "bf16", seed=11).device()
    for name in ("ws", "err"):
        kept = getattr(b, name)
        setattr(b, name, kept.cpu())
        with pytest.raises(pkv.PkvError, match="workspace" if name == "ws" else "device_error"):
            b.run()
        setattr(b, name, kept)
    b.run()
    b.verify("after the refusals")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_a_workspace_aligned_to_16_bytes_only(kv):
    """Exactly as many bytes as asked for, at 16 bytes past a 512-byte boundary; what lies around stays as it is."""
    b = Batch([3, 200], [9999, 300], 2, 4, 16, kv, seed=12).device()
    call, verify = b.run, lambda: b.verify(f"{kv} workspace at an odd 16 bytes")
    need = b.ws.numel()
    room = torch.full((need + 1024,), 0xab, dtype=torch.uint8, device="cuda")
    at = -room.data_ptr() % 512 + 16
    b.ws = room[at:at + need]
    call()
    torch.cuda.synchronize()
    verify()
    assert (room[:at] == 0xab).all() and (room[at + need:] == 0xab).all()
