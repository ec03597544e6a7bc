"""Step planning, cache writes, shared-prefix decode and cross attention together, as a decoder over an encoder would run
them: prompts as chunks, then decode steps replayed from one captured graph, a sequence finished and its row given to a new
prompt in between.  Every step is checked against attention in 64 bits over what was written; bounds in attention_ref.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B
from paged_kv_cache_71_gb300.block_manager import SequenceTables

from attention_ref import DTYPE, SCALE, attend, check, gather, make_cache

pytestmark = pytest.mark.gpu
D, S, HKV, G = 128, 16, 2, 4
HQ = HKV * G
PREFIX = [48, 48, 48, 0, 0, 16, 16]      # of each row; the last row is idle
GROUPS = [0, 3, 4, 5, 7]
PROMPT = [3, 1, 20, 5, 30, 17, 0]
STATES = [33, 64, 1, 500, 130, 65, 0]    # encoder states of each row
MAX_TOKENS = 80                          # of a step


class Loop:
    def __init__(self, kv):
        self.gen = torch.Generator().manual_seed(71)
        self.kv, self.n, nb = kv, len(PROMPT), 60
        i32 = dict(dtype=torch.int32, device="cuda")
        shared = {0: [7, 31, 2], 5: [44]}    # the prefixes' blocks, which stay out of the free stack
        shared.update({1: shared[0], 2: shared[0], 6: shared[5]})
        taken = {7, 31, 2, 44}
        free = [b for b in torch.randperm(nb, generator=self.gen).tolist() if b not in taken]
        self.host = SequenceTables(nb, S, free_order=free + sorted(taken))
        self.host.pool._top = len(free)
        self.tables = torch.full((self.n, 12), -1, dtype=torch.int32)
        for s, blocks in shared.items():
            self.tables[s, :len(blocks)] = torch.tensor(blocks, dtype=torch.int32)
        self.tables = self.tables.cuda()
        self.free = torch.tensor(free + [-1] * len(taken), **i32)
        self.count = torch.tensor([len(free)], **i32)
        self.lens = torch.tensor([p if s < self.n - 1 else 0 for s, p in enumerate(PREFIX)], **i32)
        self.new = torch.zeros(self.n, **i32)
        self.slots = torch.zeros(MAX_TOKENS, dtype=torch.int64, device="cuda")
        self.cu, self.starts = torch.zeros(self.n + 1, **i32), torch.zeros(self.n, **i32)
        self.err = torch.zeros(1, **i32)
        self.finished = torch.zeros(self.n, dtype=torch.bool, device="cuda")
        self.keep = torch.tensor([p // S for p in PREFIX], **i32)
        self.k = torch.zeros(nb, S, HKV, D, device="cuda").to(DTYPE[kv])
        self.v = torch.zeros_like(self.k)
        self.desc = pkv.CacheDesc.for_cache(self.k, SCALE[kv], SCALE[kv])
        # the encoder's states
        blocks = [-(-L // S) for L in STATES]
        self.ek, self.ev = (make_cache(self.gen, (sum(blocks) + 1, S, HKV, D), kv) for _ in range(2))
        self.etab = torch.full((self.n, max(blocks)), -1, dtype=torch.int32)
        for s, b in enumerate(blocks):
            self.etab[s, :b] = torch.arange(sum(blocks[:s]), sum(blocks[:s + 1]))
        self.dek, self.dev, self.detab = self.ek.cuda(), self.ev.cuda(), self.etab.cuda()
        self.elens = torch.tensor(STATES, **i32)
        self.edesc = pkv.CacheDesc.for_cache(self.dek, SCALE[kv], SCALE[kv])
        # the prefixes of the groups that have one
        self.cug = torch.tensor(GROUPS, **i32)
        self.pre = torch.tensor([PREFIX[g] for g in GROUPS[:-1]], **i32)
        self.scale = 1 / np.sqrt(D)
        sizes = [pkv.pkv_paged_attention_decode_prefix_workspace_size(self.desc, self.n, HQ),
                 pkv.pkv_paged_cross_attention_workspace_size(self.edesc, MAX_TOKENS, self.n, HQ),
                 pkv.pkv_paged_cross_attention_workspace_size(self.edesc, self.n, self.n, HQ)]
        self.ws = torch.full((max(sizes),), 0xff, dtype=torch.uint8, device="cuda")  # one for all calls, one after another
        self.hist = {}
        for s in (0, 5):
            kk, vv = self.rand(PREFIX[s], HKV), self.rand(PREFIX[s], HKV)
            at = torch.tensor([shared[s][p // S] * S + p % S for p in range(PREFIX[s])], device="cuda")
            pkv.pkv_reshape_and_cache(kk.cuda(), vv.cuda(), at, self.k, self.v, self.desc, self.err)
            self.hist[s] = [(self.code(kk), self.code(vv))]
        for s, like in ((1, 0), (2, 0), (6, 5)):
            self.hist[s] = list(self.hist[like])
        self.hist[3], self.hist[4] = [], []
        for s in range(self.n):
            self.host.prefill(s, 0)

    def rand(self, n, heads):
        return torch.randn(n, heads, D, generator=self.gen).to(torch.bfloat16)

    def code(self, x):
        """What the cache holds of x, unscaled, in 64 bits (the scales are powers of two)."""
        return (x.float() / SCALE[self.kv]).to(DTYPE[self.kv]).double()

    def plan(self):
        pkv.pkv_extend_sequences(self.tables, self.lens, self.new, S, self.free, self.count, self.lens, self.count,
                                 self.slots, self.cu, self.starts, self.err)

    def check_plan(self, new):
        """The same blocks and slots as the host block manager's (whose sequences are the rows' own parts)."""
        slots = [self.host.next_slot(s) for s, n in enumerate(new) for _ in range(n)]
        assert self.slots.tolist() == slots + [-1] * (MAX_TOKENS - len(slots))
        assert self.lens.tolist() == [PREFIX[s] + self.host.length(s) if self.host.length(s) else 0 for s in range(self.n)]
        assert int(self.count) == self.host.pool.num_free

    def check_row(self, got, q, s, upto, tile, what):
        k, v = (torch.cat([h[i] for h in self.hist[s]])[:upto] for i in (0, 1))
        ref, bound = attend(q[None], k, v, self.scale, self.kv, SCALE[self.kv], SCALE[self.kv], tile)
        if not tile and PREFIX[s]:  # prefix and own blocks round differently: the looser of the two
            bound = torch.maximum(bound, attend(q[None], k, v, self.scale, self.kv, SCALE[self.kv], SCALE[self.kv], True)[1])
        check(got[None], ref, bound, f"{what}, row {s}")

    def check_cross(self, got, q, s, tile, what):
        k, v = gather(self.ek, self.etab[s], STATES[s]), gather(self.ev, self.etab[s], STATES[s])
        ref, bound = attend(q, k, v, self.scale, self.kv, SCALE[self.kv], SCALE[self.kv], tile)
        check(got, ref, bound, f"{what}, row {s}")

    def prompts(self, new, what):
        """A step of prompt chunks: planned, written, causal attention and cross attention by the same cu_q."""
        q, kk, vv = self.rand(MAX_TOKENS, HQ), self.rand(MAX_TOKENS, HKV), self.rand(MAX_TOKENS, HKV)
        dq = q.cuda()
        out, cross = torch.full_like(dq, 7.0), torch.full_like(dq, 7.0)
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        self.plan()
        pkv.pkv_reshape_and_cache(kk.cuda(), vv.cuda(), self.slots, self.k, self.v, self.desc, self.err)
        pkv.pkv_paged_prefill_varlen(out, dq, self.cu, self.starts, self.lens, self.k, self.v, self.desc, self.tables,
                                     self.scale, self.err)
        pkv.pkv_paged_cross_attention(cross, dq, self.cu, self.elens, self.dek, self.dev, self.edesc, self.detab, self.scale,
                                      self.ws, self.err)
        self.check_plan(new)
        at = 0
        for s, n in enumerate(new):
            if n == 0:
                continue
            past = sum(len(h[0]) for h in self.hist[s])
            self.hist[s].append((self.code(kk[at:at + n]), self.code(vv[at:at + n])))
            for i in range(n):
                self.check_row(out[at + i], q[at + i], s, past + i + 1, True, what)
            self.check_cross(cross[at:at + n], q[at:at + n], s, True, what)
            at += n
        assert (out[at:] == 7).all() and (cross[at:] == 7).all()
        assert int(self.err) == 0

    def capture(self):
        """One decode step of all rows; a row's token is row s of q, k and v (the idle row is the last one)."""
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.q1, self.kn, self.vn = (torch.zeros(self.n, h, D, **bf) for h in (HQ, HKV, HKV))
        self.out, self.cross = torch.zeros_like(self.q1), torch.zeros_like(self.q1)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side), torch.cuda.graph(self.graph, stream=side):
            self.plan()
            pkv.pkv_reshape_and_cache(self.kn, self.vn, self.slots[:self.n], self.k, self.v, self.desc, self.err)
            pkv.pkv_paged_attention_decode_prefix(self.out, self.q1, self.k, self.v, self.desc, self.tables, self.lens,
                                                  self.cug, self.pre, self.scale, self.ws, self.err)
            pkv.pkv_paged_cross_attention(self.cross, self.q1, None, self.elens, self.dek, self.dev, self.edesc, self.detab,
                                          self.scale, self.ws, self.err)
        torch.cuda.current_stream().wait_stream(side)

    def decode(self, what):
        new = [1] * (self.n - 1) + [0]
        q, kk, vv = self.rand(self.n, HQ), self.rand(self.n, HKV), self.rand(self.n, HKV)
        for dst, src in ((self.q1, q), (self.kn, kk), (self.vn, vv), (self.new, torch.tensor(new, dtype=torch.int32))):
            dst.copy_(src)
        self.out.fill_(7.0)
        self.graph.replay()
        self.check_plan(new)
        for s in range(self.n - 1):
            self.hist[s].append((self.code(kk[s:s + 1]), self.code(vv[s:s + 1])))
            self.check_row(self.out[s], q[s], s, None, False, what)
            self.check_cross(self.cross[s:s + 1], q[s:s + 1], s, False, what)
        assert (self.out[-1] == 0).all() and (self.cross[-1] == 0).all()  # nothing to attend to
        assert int(self.err) == 0

    def finish(self, s):
        self.finished.zero_()
        self.finished[s] = True
        pkv.pkv_release_sequences(self.tables, self.lens, self.finished, S, self.free, self.count, self.lens, self.count,
                                  self.keep, self.err)
        for b in self.host.table(s):
            self.host.pool.release(b)
        self.host.prefill(s, 0)
        self.hist[s] = self.hist[s][:1] if PREFIX[s] else []
        assert self.lens[s] == 0 and int(self.count) == self.host.pool.num_free
        if PREFIX[s]:
            self.lens[s] = PREFIX[s]  # the row starts again on the prefix


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_decoder_steps_from_one_graph(kv):
    x = Loop(kv)
    x.prompts(PROMPT, f"{kv} prompts")
    x.capture()
    for t in range(18):  # every row crosses a block boundary
        x.decode(f"{kv} step {t}")
    for s in (4, 1):     # a row of its own, and one that shares a prefix
        x.finish(s)
    x.prompts([0, 6, 0, 0, 33, 0, 0], f"{kv} new prompts")
    for t in range(3):
        x.decode(f"{kv} step {t} after new prompts")


def test_a_sequence_of_length_zero_in_a_group_with_a_prefix():
    """Finished rows and padding have length 0: zero rows and no error, whichever row of the group it is."""
    x = Loop("bf16")
    x.prompts(PROMPT, "prompts")
    q = x.rand(x.n, HQ)
    for empty in (0, 2):
        lens = x.lens.clone()
        lens[empty] = 0
        out = torch.full((x.n, HQ, D), 7.0, dtype=torch.bfloat16, device="cuda")
        pkv.pkv_paged_attention_decode_prefix(out, q.cuda(), x.k, x.v, x.desc, x.tables, lens, x.cug, x.pre, x.scale, x.ws,
                                              x.err)
        assert int(x.err) == 0 and (out[empty] == 0).all() and (out[-1] == 0).all()
        for s in range(x.n - 1):
            if s != empty:
                x.check_row(out[s], q[s], s, None, False, "beside an empty row")
