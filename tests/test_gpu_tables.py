"""Step planning on the GPU (pkv_extend_sequences, pkv_release_sequences) against the host block manager.

Everything is whole numbers: block tables, lengths, slots and the free stack must equal what SequenceTables gives when
it takes and returns the blocks one by one.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B
from paged_kv_cache_71_gb300.block_manager import SequenceTables

pytestmark = pytest.mark.gpu


class Device:
    """A program's device state: tables, lengths and the free stack, plus a step's outputs."""

    def __init__(self, n, width, nb, S, order, max_tokens):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.S, self.nb, self.n = S, nb, n
        self.tables = torch.full((n, width), -7, **i32)
        self.lens = torch.zeros(n, **i32)
        self.free = torch.tensor(np.asarray(order), **i32)
        self.count = torch.tensor([nb], **i32)
        self.new = torch.zeros(n, **i32)
        self.done = torch.zeros(n, dtype=torch.bool, device="cuda")
        self.keep = torch.zeros(n, **i32)
        self.slots = torch.full((max_tokens,), -99, dtype=torch.int64, device="cuda")
        self.cu = torch.full((n + 1,), -9, **i32)
        self.starts = torch.full((n,), -9, **i32)
        self.err = torch.zeros(1, **i32)

    def extend(self, new, stream=None):
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        pkv.pkv_extend_sequences(self.tables, self.lens, self.new, self.S, self.free, self.count, self.lens, self.count,
                                 self.slots, self.cu, self.starts, self.err, stream)

    def release(self, done, keep=None):
        self.done.copy_(torch.tensor(done, dtype=torch.bool))
        if keep is not None:
            self.keep.copy_(torch.tensor(keep, dtype=torch.int32))
        pkv.pkv_release_sequences(self.tables, self.lens, self.done, self.S, self.free, self.count, self.lens,
                                  self.count, None if keep is None else self.keep, self.err)


def _host_extend(host, new):
    slots, starts = [], []
    for s, n in enumerate(new):
        starts.append(host.length(s))
        slots += [host.next_slot(s) for _ in range(n)]
    return slots, starts


def _compare(dev, host, slots=None, starts=None, new=None):
    assert int(dev.err) == 0
    lens = dev.lens.tolist()
    assert lens == [host.length(s) for s in range(dev.n)]
    table = dev.tables.cpu().numpy()
    for s in range(dev.n):
        t = host.table(s)
        assert table[s, : len(t)].tolist() == t, s
    top = int(dev.count)
    assert top == host.pool.num_free
    assert dev.free[:top].tolist() == host.pool._stack[:top].tolist()
    if slots is not None:
        assert dev.slots.tolist() == slots + [-1] * (dev.slots.numel() - len(slots))
        assert dev.starts.tolist() == starts
        assert dev.cu.tolist() == np.concatenate([[0], np.cumsum(new)]).tolist()


@pytest.mark.parametrize("n,S,budget", [(1, 16, 40), (3, 4, 70), (33, 8, 500), (256, 16, 900), (257, 32, 3000),
                                        (1025, 16, 20000)])
def test_steps_follow_the_host_block_manager(n, S, budget):
    """Several steps of prompts, decode tokens, idle sequences and releases, in place."""
    rng = np.random.default_rng(n + S)
    width = 4 * (budget // S) // max(1, n // 8) + 40
    nb = n * 24 + 8 * budget // S
    order = rng.permutation(nb)
    host = SequenceTables(nb, S, free_order=order)
    for s in range(n):
        host.prefill(s, 0)
    dev = Device(n, width, nb, S, order, budget)
    for step in range(7):
        left = budget
        new = []
        for s in range(n):
            want = int(rng.choice([0, 1, 1, 1, S - 1, S, S + 1, int(rng.integers(1, 3 * S))]))
            want = min(want, left, width * S - host.length(s))
            left -= want
            new.append(want)
        slots, starts = _host_extend(host, new)
        dev.extend(new)
        _compare(dev, host, slots, starts, new)
        if step % 2:
            done = rng.random(n) < 0.4
            for s in np.flatnonzero(done):
                host.drop(int(s))
                host.prefill(int(s), 0)
            dev.release(done.tolist())
            _compare(dev, host)
    assert (dev.tables[:, -1] == -7).all()  # entries that no sequence reached stay as they were


def test_largest_batch_and_a_long_step():
    """8192 sequences; one long prompt beside decode tokens (the cluster form), slot map at an odd 8-byte address."""
    n, S, rng = 8192, 16, np.random.default_rng(0)
    nb = 60000
    order = rng.permutation(nb)
    host = SequenceTables(nb, S, free_order=order)
    for s in range(n):
        host.prefill(s, 0)
    dev = Device(n, 4096, nb, S, order, 100000)
    odd = torch.full((100001,), -99, dtype=torch.int64, device="cuda")[1:]
    assert odd.data_ptr() % 16 == 8
    dev.slots = odd
    new = [1] * n
    new[5000] = 60001
    for _ in range(2):
        slots, starts = _host_extend(host, new)
        dev.extend(new)
        _compare(dev, host, slots, starts, new)
        new = rng.integers(0, 3, size=n).tolist()
    done = [s % 3 == 0 or s == 5000 for s in range(n)]
    for s, d in enumerate(done):
        if d:
            host.drop(s)
            host.prefill(s, 0)
    dev.release(done)
    _compare(dev, host)


def test_separate_outputs_leave_the_inputs_alone():
    order = list(range(20))
    dev = Device(2, 5, 20, 8, order, 16)
    lens, count = torch.tensor([7, 9], dtype=torch.int32, device="cuda"), torch.tensor([17], dtype=torch.int32, device="cuda")
    dev.tables[0, 0], dev.tables[1, 0], dev.tables[1, 1] = 19, 18, 17
    new = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    out_lens, out_count = torch.zeros_like(lens), torch.zeros_like(count)
    for _ in range(2):  # the same call again gives the same answer
        pkv.pkv_extend_sequences(dev.tables, lens, new, 8, dev.free, count, out_lens, out_count, dev.slots)
        assert (lens.tolist(), int(count)) == ([7, 9], 17)
        assert (out_lens.tolist(), int(out_count)) == ([9, 9], 16)
        assert dev.slots[:2].tolist() == [19 * 8 + 7, 16 * 8] and (dev.slots[2:] == -1).all()
        assert dev.tables[0].tolist() == [19, 16, -7, -7, -7]


def test_shared_prefix_blocks_stay_when_a_sequence_is_released():
    """Two sequences start on the same two prefix blocks; released with keep_blocks, only their own come back."""
    S, nb = 8, 12
    dev = Device(2, 6, nb, S, list(range(nb)), 32)
    dev.count.fill_(10)  # blocks 10 and 11 hold the prefix
    dev.tables[:, 0], dev.tables[:, 1] = 11, 10
    dev.lens.fill_(2 * S)
    dev.extend([9, 1])
    assert dev.tables[:, :4].tolist() == [[11, 10, 9, 8], [11, 10, 7, -7]]
    assert dev.slots[:10].tolist() == [9 * 8 + i for i in range(8)] + [8 * 8, 7 * 8]
    dev.release([True, True], [2, 2])
    assert int(dev.err) == 0 and int(dev.count) == 10 and dev.lens.tolist() == [0, 0]
    assert dev.free[:10].tolist() == list(range(7)) + [9, 8, 7]
    dev.lens.fill_(S)
    dev.release([True, False], [5, 0])  # keeps more than it holds: nothing comes back
    assert int(dev.count) == 10 and dev.lens.tolist() == [0, S] and int(dev.err) == 0


@pytest.mark.parametrize("what,bit", [("blocks", B.DEVERR_BAD_SLOT), ("tokens", B.DEVERR_BAD_LENGTH),
                                      ("row", B.DEVERR_BAD_LENGTH), ("negative", B.DEVERR_BAD_LENGTH),
                                      ("past", B.DEVERR_BAD_LENGTH), ("count", B.DEVERR_BAD_SLOT)])
def test_a_refused_step_changes_nothing(what, bit):
    nb = 32 if what == "tokens" else 8
    dev = Device(3, 4, nb, 16, list(range(nb)), 100)
    dev.extend([20, 16, 0])
    if what == "past":
        dev.lens[1] = -1
    if what == "count":
        dev.count.fill_(9)
    before = [t.clone() for t in (dev.tables, dev.lens, dev.free)]
    lens, count = dev.lens.tolist(), int(dev.count)
    dev.extend({"blocks": [44, 48, 8], "tokens": [30, 30, 41], "row": [0, 60, 0], "negative": [1, -1, 1],
                "past": [1, 1, 1], "count": [1, 1, 1]}[what])
    assert int(dev.err) == bit
    assert torch.equal(dev.tables, before[0]) and torch.equal(dev.free, before[2])
    assert dev.lens.tolist() == lens and int(dev.count) == count
    assert (dev.slots == -1).all() and (dev.cu == 0).all() and dev.starts.tolist() == lens


@pytest.mark.parametrize("what,bit", [("length", B.DEVERR_BAD_LENGTH), ("keep", B.DEVERR_BAD_LENGTH),
                                      ("full", B.DEVERR_BAD_SLOT)])
def test_a_refused_release_changes_nothing(what, bit):
    dev = Device(2, 4, 8, 16, list(range(8)), 64)
    dev.extend([20, 33])
    dev.free[3:] = -5  # the ids taken are no longer on the stack
    if what == "length":
        dev.lens[0] = 65
    if what == "full":
        dev.count.fill_(5)
    free, lens, count = dev.free.clone(), dev.lens.tolist(), int(dev.count)
    dev.release([True, True], [0, -1] if what == "keep" else None)
    assert int(dev.err) == bit
    assert torch.equal(dev.free, free) and dev.lens.tolist() == lens and int(dev.count) == count


def test_ids_outside_the_pool_are_reported_and_get_no_slot():
    dev = Device(3, 3, 8, 8, [0, 1, 2, 3, 4, 5, 99, 7], 32)
    dev.lens[1] = 4
    dev.tables[1, 0] = 8  # one past the pool
    dev.extend([9, 2, 1])  # takes 7, then 99, then 5
    assert int(dev.err) == B.DEVERR_BAD_BLOCK
    assert dev.slots[:12].tolist() == [56 + i for i in range(8)] + [-1, -1, -1, 40]
    assert dev.tables[0, :2].tolist() == [7, -1]
    dev.err.zero_()
    dev.release([True, False, False])
    assert int(dev.err) == B.DEVERR_BAD_BLOCK
    assert dev.free[5:7].tolist() == [7, -1] and int(dev.count) == 7


def test_empty_batch_and_empty_step():
    dev = Device(0, 4, 8, 16, list(range(8)), 5)
    dev.extend([])
    assert int(dev.err) == 0 and (dev.slots == -1).all() and dev.cu.tolist() == [0] and int(dev.count) == 8
    dev.release([])
    assert int(dev.err) == 0 and int(dev.count) == 8
    dev = Device(2, 4, 8, 16, list(range(8)), 0)
    dev.extend([0, 0])
    assert int(dev.err) == 0 and dev.lens.tolist() == [0, 0] and dev.cu.tolist() == [0, 0, 0]


def test_captured_steps_replay_on_another_stream():
    """One captured decode step, replayed across block boundaries: each replay goes on where the last one ended."""
    n, S, nb, rng = 5, 4, 64, np.random.default_rng(3)
    order = rng.permutation(nb)
    host = SequenceTables(nb, S, free_order=order)
    for s in range(n):
        host.prefill(s, 0)
    dev = Device(n, 12, nb, S, order, 16)
    dev.new.fill_(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            pkv.pkv_extend_sequences(dev.tables, dev.lens, dev.new, S, dev.free, dev.count, dev.lens, dev.count,
                                     dev.slots, dev.cu, dev.starts, dev.err)
        for step in range(11):
            if step == 6:
                dev.new[2] = 0
            graph.replay()
            side.synchronize()
            new = [0 if s == 2 and step >= 6 else 1 for s in range(n)]
            slots, starts = _host_extend(host, new)
            _compare(dev, host, slots, starts, new)
