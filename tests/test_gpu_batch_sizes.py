"""Step planning over every size of batch: around the sizes at which the kernels' shared memory passes what every kernel may
have (4075 sequences an extend, 6112 a release), in a process that has had no larger batch, and from two host threads at once."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import paged_kv_cache_71_gb300 as pkv

pytestmark = pytest.mark.gpu
S, WIDTH = 16, 4


class Plan:
    """n sequences with two tokens each; an extend takes 15 more, a release hands every second sequence's blocks back."""

    def __init__(self, n):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.n, self.nb = n, 2 * n + 1
        self.tables = torch.full((n, WIDTH), -1, **i32)
        self.tables[:, 0] = torch.arange(n, device="cuda")
        self.lens, self.new = torch.full((n,), 2, **i32), torch.full((n,), 15, **i32)
        self.free, self.count = torch.arange(self.nb, **i32).flip(0).contiguous(), torch.tensor([n + 1], **i32)
        self.slots = torch.zeros(15 * n, dtype=torch.int64, device="cuda")
        self.out, self.left, self.err = torch.zeros(n, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)
        self.done = torch.arange(n, device="cuda") % 2 == 0

    def extend(self, in_place=False):
        pkv.pkv_extend_sequences(self.tables, self.lens, self.new, S, self.free, self.count,
                                 self.lens if in_place else self.out, self.count if in_place else self.left, self.slots,
                                 device_error=self.err)

    def release(self, in_place=False):
        pkv.pkv_release_sequences(self.tables, self.lens, self.done, S, self.free, self.count,
                                  self.lens if in_place else self.out, self.count if in_place else self.left,
                                  device_error=self.err)

    def check_extend(self):
        """Sequence s takes the s-th id from the top of the stack: position 16 of each is the first slot of its new block."""
        s = torch.arange(self.n, device="cuda")
        ids = self.free[self.n - s].long()
        assert torch.equal(self.tables[:, 1].long(), ids)
        slots = self.slots.view(self.n, 15)
        assert torch.equal(slots[:, :14], s[:, None] * S + 2 + torch.arange(14, device="cuda"))
        assert torch.equal(slots[:, 14], ids * S)
        assert int(self.err) == 0


def sizes(ns):
    """Extends and releases of these sizes, small ones first (run in a process of its own)."""
    for n in ns:
        for in_place in (False, True):
            p = Plan(n)
            p.extend(in_place)
            p.check_extend()
            lens, count = (p.lens, p.count) if in_place else (p.out, p.left)
            assert (lens == 17).all() and int(count) == 1
            p.lens.fill_(17)
            p.count.fill_(1)
            p.release(in_place)
            lens, count = (p.lens, p.count) if in_place else (p.out, p.left)
            assert torch.equal(lens, torch.where(p.done, 0, 17).int()) and int(count) == 1 + 2 * ((n + 1) // 2)
            back = p.tables[::2, :2].reshape(-1)
            assert torch.equal(p.free[1:1 + back.numel()], back) and int(p.err) == 0


@pytest.mark.parametrize("ns", [[4075], [4095], [6112], [6143], [4009, 4010, 4074, 4096, 6015, 6016, 6111, 6144, 8192]])
def test_sizes_in_a_process_that_has_had_no_larger_one(ns):
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", f"import test_gpu_batch_sizes as t; t.sizes([64] + {ns})"], text=True,
                       capture_output=True, timeout=300, cwd=here, env={**os.environ, "PYTHONPATH": os.path.dirname(here)})
    assert r.returncode == 0, r.stderr[-800:]


@pytest.mark.parametrize("call", ["extend", "release"])
def test_two_host_threads_with_different_batches(call):
    """Both batches need more shared memory than every kernel may have; each thread has its own stream and arrays."""
    failed = []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                p = Plan(n)
                if call == "release":
                    p.lens.fill_(16)
                torch.cuda.current_stream().synchronize()
                for _ in range(1500):
                    getattr(p, call)()
                torch.cuda.current_stream().synchronize()
                if call == "extend":
                    p.check_extend()
                else:
                    assert int(p.err) == 0 and int(p.left) == n + 1 + (n + 1) // 2
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(n,)) for n in (6200, 8192)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
