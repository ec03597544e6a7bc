"""Host threads that call the same attention operator with batches of different sizes, whose kernels take different
amounts of shared memory; each thread has its own stream, outputs and workspace.  Every call must launch, and the last ones
give what the same call gives alone."""
import sys
import threading

import pytest
import torch

import paged_kv_cache_71_gb300 as pkv

pytestmark = pytest.mark.gpu
D, S = 128, 16


class Case:
    def __init__(self, call, kv, B, G):
        i32 = dict(dtype=torch.int32, device="cuda")
        gen = torch.Generator(device="cuda").manual_seed(B)
        dt = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}[kv]
        self.call, self.B, self.G = call, B, G
        self.tables = torch.randperm(2 * B, generator=gen, device="cuda").to(torch.int32).view(B, 2)
        self.lens = torch.randint(S + 1, 2 * S + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        self.k, self.v = (torch.randn(2 * B, S, 1, D, generator=gen, device="cuda").to(dt) for _ in range(2))
        self.q = torch.randn(B, G, D, generator=gen, device="cuda").to(torch.bfloat16)
        self.out = torch.zeros_like(self.q)
        self.desc = pkv.CacheDesc.for_cache(self.k)
        self.cu, self.pre = torch.tensor([0, B], **i32), torch.zeros(1, **i32)
        self.cu_q, self.starts = torch.arange(B + 1, **i32), self.lens - 1
        self.err = torch.zeros(1, **i32)
        size = {"decode": lambda: pkv.pkv_paged_attention_workspace_size(self.desc, B, G, 0),
                "prefix": lambda: pkv.pkv_paged_attention_decode_prefix_workspace_size(self.desc, B, G),
                "mixed": lambda: pkv.pkv_paged_attention_mixed_workspace_size(self.desc, B, G)}[call]()
        self.ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def run(self):
        if self.call == "decode":
            pkv.pkv_paged_attention_decode(self.out, self.q, self.k, self.v, self.desc, self.tables, self.lens, 0.1,
                                           workspace=self.ws, device_error=self.err)
        elif self.call == "prefix":
            pkv.pkv_paged_attention_decode_prefix(self.out, self.q, self.k, self.v, self.desc, self.tables, self.lens, self.cu,
                                                  self.pre, 0.1, self.ws, self.err)
        else:
            pkv.pkv_paged_attention_mixed(self.out, self.q, self.cu_q, self.starts, self.lens, self.k, self.v, self.desc,
                                          self.tables, self.B, 0.1, self.ws, self.err)


@pytest.mark.parametrize("call,kv,G,sizes", [("decode", "bf16", 4, (5, 600)), ("decode", "fp8", 4, (5, 2000)),
                                             ("decode", "bf16", 8, (5, 2000)), ("prefix", "bf16", 4, (5, 600)),
                                             ("prefix", "fp8", 4, (5, 2000)), ("mixed", "bf16", 4, (5, 1900))])
def test_batches_of_different_sizes_at_once(call, kv, G, sizes):
    cases = [Case(call, kv, n, G) for n in sizes for _ in range(3)]
    alone = []
    for c in cases:
        c.run()
        alone.append(c.out.clone())
        c.out.zero_()
    torch.cuda.synchronize()
    failed = []

    def work(c):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for i in range(2500):
                    c.run()
                    if i % 250 == 249:  # (a full queue would have the threads wait inside their launches)
                        torch.cuda.current_stream().synchronize()
        except BaseException as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    sys.setswitchinterval(interval)
    assert not failed, failed
    for c, want in zip(cases, alone):
        assert int(c.err) == 0 and torch.equal(c.out, want)
