"""The first CUDA call of a host thread is the library's: every call launches and gives what it gives on the main thread."""
import threading

import pytest
import torch

import paged_kv_cache_71_gb300 as pkv

pytestmark = pytest.mark.gpu
D, S, B, G, HKV = 128, 16, 7, 4, 2


def _calls(kv):
    i32 = dict(dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    tables = torch.randperm(4 * B, generator=gen, device="cuda").to(torch.int32).view(B, 4)
    lens = torch.randint(S + 1, 4 * S + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    k, v = (torch.randn(4 * B, S, HKV, D, generator=gen, device="cuda").to(kv) for _ in range(2))
    q = torch.randn(B, HKV * G, D, generator=gen, device="cuda").to(torch.bfloat16)
    desc = pkv.CacheDesc.for_cache(k)
    cu, pre, cu_q, err = torch.tensor([0, B], **i32), torch.zeros(1, **i32), torch.arange(B + 1, **i32), torch.zeros(1, **i32)
    hq = HKV * G
    sizes = [pkv.pkv_paged_attention_workspace_size(desc, B, hq, 0), pkv.pkv_paged_attention_mixed_workspace_size(desc, B, hq),
             pkv.pkv_paged_attention_decode_prefix_workspace_size(desc, B, hq),
             pkv.pkv_paged_cross_attention_workspace_size(desc, B, B, hq)]
    ws = torch.empty(max(sizes), dtype=torch.uint8, device="cuda")
    starts = lens - 1
    return err, {
        "decode": lambda o, st: pkv.pkv_paged_attention_decode(o, q, k, v, desc, tables, lens, 0.1, workspace=ws,
                                                               device_error=err, stream=st),
        "shared": lambda o, st: pkv.pkv_paged_attention_decode_shared(o, q, k, v, desc, tables, lens, 0.1, workspace=ws,
                                                                      device_error=err, stream=st),
        "mixed": lambda o, st: pkv.pkv_paged_attention_mixed(o, q, cu_q, starts, lens, k, v, desc, tables, B, 0.1, ws, err, st),
        "varlen": lambda o, st: pkv.pkv_paged_prefill_varlen(o, q, cu_q, starts, lens, k, v, desc, tables, 0.1, err, st),
        "prefix": lambda o, st: pkv.pkv_paged_attention_decode_prefix(o, q, k, v, desc, tables, lens, cu, pre, 0.1, ws, err, st),
        "cross": lambda o, st: pkv.pkv_paged_cross_attention(o, q, cu_q, lens, k, v, desc, tables, 0.1, ws, err, st),
        "single": lambda o, st: pkv.pkv_paged_cross_attention(o, q, None, lens, k, v, desc, tables, 0.1, ws, err, st),
    }, q


@pytest.mark.parametrize("call", ["decode", "shared", "mixed", "varlen", "prefix", "cross", "single"])
@pytest.mark.parametrize("kv", [torch.bfloat16, torch.float8_e4m3fn])
def test_first_call_of_a_thread(call, kv):
    err, calls, q = _calls(kv)
    stream = torch.cuda.Stream()
    outs, failed = [torch.zeros_like(q) for _ in range(2)], []
    calls[call](outs[0], stream)
    stream.synchronize()

    def work():
        try:
            calls[call](outs[1], stream)
        except BaseException as e:
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    stream.synchronize()
    assert not failed, failed
    assert int(err) == 0 and torch.equal(outs[0], outs[1]) and (outs[0] != 0).any()
