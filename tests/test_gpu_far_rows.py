"""Query rows and records past 2^31 elements: sampled rows against attention in 64 bits, bounds in attention_ref.py."""
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv

from attention_ref import DTYPE, SCALE, attend, check, gather

pytestmark = pytest.mark.gpu
D = 128


def _cache(gen, shape, kv):
    x = torch.randn(shape, generator=gen, device="cuda") / SCALE[kv]
    return (x.clamp(-448, 448) if kv == "fp8" else x).to(DTYPE[kv])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_cross_attention_over_more_than_two_to_the_31_elements(kv):
    """262 444 query tokens of 64 heads: q, out and the records (O: four times as far) pass 2^31 elements."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    Hq, Hkv, S, tokens, states = 64, 8, 16, [262144, 200, 100], [70, 0, 333]
    n = sum(tokens)
    k, v = (_cache(gen, (30, S, Hkv, D), kv) for _ in range(2))
    tables = torch.randperm(30, generator=gen, device="cuda").to(torch.int32)[None].repeat(3, 1)
    q = torch.randn(n, Hq, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    assert q.numel() > 2 ** 31
    out = torch.full_like(q, 7.0)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, lens, err = torch.tensor([0, tokens[0], tokens[0] + tokens[1], n], **i32), torch.tensor(states, **i32), torch.zeros(1, **i32)
    desc = pkv.CacheDesc.for_cache(k, SCALE[kv], SCALE[kv])
    ws = torch.empty(pkv.pkv_paged_cross_attention_workspace_size(desc, n, 3, Hq), dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_cross_attention(out, q, cu, lens, k, v, desc, tables, 0.09, ws, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    k, v, row = k.cpu(), v.cpu(), tables[0].cpu()
    for s, rows in ((0, [0, 1, 65535, 131071, 131072, 200000, 262142, 262143]), (2, [262344, 262345, 262443])):
        kk, vv = gather(k, row, states[s]), gather(v, row, states[s])
        ref, bound = attend(q[rows].cpu(), kk, vv, 0.09, kv, SCALE[kv], SCALE[kv], True)
        check(out[rows], ref, bound, f"{kv} sequence {s}")
    assert (out[262144:262344] == 0).all()


def test_shared_prefixes_over_more_than_two_to_the_31_elements():
    """8192 sequences of 2056 heads on one block of prefix."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    Hkv, G, S, n = 257, 8, 8, 8192
    Hq = Hkv * G
    i32 = dict(dtype=torch.int32, device="cuda")
    k, v = (torch.randn(n + 1, S, Hkv, D, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    tables = torch.stack([torch.full((n,), n, **i32), torch.randperm(n, generator=gen, device="cuda").to(torch.int32)], 1).contiguous()
    own = torch.randint(0, S + 1, (n,), generator=gen, **i32)
    own[-1], own[-2] = 5, 0
    lens = own + S
    q = torch.randn(n, Hq, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    assert q.numel() > 2 ** 31
    out, err = torch.full_like(q, 7.0), torch.zeros(1, **i32)
    cu, pre = torch.tensor([0, n], **i32), torch.tensor([S], **i32)
    desc = pkv.CacheDesc.for_cache(k)
    ws = torch.empty(pkv.pkv_paged_attention_decode_prefix_workspace_size(desc, n, Hq), dtype=torch.uint8, device="cuda")
    pkv.pkv_paged_attention_decode_prefix(out, q, k, v, desc, tables, lens, cu, pre, 0.09, ws, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    for s in (0, 1, 4095, 8159, 8160, 8190, 8191):
        blocks = tables[s].long()
        kk, vv = (c[blocks].cpu().double().reshape(2 * S, Hkv, D)[: int(lens[s])] for c in (k, v))
        ref, bound = attend(q[s:s + 1].cpu(), kk, vv, 0.09, "bf16", 1.0, 1.0, True)
        check(out[s:s + 1], ref, bound, f"sequence {s}")
