"""The widest table rows that the decode forms take (just below 2^31 tokens), with short contexts: as over a narrow table."""
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [16, 32])
@pytest.mark.parametrize("G", [1, 8])
def test_decode_and_single_token_cross_attention(S, G):
    gen = torch.Generator(device="cuda").manual_seed(S + G)
    k, v = (torch.randn(20, S, 1, 128, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(1, G, 128, generator=gen, device="cuda").to(torch.bfloat16)
    row = torch.randperm(20, generator=gen, device="cuda").to(torch.int32)[None]
    wide = torch.zeros(1, 2 ** 31 // S - 1, dtype=torch.int32, device="cuda")
    wide[:, :20] = row
    desc, err = pkv.CacheDesc.for_cache(k), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkv.pkv_paged_cross_attention_workspace_size(desc, 1, 1, G), dtype=torch.uint8, device="cuda")
    lens = torch.tensor([20 * S - 3], dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(q) for _ in range(5)]
    pkv.pkv_paged_attention_decode(outs[0], q, k, v, desc, row, lens, 0.1, workspace=ws, device_error=err)
    pkv.pkv_paged_attention_decode(outs[1], q, k, v, desc, wide, lens, 0.1, workspace=ws, device_error=err)
    pkv.pkv_paged_cross_attention(outs[2], q, None, lens, k, v, desc, wide, 0.1, ws, err)
    pkv.pkv_paged_attention_decode(outs[3], q, k, v, desc, row, lens, 0.1, num_splits=3, max_context_len=20 * S, workspace=ws,
                                   device_error=err)
    pkv.pkv_paged_attention_decode(outs[4], q, k, v, desc, wide, lens, 0.1, num_splits=3, max_context_len=20 * S, workspace=ws,
                                   device_error=err)
    assert int(err) == 0 and (outs[0] != 0).any()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and torch.equal(outs[3], outs[4])
