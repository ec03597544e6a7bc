"""The CUDA-core decode, and single-token cross attention through it, at batch sizes whose block counts leave the warps'
pipelines just less room than one more stage, or just as much: short contexts, against attention in 64 bits.  Tolerances in
parity.py."""
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv

from parity import TOL

pytestmark = pytest.mark.gpu

DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}

# head dim, block size, cache, GQA group, batches
SHAPES = [(64, 4, "f32", 4, (640, 927)), (64, 4, "f32", 8, (5248, 5439)), (64, 8, "f32", 1, (4864, 5215)),
          (64, 8, "f32", 2, (1408, 1727)), (64, 16, "bf16", 1, (6400, 6751)), (64, 16, "bf16", 2, (4480, 4799)),
          (64, 16, "bf16", 4, (640, 927)), (64, 16, "f32", 4, (1600, 1823)), (64, 32, "e4m3", 1, (6400, 6751)),
          (64, 32, "e4m3", 2, (4480, 4799)), (64, 32, "e4m3", 4, (640, 927)), (64, 32, "bf16", 4, (3712, 4895)),
          (64, 32, "bf16", 8, (832, 1023)), (64, 32, "f32", 8, (1696, 1887)), (128, 4, "bf16", 4, (640, 927)),
          (128, 4, "f32", 8, (6400, 6591)), (128, 8, "bf16", 1, (4864, 5215)), (128, 8, "bf16", 2, (1408, 1727)),
          (128, 16, "bf16", 1, (6400, 7039)), (128, 16, "bf16", 2, (4480, 5311)),
          (128, 16, "bf16", 4, (639, 640, 927, 928, 1600, 1823)), (128, 16, "f32", 4, (1600, 2271)),
          (128, 32, "bf16", 1, (7552, 7967)), (128, 32, "bf16", 4, (4672, 5343)), (128, 32, "f32", 8, (1984, 2175)),
          (128, 16, "bf16", 4, (8192,)), (128, 32, "f32", 8, (8192,))]


@pytest.mark.parametrize("D,S,kv,G,B", [(*s[:4], b) for s in SHAPES for b in s[4]])
@pytest.mark.parametrize("call", ["decode", "cross"])
def test_every_batch_launches(D, S, kv, G, B, call):
    gen = torch.Generator(device="cuda").manual_seed(B)
    Hkv = 1
    q_dtype = torch.float32 if kv == "f32" else torch.bfloat16
    lens = torch.randint(0, 2 * S + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    tables = torch.randperm(2 * B, generator=gen, device="cuda").to(torch.int32).view(B, 2)
    k, v = (torch.randn(2 * B, S, Hkv, D, generator=gen, device="cuda").to(DTYPE[kv]) for _ in range(2))
    q = torch.randn(B, Hkv * G, D, generator=gen, device="cuda").to(q_dtype)
    out = torch.full_like(q, 7.0)
    desc = pkv.CacheDesc.for_cache(k)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = D ** -0.5
    if call == "decode":
        ws = torch.empty(pkv.pkv_paged_attention_workspace_size(desc, B, G, 0), dtype=torch.uint8, device="cuda")
        pkv.pkv_paged_attention_decode(out, q, k, v, desc, tables, lens, scale, workspace=ws, device_error=err)
    else:
        ws = torch.empty(pkv.pkv_paged_cross_attention_workspace_size(desc, B, B, G), dtype=torch.uint8, device="cuda")
        pkv.pkv_paged_cross_attention(out, q, None, lens, k, v, desc, tables, scale, ws, err)
    assert int(err) == 0
    kk, vv = (c.to(torch.float32)[tables.long()].reshape(B, 2 * S, D).double() for c in (k, v))
    s = torch.einsum("bgd,btd->bgt", q.double(), kk) * scale
    s = s.masked_fill(torch.arange(2 * S, device="cuda") >= lens[:, None, None], float("-inf"))
    ref = torch.einsum("bgt,btd->bgd", torch.softmax(s, -1).nan_to_num(0.0), vv)  # rows without keys are zero
    atol, rtol = TOL[kv]
    assert ((out.double() - ref).abs() <= atol + rtol * ref.abs()).all()
