"""Groups that overlap until the stream's units are just below what 32 bits hold: reported, nothing read out of place."""
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B

pytestmark = pytest.mark.gpu
D = 128


def test_units_just_below_two_to_the_31():
    """1016 groups of the whole batch, of 64 pairs of query tiles for each of 32 heads and 512 key tiles (1032 units an item),
    and eight of one sequence: 2^31 - 64 units, which with the CTAs added would pass 2^31."""
    n, Hkv, G, S, width, tile = 2048, 32, 8, 8, 4096, 64
    cu = [0, n] * 1016 + list(range(9))
    pre = [width * S] * 2032 + [512 * tile] * 7 + [478 * tile]
    items = n * G // 256 * Hkv
    assert 1016 * items * (2 * 512 + 8) + Hkv * (7 * (512 + 4) + 478 + 4) == 2 ** 31 - 64
    i32 = dict(dtype=torch.int32, device="cuda")
    k = torch.zeros(2, S, Hkv, D, dtype=torch.bfloat16, device="cuda")
    desc = pkv.CacheDesc.for_cache(k)
    tables = torch.zeros(n, width, **i32)
    lens = torch.full((n,), width * S, **i32)
    q = torch.zeros(n, Hkv * G, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    ws = torch.zeros(pkv.pkv_paged_attention_decode_prefix_workspace_size(desc, n, Hkv * G), dtype=torch.uint8, device="cuda")
    err = torch.zeros(1, **i32)
    pkv.pkv_paged_attention_decode_prefix(out, q, k, k, desc, tables, lens, torch.tensor(cu, **i32), torch.tensor(pre, **i32),
                                          0.1, ws, err)
    assert int(err) & B.DEVERR_BAD_LENGTH
    assert (out == 0).all()
