"""What the binding of the shared-prefix decode, cross attention and step planning refuses before the library is called."""
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B

BF, FP8, I8, U8 = torch.bfloat16, torch.float8_e4m3fn, torch.int8, torch.uint8


def _z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def _desc(dtype, num_blocks=4):
    return B.CacheDesc(num_blocks=num_blocks, block_size=16, num_kv_heads=2, head_dim=128, dtype=dtype, k_scale=1.0,
                       v_scale=1.0)


def _prefix(desc, k, v, **o):
    a = dict(out=_z(2, 8, 128, dtype=BF), q=_z(2, 8, 128, dtype=BF), bt=_z(2, 4), lens=_z(2), cu=_z(2), pre=_z(1), ws=None)
    a.update(o)
    pkv.pkv_paged_attention_decode_prefix(a["out"], a["q"], k, v, desc, a["bt"], a["lens"], a["cu"], a["pre"], 0.1, a["ws"])


def _cross(desc, k, v, **o):
    a = dict(out=_z(2, 8, 128, dtype=BF), q=_z(2, 8, 128, dtype=BF), bt=_z(2, 4), lens=_z(2), cu=_z(3), ws=None)
    a.update(o)
    pkv.pkv_paged_cross_attention(a["out"], a["q"], a["cu"], a["lens"], k, v, desc, a["bt"], 0.1, a["ws"])


@pytest.mark.parametrize("call", [_prefix, _cross])
@pytest.mark.parametrize("code,dtype", [(B.PKV_BF16, FP8), (B.PKV_BF16, I8), (B.PKV_BF16, U8), (B.PKV_FP8_E4M3, BF),
                                        (B.PKV_FP8_E4M3, I8), (B.PKV_INT8, FP8), (B.PKV_INT8, BF), (B.PKV_F32, BF)])
def test_caches_of_another_type_than_the_descriptor_says(call, code, dtype):
    """A bf16 descriptor over one-byte caches would have the copies read up to twice the tensors."""
    cache = _z(4, 16, 2, 128, dtype=dtype)
    with pytest.raises(pkv.PkvError, match="k_cache has dtype"):
        call(_desc(code), cache, cache)


@pytest.mark.parametrize("call", [_prefix, _cross])
@pytest.mark.parametrize("code,dtype", [(B.PKV_BF16, BF), (B.PKV_FP8_E4M3, FP8), (B.PKV_FP8_E4M3, U8), (B.PKV_INT8, I8)])
def test_caches_of_the_descriptors_type_pass_that_check(call, code, dtype):
    """(They are on the CPU here, which is refused next.)"""
    cache = _z(4, 16, 2, 128, dtype=dtype)
    with pytest.raises((pkv.PkvError, RuntimeError), match="CUDA"):
        call(_desc(code), cache, cache)
