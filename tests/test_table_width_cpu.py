"""Tables whose rows hold more tokens than 32 bits count are refused on the host by every decode form, before the device is
asked for."""
import ctypes

import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B

OUT_OF_RANGE, CUDA = 3, 5


def _desc(S):
    return ctypes.byref(B.CacheDesc(num_blocks=16, block_size=S, num_kv_heads=1, head_dim=128, dtype=B.PKV_BF16, k_scale=1.0,
                                    v_scale=1.0))


def _call(name, S, width):
    L = pkv.lib()
    if name in ("decode", "shared"):
        f = L.pkv_paged_attention_decode if name == "decode" else L.pkv_paged_attention_decode_shared
        return f(16, 16, B.PKV_BF16, 16, 16, _desc(S), 16, width, 16, 1, 8, 0.1, 1, 0, None, 0, None, None)
    if name == "cross":
        return L.pkv_paged_cross_attention(16, 16, B.PKV_BF16, 1, None, 16, 16, 16, _desc(S), 16, width, 1, 8, 0.1, 16, 1 << 30,
                                           None, None)
    return L.pkv_paged_attention_mixed(16, 16, B.PKV_BF16, 1, 16, 16, 16, 16, 16, _desc(S), 16, width, 1, 1, 8, 0.1, 16,
                                       1 << 30, None, None)


FORMS = [(n, S) for n in ("decode", "shared", "cross") for S in (4, 8, 16, 32)] + [("mixed", 16)]


@pytest.mark.skipif(torch.cuda.is_available(), reason="16 is no device address: for a machine without a device")
@pytest.mark.parametrize("name,S", FORMS)
def test_rows_of_two_to_the_31_tokens_and_more(name, S):
    """(2^32 / S + 1 blocks would wrap to a row of S tokens.)  The widest row below passes, and the device is asked for."""
    for width in (2 ** 31 // S, 2 ** 31 // S + 1, 2 ** 32 // S + 1):
        if width < 2 ** 31 - 64:
            assert _call(name, S, width) == OUT_OF_RANGE
            assert "2^31-1 tokens" in pkv.pkv_last_error()
    assert _call(name, S, 2 ** 31 // S - 1) == CUDA
