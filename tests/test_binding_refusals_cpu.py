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


@pytest.mark.parametrize("call", [_prefix, _cross])
@pytest.mark.parametrize("kw,text", [(dict(q=_z(16, 128, dtype=BF)), "q has shape"), (dict(q=_z(1, dtype=BF)), "q has shape"),
                                     (dict(bt=_z(8)), "block_tables has shape"), (dict(bt=_z(())), "block_tables has shape"),
                                     (dict(bt=_z(1, 2, 4)), "block_tables has shape"), (dict(lens=_z(2, 1)), "shape"),
                                     (dict(cu=_z(1, 3)), "cu_[qg].* has shape")])
def test_shapes_that_sizes_are_taken_from(call, kw, text):
    cache = _z(4, 16, 2, 128, dtype=BF)
    with pytest.raises(pkv.PkvError, match=text):
        call(_desc(B.PKV_BF16), cache, cache, **kw)


@pytest.mark.parametrize("call", ["pkv_extend_sequences", "pkv_release_sequences"])
@pytest.mark.parametrize("name,bad", [("past", (2, 1)), ("past", ()), ("bt", (8,)), ("bt", ()), ("bt", (1, 2, 4))])
def test_shapes_of_step_planning(call, name, bad):
    a = dict(bt=_z(2, 4), past=_z(2))
    a[name] = _z(bad)
    with pytest.raises(pkv.PkvError, match="past_lens has shape" if name == "past" else "block_tables has shape"):
        if call == "pkv_extend_sequences":
            pkv.pkv_extend_sequences(a["bt"], a["past"], _z(2), 16, _z(8), _z(1), _z(2), _z(1), _z(8, dtype=torch.int64))
        else:
            pkv.pkv_release_sequences(a["bt"], a["past"], _z(2, dtype=torch.bool), 16, _z(8), _z(1), _z(2), _z(1))


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int16, torch.bool])
def test_an_error_word_that_is_too_small(dtype):
    """The kernels OR into 4 aligned bytes.  (Device -1 stands for where the tensors are.)"""
    with pytest.raises(pkv.PkvError, match="device_error has dtype"):
        B._refuse("call", -1, device_error=_z(1, dtype=dtype))
    assert not B._word(_z(1, dtype=dtype), -1) and B._word(_z(1), -1) and B._word(None, 0) and B._word(4096, 0)


def test_workspaces_without_a_size():
    """A raw pointer has no size, and a view that repeats one element has less room than its size says."""
    for ws, text in ((1 << 20, "raw pointer"), (torch.empty(1, dtype=torch.uint8).expand(1 << 20), "contiguous")):
        with pytest.raises(pkv.PkvError, match=text) as e:
            B._refuse("call", -1, workspace=ws)
        assert e.value.status == 4 and not B._room(ws, -1)
    assert B._room(None, 0) and B._room(_z(4), -1) and not B._room(_z(4), 0)


@pytest.mark.gpu
@pytest.mark.parametrize("call", [_prefix, _cross])
def test_a_raw_pointer_as_workspace_on_the_device(call):
    cache = _z(4, 16, 2, 128, dtype=BF).cuda()
    on = dict(out=_z(2, 8, 128, dtype=BF).cuda(), q=_z(2, 8, 128, dtype=BF).cuda(), bt=_z(2, 4).cuda(), lens=_z(2).cuda(),
              cu=_z(2 if call is _prefix else 3).cuda(), pre=_z(1).cuda())
    with pytest.raises(pkv.PkvError, match="raw pointer"):
        call(_desc(B.PKV_BF16), cache, cache, ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda").data_ptr(), **on)
