"""Speculative decoding without a GPU: masks and rotary frequencies made on the host, and what the new calls refuse."""
import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B

BF, FP8, I8 = torch.bfloat16, torch.float8_e4m3fn, torch.int8


def _z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


def _desc(dtype=B.PKV_BF16, **kw):
    d = dict(num_blocks=4, block_size=16, num_kv_heads=2, head_dim=128, dtype=dtype, k_scale=1.0, v_scale=1.0)
    d.update(kw)
    return B.CacheDesc(**d)


# ------------------------------------------------------------------ masks and frequencies

def test_masks_of_a_small_tree():
    #        0
    #      1   2
    #     3 4   5
    masks, depths = pkv.draft_tree_masks([-1, 0, 0, 1, 1, 2])
    assert masks.dtype == np.int64 and masks[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10011, 0b100101]
    assert depths.tolist() == [0, 1, 1, 2, 2, 2]


def test_masks_of_long_runs_forests_and_none():
    masks, depths = pkv.draft_tree_masks(list(range(-1, 129)))  # a chain of 130
    assert masks.shape == (130, 3) and depths.tolist() == list(range(130))
    bits = [sum((int(w) & (1 << 64) - 1) << 64 * i for i, w in enumerate(row)) for row in masks]
    assert bits == [(1 << i + 1) - 1 for i in range(130)]
    masks, depths = pkv.draft_tree_masks([-1] * 70, words=4)
    assert masks.shape == (70, 4) and depths.tolist() == [0] * 70
    assert [int(m[i // 64]) & (1 << 64) - 1 for i, m in enumerate(masks)] == [1 << i % 64 for i in range(70)]
    assert pkv.draft_tree_masks([])[0].shape == (0, 1)


@pytest.mark.parametrize("parents,words", [([0], None), ([-1, 1], None), ([-2], None), ([-1, 0, 5], None), ([-1] * 65, 1)])
def test_masks_refuse(parents, words):
    with pytest.raises(ValueError):
        pkv.draft_tree_masks(parents, words)


def test_plain_and_interpolated_frequencies():
    f, s = pkv.rotary_frequencies(128, 500000.0)
    assert f.dtype == np.float32 and s == 1.0 and f.shape == (64,)
    assert f.tolist() == [np.float32(500000.0 ** (-2 * i / 128)) for i in range(64)]
    g, s = pkv.rotary_frequencies(128, 500000.0, "linear", 8.0)
    assert s == 1.0 and g.tolist() == [np.float32(500000.0 ** (-2 * i / 128) / 8) for i in range(64)]


def test_ntk_keeps_the_fastest_and_stretches_the_slowest():
    f, _ = pkv.rotary_frequencies(64)
    g, s = pkv.rotary_frequencies(64, scaling="ntk", factor=4.0)
    assert s == 1.0 and g[0] == f[0] == 1.0 and math.isclose(float(g[-1]), float(f[-1]) / 4, rel_tol=1e-6)


def test_llama3_by_wavelength():
    L, lo, hi, fac = 8192, 1.0, 4.0, 8.0
    f = [500000.0 ** (-2 * i / 128) for i in range(64)]
    g, s = pkv.rotary_frequencies(128, 500000.0, "llama3", fac, L, lo, hi)
    assert s == 1.0
    for x, y in zip(f, g.tolist()):
        wave = 2 * math.pi / x
        if wave < L / hi:
            want = x
        elif wave > L / lo:
            want = x / fac
        else:
            w = (L / wave - lo) / (hi - lo)
            want = (1 - w) * x / fac + w * x
        assert math.isclose(y, want, rel_tol=2.0 ** -23)
    kinds = [2 * math.pi / x < L / hi for x in f], [2 * math.pi / x > L / lo for x in f]
    assert any(kinds[0]) and any(kinds[1]) and not all(a or b for a, b in zip(*kinds))


def test_yarn_ramp_and_factor():
    f, _ = pkv.rotary_frequencies(128, 10000.0)
    g, s = pkv.rotary_frequencies(128, 10000.0, "yarn", 16.0, 4096)
    assert math.isclose(s, 0.1 * math.log(16.0) + 1)
    ratio = g.astype(np.float64) / f
    turns = 4096 * f / (2 * np.pi)
    assert np.allclose(ratio[turns > 33], 1.0, rtol=1e-6) and np.allclose(ratio[turns < 0.9], 1 / 16, rtol=1e-6)
    assert (np.diff(ratio) <= 1e-7).all() and ((ratio > 0.07) & (ratio < 0.99)).any()
    assert pkv.rotary_frequencies(128, scaling="yarn", factor=1.0)[1] == 1.0


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, base=1.0), dict(rot_dim=64, factor=0.5),
                                dict(rot_dim=64, scaling="longest"), dict(rot_dim=2, scaling="ntk", factor=2.0),
                                dict(rot_dim=64, scaling="llama3", low_freq_factor=4.0),
                                dict(rot_dim=64, scaling="yarn", beta_fast=1.0), dict(rot_dim=64, base=float("nan"))])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        pkv.rotary_frequencies(**kw)


# ------------------------------------------------------------------ the C entry points' checks

PTR = ctypes.c_void_p(1 << 20)  # aligned and never dereferenced: the checks come first
ODD = ctypes.c_void_p((1 << 20) + 4)


def _tree(q_dtype=B.PKV_BF16, tokens=8, cu=PTR, lens=PTR, mask=PTR, words=1, cache=PTR, desc=None, tables=PTR, width=4, n=2, heads=8,
          scale=0.1, ws=None, out=PTR, q=PTR):
    return pkv.lib().pkv_paged_attention_tree(out, q, q_dtype, tokens, cu, lens, mask, words, cache, cache, ctypes.byref(desc or _desc()),
                                              tables, width, n, heads, scale, ws, 0, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(words=0), 1), (dict(mask=None, words=1), 1), (dict(mask=ODD), 1), (dict(mask=None, words=-1), 1), (dict(q_dtype=B.PKV_F32), 2),
    (dict(desc=_desc(head_dim=64)), 2), (dict(desc=_desc(block_size=4)), 2), (dict(desc=_desc(dtype=B.PKV_F32)), 2), (dict(heads=7), 1),
    (dict(heads=6), 2), (dict(n=2049), 2), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(tokens=-1), 1), (dict(width=0), 1),
    (dict(cu=None), 1), (dict(lens=None), 1), (dict(out=ODD), 1), (dict(tables=None), 1), (dict(width=1 << 30), 3),
])
def test_tree_attention_checks(kw, status):
    assert _tree(**kw) == status, pkv.pkv_last_error()
    assert pkv.pkv_last_error()


def test_nothing_to_do_is_done():
    assert _tree(tokens=0) == 0 and _tree(n=0) == 0
    assert _rope(tokens=0) == 0 and _rope(q=None, q_out=None, heads=0, k=None, v=None) == 0
    assert _commit(n=0) == 0


def test_tree_workspace_size_checks():
    f, out = pkv.lib().pkv_paged_attention_tree_workspace_size, ctypes.c_size_t(0)
    assert f(ctypes.byref(_desc()), 8, 2, 7, ctypes.byref(out)) == 1 and f(ctypes.byref(_desc()), -1, 2, 8, ctypes.byref(out)) == 1
    assert f(ctypes.byref(_desc()), 8, 2, 8, None) == 1 and f(None, 8, 2, 8, ctypes.byref(out)) == 1


def _rope(q_out=PTR, q=PTR, k=PTR, v=PTR, src=B.PKV_BF16, strides=(1024, 1024, 256, 256), pos=PTR, slots=PTR, tokens=4, heads=8, inv=PTR,
          rot=128, scale=1.0, cache=PTR, desc=None):
    return pkv.lib().pkv_rope_and_cache(q_out, q, k, v, src, *strides, pos, slots, tokens, heads, inv, rot, 0, scale, cache, cache,
                                        ctypes.byref(desc or _desc()), None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), 2), (dict(rot=136), 2), (dict(rot=12), 2), (dict(rot=72, desc=_desc(head_dim=64)), 2), (dict(src=B.PKV_FP8_E4M3), 2),
    (dict(tokens=-1), 1), (dict(heads=-1), 1), (dict(heads=0), 1), (dict(q=None), 1), (dict(q_out=None), 1), (dict(k=None), 1),
    (dict(v=None), 1), (dict(slots=None), 1), (dict(pos=None), 1), (dict(inv=None), 1), (dict(cache=None), 1), (dict(scale=0.0), 1),
    (dict(scale=float("inf")), 1), (dict(q=ODD), 1), (dict(k=ODD), 1), (dict(slots=ODD), 1), (dict(strides=(1024, 1020, 256, 256)), 1),
    (dict(strides=(1024, 1016, 256, 256)), 1), (dict(strides=(0, 1024, 256, 256)), 1), (dict(strides=(1024, 1024, 248, 256)), 1),
    (dict(strides=(1024, 1024, 256, -256)), 1), (dict(desc=_desc(block_size=5)), 2),
    (dict(heads=1 << 20, strides=(1 << 27, 1 << 27, 256, 256)), 3),
])
def test_rope_checks(kw, status):
    assert _rope(**kw) == status, pkv.pkv_last_error()
    assert pkv.pkv_last_error()


def _commit(ks=(1 << 20, 1 << 21), vs=(1 << 22, 1 << 23), layers=None, tables=PTR, width=4, cu=PTR, past=PTR, ids=PTR, tokens=8, n=2,
            accepted=PTR, lens=ctypes.c_void_p(1 << 19), keep=None, desc=None):
    arr = [None if x is None else (ctypes.c_void_p * max(1, len(x)))(*x) for x in (ks, vs)]
    return pkv.lib().pkv_commit_tree(*arr, len(ks or vs) if layers is None else layers, ctypes.byref(desc or _desc()), tables, width, cu,
                                     past, ids, ids, ids, tokens, n, accepted, PTR, lens, PTR, keep, None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(layers=0), 1), (dict(layers=129), 2), (dict(ks=None), 1), (dict(vs=None), 1), (dict(ks=(1 << 20, 0)), 1),
    (dict(vs=(1 << 20, (1 << 20) + 8)), 1), (dict(tables=None), 1), (dict(width=0), 1), (dict(cu=None), 1), (dict(past=None), 1),
    (dict(ids=None), 1), (dict(accepted=None), 1), (dict(tokens=-1), 1), (dict(n=-1), 1), (dict(n=8193), 2), (dict(lens=PTR), 1),
    (dict(lens=None), 1), (dict(keep=ctypes.c_void_p(3)), 1), (dict(width=1 << 28), 3),
])
def test_commit_checks(kw, status):
    assert _commit(**kw) == status, pkv.pkv_last_error()
    assert pkv.pkv_last_error()


# ------------------------------------------------------------------ the binding's checks

def _btree(**o):
    a = dict(out=_z(2, 8, 128, dtype=BF), q=_z(2, 8, 128, dtype=BF), cu=_z(3), lens=_z(2), mask=_z(2, 1, dtype=torch.int64),
             k=_z(4, 16, 2, 128, dtype=BF), v=_z(4, 16, 2, 128, dtype=BF), desc=_desc(), bt=_z(2, 4))
    a.update(o)
    pkv.pkv_paged_attention_tree(a["out"], a["q"], a["cu"], a["lens"], a["mask"], a["k"], a["v"], a["desc"], a["bt"], 0.1)


@pytest.mark.parametrize("kw,text", [
    (dict(q=_z(16, 128, dtype=BF)), "q has shape"), (dict(bt=_z(8)), "block_tables has shape"), (dict(mask=_z(2, dtype=torch.int64)), "tree_mask has shape"),
    (dict(mask=_z(3, 1, dtype=torch.int64)), "tree_mask has shape"), (dict(mask=_z(2, 0, dtype=torch.int64)), "no words"), (dict(mask=_z(2, 1)), "tree_mask has dtype"),
    (dict(mask=_z(2, 4, dtype=torch.int64)[:, ::2]), "tree_mask must be contiguous"), (dict(cu=_z(2)), "cu_q has shape"),
    (dict(lens=_z(2, dtype=torch.int64)), "kv_lens has dtype"), (dict(k=_z(4, 16, 2, 128, dtype=FP8)), "k_cache has dtype"),
    (dict(desc=_desc(B.PKV_INT8)), "k_cache has dtype"), (dict(out=_z(2, 8, 128)), "out has dtype"), (dict(), "CUDA"),
])
def test_tree_binding_refuses(kw, text):
    with pytest.raises((pkv.PkvError, RuntimeError), match=text):
        _btree(**kw)


def _brope(**o):
    a = dict(q_out=_z(3, 8, 128, dtype=BF), q=_z(3, 8, 128, dtype=BF), k=_z(3, 2, 128, dtype=BF), v=_z(3, 2, 128, dtype=BF), pos=_z(3),
             slots=_z(3, dtype=torch.int64), inv=_z(64, dtype=torch.float32), kc=_z(4, 16, 2, 128, dtype=BF), vc=_z(4, 16, 2, 128, dtype=BF))
    a.update(o)
    pkv.pkv_rope_and_cache(a["q_out"], a["q"], a["k"], a["v"], a["pos"], a["slots"], a["inv"], a["kc"], a["vc"], _desc())


@pytest.mark.parametrize("kw,text", [
    (dict(q=None), "comes with"), (dict(k=None), "comes with"), (dict(q=None, q_out=None, k=None, v=None), "needed"),
    (dict(slots=None), "need slot_mapping"), (dict(q=_z(3, 1024, dtype=BF)), "q has shape"), (dict(q=_z(3, 8, 64, dtype=BF)), "q has shape"),
    (dict(q_out=_z(3, 4, 128, dtype=BF)), "q_out has shape"), (dict(q_out=_z(3, 8, 128)), "q_out has dtype"),
    (dict(k=_z(3, 2, 128, dtype=torch.float32)), "k_new has dtype"), (dict(v=_z(2, 2, 128, dtype=BF)), "v_new has shape"),
    (dict(q=_z(3, 8, 256, dtype=BF)[..., ::2]), "contiguous, separate tokens"), (dict(q=_z(3, 128, 8, dtype=BF).transpose(1, 2)), "separate tokens"),
    (dict(k=_z(1, 2, 128, dtype=BF).expand(3, 2, 128)), "separate tokens"), (dict(pos=_z(3, 1)), "positions has shape"),
    (dict(inv=_z(64, dtype=torch.float64)), "inv_freq has dtype"), (dict(slots=_z(3)), "slot_mapping has dtype"),
    (dict(kc=_z(4, 16, 2, 128, dtype=FP8)), "k_cache has dtype"), (dict(vc=_z(4, 16, 2, 64, dtype=BF)), "v_cache has shape"), (dict(), "CUDA"),
])
def test_rope_binding_refuses(kw, text):
    with pytest.raises((pkv.PkvError, RuntimeError), match=text):
        _brope(**kw)


def test_layer_caches_refuse():
    k = _z(4, 16, 2, 128, dtype=BF)
    for ks, vs in (([], []), ([k], []), ([k], [k, k]), ([k], [_z(4, 16, 2, 64, dtype=BF)]), ([k, k], [k, _z(4, 16, 2, 128, dtype=FP8)]),
                   ([_z(4, 16, 256, dtype=BF)], [k]), ([k.double()], [k.double()]), ([k[:, ::2]], [k[:, ::2]])):
        with pytest.raises(pkv.PkvError):
            pkv.LayerCaches(ks, vs)
    with pytest.raises(pkv.PkvError, match="same memory"):  # every layer's tokens would move twice
        pkv.LayerCaches([k, k], [k.clone(), k.clone()])
    pools = [k.clone() for _ in range(4)]
    layers = pkv.LayerCaches(pools[:2], pools[2:])
    assert layers.num_layers == 2 and layers.desc.num_blocks == 4 and layers.k_pointers[1] == pools[1].data_ptr()


def _bcommit(**o):
    k = _z(4, 16, 2, 128, dtype=BF)
    a = dict(bt=_z(2, 4), cu=_z(3), past=_z(2), parents=_z(9), draft=_z(9), target=_z(9), accepted=_z(9), count=_z(2), lens=_z(2), nxt=_z(2), keep=_z(2))
    a.update(o)
    pkv.pkv_commit_tree(pkv.LayerCaches([k], [k.clone()]), a["bt"], a["cu"], a["past"], a["parents"], a["draft"], a["target"], a["accepted"], a["count"],
                        a["lens"], a["nxt"], a["keep"])


@pytest.mark.parametrize("kw,text", [
    (dict(bt=_z(8)), "block_tables has shape"), (dict(bt=_z(3, 4)), "block_tables has shape"), (dict(cu=_z(2)), "cu_q has shape"),
    (dict(past=_z(2, 1)), "past_lens has shape"), (dict(draft=_z(8)), "draft_tokens has shape"), (dict(target=_z(9, dtype=torch.int64)), "target_tokens has dtype"),
    (dict(accepted=_z(10)), "accepted has shape"), (dict(count=_z(3)), "num_accepted has shape"), (dict(keep=_z(4)[::2]), "keep_blocks must be contiguous"),
    (dict(), "CUDA"),
])
def test_commit_binding_refuses(kw, text):
    with pytest.raises((pkv.PkvError, RuntimeError), match=text):
        _bcommit(**kw)
