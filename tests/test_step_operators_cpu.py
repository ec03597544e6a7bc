"""Step planning, shared-prefix decode and cross attention without a GPU: what the host refuses before any device work."""
import ctypes

import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B
from paged_kv_cache_71_gb300.block_manager import SequenceTables


def _desc(**kw):
    d = dict(num_blocks=16, block_size=16, num_kv_heads=8, head_dim=128, dtype=B.PKV_BF16, k_scale=1.0, v_scale=1.0)
    d.update(kw)
    return B.CacheDesc(**d)


def _extend(**o):
    a = dict(bt=16, mb=4, past=16, new=16, n=2, S=16, free=16, count=16, nb=8, lens=16, out=16, slots=16, max=8, cu=None,
             qs=None)
    a.update(o)
    return pkv.lib().pkv_extend_sequences(a["bt"], a["mb"], a["past"], a["new"], a["n"], a["S"], a["free"], a["count"],
                                          a["nb"], a["lens"], a["out"], a["slots"], a["max"], a["cu"], a["qs"], None, None)


def _release(**o):
    a = dict(bt=16, mb=4, past=16, done=16, keep=None, n=2, S=16, free=16, count=16, nb=8, lens=16, out=16)
    a.update(o)
    return pkv.lib().pkv_release_sequences(a["bt"], a["mb"], a["past"], a["done"], a["keep"], a["n"], a["S"], a["free"],
                                           a["count"], a["nb"], a["lens"], a["out"], None, None)


@pytest.mark.parametrize("kw,status", [(dict(n=-1), 1), (dict(mb=0), 1), (dict(nb=0), 1), (dict(S=12), 2), (dict(S=64), 2),
                                       (dict(n=8193), 2), (dict(nb=1 << 30), 3), (dict(n=8192, mb=1 << 20), 3),
                                       (dict(n=1, mb=1 << 28), 3), (dict(past=None), 1), (dict(count=None), 1),
                                       (dict(free=None), 1), (dict(lens=18), 1), (dict(out=None), 1)])
def test_step_planning_host_checks(kw, status):
    assert _extend(**kw) == status and pkv.pkv_last_error()
    assert _release(**kw) == status and pkv.pkv_last_error()


def test_step_planning_host_checks_of_one_call():
    assert _extend(max=-1) == 1
    assert _extend(max=2 ** 31 - 1) == 3
    assert _extend(slots=None) == 1
    assert _extend(slots=12) == 1
    assert _extend(cu=17) == 1
    assert _extend(qs=18) == 1
    assert _release(done=None) == 1
    assert _release(keep=18) == 1


def _prefix(desc=None, **o):
    a = dict(out=16, q=16, dt=B.PKV_BF16, k=16, v=16, bt=16, mb=4, cl=16, n=2, Hq=32, scale=0.1, cu=16, pre=16, ng=1,
             ws=16, wsb=1 << 30)
    a.update(o)
    d = desc or _desc()
    return pkv.lib().pkv_paged_attention_decode_prefix(
        a["out"], a["q"], a["dt"], a["k"], a["v"], ctypes.byref(d), a["bt"], a["mb"], a["cl"], a["n"], a["Hq"], a["scale"],
        a["cu"], a["pre"], a["ng"], a["ws"], a["wsb"], None, None)


def test_prefix_decode_host_checks():
    assert _prefix(Hq=30) == 1
    assert _prefix(Hq=24) == 2                        # G = 3
    assert _prefix(Hq=8 * 16) == 2                    # G = 16
    assert _prefix(dt=B.PKV_F32) == 2
    assert _prefix(desc=_desc(dtype=B.PKV_F32)) == 2
    assert _prefix(desc=_desc(head_dim=64)) == 2
    assert _prefix(desc=_desc(block_size=4)) == 2
    assert _prefix(desc=_desc(block_size=12)) == 2
    assert _prefix(n=-1) == 1
    assert _prefix(n=8193) == 2
    assert _prefix(ng=2049) == 2
    assert _prefix(ng=0) == 1                         # every sequence belongs to a group
    assert _prefix(n=8192, mb=1 << 16) == 3
    assert _prefix(desc=_desc(num_kv_heads=1), Hq=8, n=1, mb=1 << 28) == 3
    assert _prefix(scale=0.0) == 1
    assert _prefix(scale=float("nan")) == 1
    assert _prefix(scale=-1.0) == 1
    assert _prefix(cu=None) == 1
    assert _prefix(pre=18) == 1
    assert _prefix(q=24) == 1
    assert _prefix(n=0, ng=0) == 0                    # an empty batch is a no-op
    size = ctypes.c_size_t(0)
    f = pkv.lib().pkv_paged_attention_decode_prefix_workspace_size
    assert f(ctypes.byref(_desc()), -1, 32, ctypes.byref(size)) == 1
    assert f(ctypes.byref(_desc()), 4, 30, ctypes.byref(size)) == 1
    assert f(ctypes.byref(_desc()), 4, 32, None) == 1


def _cross(desc=None, **o):
    a = dict(out=16, q=16, dt=B.PKV_BF16, nq=4, cu=16, kl=16, k=16, v=16, bt=16, mb=4, n=2, Hq=32, scale=0.1, ws=16,
             wsb=1 << 30)
    a.update(o)
    d = desc or _desc()
    return pkv.lib().pkv_paged_cross_attention(a["out"], a["q"], a["dt"], a["nq"], a["cu"], a["kl"], a["k"], a["v"],
                                               ctypes.byref(d), a["bt"], a["mb"], a["n"], a["Hq"], a["scale"], a["ws"],
                                               a["wsb"], None, None)


def test_cross_attention_host_checks():
    assert _cross(Hq=30) == 1
    assert _cross(Hq=24) == 2                         # G = 3 does not divide 128
    assert _cross(Hq=8 * 256) == 2
    assert _cross(dt=B.PKV_F32) == 2
    assert _cross(desc=_desc(dtype=B.PKV_F32)) == 2
    assert _cross(desc=_desc(head_dim=64)) == 2
    assert _cross(desc=_desc(block_size=4)) == 2
    assert _cross(nq=-1) == 1
    assert _cross(n=2049) == 2
    assert _cross(n=2048, mb=1 << 21) == 3
    assert _cross(scale=-1.0) == 1
    assert _cross(kl=None) == 1
    assert _cross(cu=18) == 1
    assert _cross(out=8) == 1
    assert _cross(nq=0) == 0
    assert _cross(n=0, nq=0) == 0
    assert _cross(cu=None) == 1                       # one token a sequence: as many tokens as sequences
    assert _cross(cu=None, nq=2, Hq=24) == 2          # and the decode's own checks
    assert _cross(cu=None, nq=0, n=0) == 0
    size = ctypes.c_size_t(0)
    f = pkv.lib().pkv_paged_cross_attention_workspace_size
    assert f(ctypes.byref(_desc()), -1, 2, 32, ctypes.byref(size)) == 1
    assert f(ctypes.byref(_desc()), 4, 2, 30, ctypes.byref(size)) == 1
    assert f(ctypes.byref(_desc()), 4, 2, 32, None) == 1


def _z(*shape, dtype=torch.int32):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("kw,text", [
    (dict(past=_z(2, dtype=torch.int64)), "dtype"), (dict(new=_z(3)), "shape"), (dict(bt=_z(4, 2).t()), "contiguous"),
    (dict(slots=_z(8)), "dtype"), (dict(cu=_z(2)), "shape"), (dict(count=_z(2)), "shape"), (dict(), "CUDA"),
])
def test_the_binding_refuses_tensors_that_do_not_fit_extend(kw, text):
    a = dict(bt=_z(2, 4), past=_z(2), new=_z(2), free=_z(8), count=_z(1), lens=_z(2), out=_z(1),
             slots=_z(8, dtype=torch.int64), cu=None)
    a.update(kw)
    if text == "CUDA" and torch.cuda.is_available():
        pytest.skip("for a machine without a device")
    with pytest.raises((pkv.PkvError, RuntimeError), match=text):
        pkv.pkv_extend_sequences(a["bt"], a["past"], a["new"], 16, a["free"], a["count"], a["lens"], a["out"], a["slots"],
                                 a["cu"])


def test_the_binding_refuses_tensors_that_do_not_fit_the_attention_calls():
    bf = torch.bfloat16
    desc = _desc(num_blocks=4, num_kv_heads=2)
    cache, q = _z(4, 16, 2, 128, dtype=bf), _z(2, 8, 128, dtype=bf)

    def prefix(out=q, qq=q, k=cache, v=cache, bt=_z(2, 4), lens=_z(2), cu=_z(2), pre=_z(1)):
        pkv.pkv_paged_attention_decode_prefix(out, qq, k, v, desc, bt, lens, cu, pre, 0.1)

    def cross(out=q, qq=q, cu=_z(3), lens=_z(2), k=cache, v=cache, bt=_z(2, 4)):
        pkv.pkv_paged_cross_attention(out, qq, cu, lens, k, v, desc, bt, 0.1)

    for f in (prefix, cross):
        for kw, text in ((dict(out=q.float()), "dtype"), (dict(out=_z(2, 8, 64, dtype=bf)), "shape"),
                         (dict(qq=_z(8, 2, 128, dtype=bf).transpose(0, 1)), "contiguous"),
                         (dict(k=_z(5, 16, 2, 128, dtype=bf)), "shape"), (dict(v=cache.to(torch.int8)), "dtype"),
                         (dict(bt=_z(3, 4)), "shape"), (dict(lens=_z(2, dtype=torch.int64)), "dtype"),
                         (dict(cu=_z(5)), "shape")):
            with pytest.raises(pkv.PkvError, match=text):
                f(**kw)


def test_the_calls_fail_loudly_without_the_library(monkeypatch, tmp_path):
    monkeypatch.setattr(B, "_lib", None)
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "libpkv.so"))
    with pytest.raises(RuntimeError, match="not built"):
        pkv.pkv_extend_sequences(_z(2, 4), _z(2), _z(2), 16, _z(8), _z(1), _z(2), _z(1), _z(8, dtype=torch.int64))
    with pytest.raises(RuntimeError, match="not built"):
        pkv.pkv_paged_cross_attention_workspace_size(_desc(), 4, 2, 32)


def _tables(lengths, forks=()):
    tabs = SequenceTables(64, 4)
    for sid, n in lengths.items():
        tabs.prefill(sid, n)
    for parent, child, own in forks:
        tabs.fork(parent, child)
        for _ in range(own):
            tabs.next_slot(child)
    return tabs


def test_prefix_groups_of_the_block_manager():
    """Forks of two sequences beside sequences of their own; the partly filled block is no one's prefix."""
    tabs = _tables({"a": 10, "b": 9, "c": 3}, [("a", "a1", 5), ("a", "a2", 0), ("b", "b1", 2)])
    cu, pre = tabs.prefix_groups(["a", "a1", "a2", "b", "b1", "c"])
    assert cu.tolist() == [0, 3, 5, 6] and pre.tolist() == [8, 8, 0]
    assert cu.dtype == pre.dtype == "int32"
    cu, pre = tabs.prefix_groups(["c", "a", "b", "a1"])      # apart from one another they share nothing
    assert cu.tolist() == [0, 1, 2, 3, 4] and pre.tolist() == [0, 0, 0, 0]
    cu, pre = tabs.prefix_groups([])
    assert cu.tolist() == [0] and pre.tolist() == []


def test_prefix_groups_keep_the_larger_saving():
    """Three sequences over 5 blocks save 10 block reads; a fourth over 1 block would leave 3, over 4 blocks 12."""
    tabs = _tables({"root": 4})
    tabs.fork("root", "long")
    for _ in range(16):
        tabs.next_slot("long")
    for child in ("x", "y"):
        tabs.fork("long", child)
    tabs.fork("root", "short")
    for _ in range(16):
        tabs.next_slot("short")
    cu, pre = tabs.prefix_groups(["long", "x", "y", "short"])
    assert cu.tolist() == [0, 3, 4] and pre.tolist() == [20, 0]
    tabs = _tables({"root": 16})
    for child, own in (("x", 4), ("z", 0)):
        tabs.fork("root", child)
        for _ in range(own):
            tabs.next_slot(child)
    tabs.fork("x", "y")
    cu, pre = tabs.prefix_groups(["x", "y", "root", "z"])    # 5 blocks, 5 blocks, then 4 of all three and of all four
    assert cu.tolist() == [0, 4] and pre.tolist() == [16]


def test_workspaces_and_error_words_must_be_where_the_tensors_are():
    assert B._extra(None, 0) and B._extra(4096, 0) and B._extra(_z(1), -1)
    assert not B._extra(_z(1), 0) and not B._extra(_z(1), -2)
    for name, kw in (("device_error", dict(device_error=_z(1))), ("workspace", dict(workspace=_z(16)))):
        with pytest.raises(pkv.PkvError, match=name):
            B._refuse("call", 0, **kw)
