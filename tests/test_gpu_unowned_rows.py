"""Query rows that no chunk owns (padding before the first and behind the last): their q may hold anything, they raise no error
and stay as they are, in the varlen prefill, the mixed step and cross attention over one-byte caches.  Bounds in
attention_ref.py."""
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B

from attention_ref import attend, check, gather
from test_gpu_cross import Batch

pytestmark = pytest.mark.gpu


def _case(kv, value, lead):
    b = Batch([1, 1, 40, 3, 70], [33, 20, 100, 3, 200], 2, 4, 16, kv, seed=90, lead=lead, tail=37)
    b.q[:lead] = b.q[b.cu[-1]:] = value
    return b.device()


def _call(b, call):
    starts = b.dl - torch.diff(b.dcu)
    if call == "cross":
        b.run()
    elif call == "varlen":
        pkv.pkv_paged_prefill_varlen(b.out, b.dq, b.dcu, starts, b.dl, b.dk, b.dv, b.desc, b.dt, b.scale, b.err)
    else:
        ws = torch.empty(pkv.pkv_paged_attention_mixed_workspace_size(b.desc, 2, b.Hq), dtype=torch.uint8, device="cuda")
        pkv.pkv_paged_attention_mixed(b.out, b.dq, b.dcu, starts, b.dl, b.dk, b.dv, b.desc, b.dt, 2, b.scale, ws, b.err)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("call", ["cross", "varlen", "mixed"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e30])
def test_padding_rows_may_hold_anything(kv, call, value):
    b = _case(kv, value, 0 if call == "mixed" else 3)
    _call(b, call)
    assert int(b.err) == 0
    assert (b.out[:b.cu[0]] == 7).all() and (b.out[b.cu[-1]:] == 7).all()
    for s in range(b.n):
        n = b.cu[s + 1] - b.cu[s]
        for i in range(0, n, 13):
            keys = b.lens[s] if call == "cross" else b.lens[s] - n + i + 1
            k, v = gather(b.k, b.tables[s], keys), gather(b.v, b.tables[s], keys)
            row = b.cu[s] + i
            # (the mixed step's decode tokens round like the decode: the looser of the two bounds holds for either)
            ref, bound = attend(b.q[row:row + 1], k, v, b.scale, kv, b.ks, b.vs, True)
            if call == "mixed":
                bound = torch.maximum(bound, attend(b.q[row:row + 1], k, v, b.scale, kv, b.ks, b.vs, False)[1])
            check(b.out[row:row + 1], ref, bound, f"{kv} {call} sequence {s} token {i}")


@pytest.mark.parametrize("kv", ["fp8", "int8"])
@pytest.mark.parametrize("call", ["cross", "varlen", "mixed"])
@pytest.mark.parametrize("row", [2, 41, 44, 114])
def test_rows_of_a_chunk_are_still_reported(kv, call, row):
    """The first and last tokens of chunks, in either query tile."""
    b = _case(kv, 0.0, 0)
    b.dq[row, 7, 100] = float("inf")
    _call(b, call)
    assert int(b.err) == B.DEVERR_Q_RANGE
