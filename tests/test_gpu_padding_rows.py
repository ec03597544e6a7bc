"""Rows of length 0 (finished sequences, padding) in groups with a prefix: their q may hold anything; they are zero and raise
no error, and the other rows are as ever.  Bounds in attention_ref.py."""
import pytest
import torch

from paged_kv_cache_71_gb300 import _binding as B

from attention_ref import check
from test_gpu_prefix import Batch

pytestmark = pytest.mark.gpu

GROUPS = [(64, [3, 20, 7]), (32, [5]), (0, [9, 4]), (96, [1 + i % 5 for i in range(70)])]
PADDING = [0, 2, 5, 6, 40, 75]  # a group's first row among them, and a row without a prefix


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e30])
def test_q_of_padding_rows_may_hold_anything(kv, value):
    b = Batch(GROUPS, 2, 4, 16, kv, seed=80)
    keep = b.q.clone()
    b.q[PADDING] = value
    b.device()
    b.dl[PADDING] = 0
    out = b.run()
    torch.cuda.synchronize()
    assert int(b.err) == 0
    assert (out[PADDING] == 0).all()
    b.q = keep
    rows = [s for s in range(b.B) if s not in PADDING]
    ref, bound = b.reference(rows)
    check(out[rows], ref, bound, f"{kv} beside padding rows of {value}")


@pytest.mark.parametrize("kv", ["fp8", "int8"])
def test_q_of_the_other_rows_is_still_reported(kv):
    b = Batch(GROUPS, 2, 4, 16, kv, seed=81)
    b.q[1, 3, 5] = float("inf")
    b.device()
    b.dl[PADDING] = 0
    b.run()
    torch.cuda.synchronize()
    assert int(b.err) == B.DEVERR_Q_RANGE
