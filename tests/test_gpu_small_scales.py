"""Queries and key scales so small that the scores' factor is below what fp32 holds: every key weighs the same.  Against
attention in 64 bits; bounds in attention_ref.py."""
import pytest
import torch

from attention_ref import check
from test_gpu_cross import Batch as Cross
from test_gpu_prefix import Batch as Prefix

pytestmark = pytest.mark.gpu


def _small(b, k_scale, scale):
    """The same batch under another key scale and softmax scale; some rows of q are zero."""
    b.q[::2] = 0
    b.ks, b.scale = k_scale, scale
    b.device()
    b.desc.k_scale = k_scale
    return b


@pytest.mark.parametrize("kv,k_scale,scale", [("fp8", 2.0 ** -40, 0.09), ("fp8", 2.0 ** -18, 0.09), ("fp8", 1.0, 1e-30),
                                              ("int8", 1e-30, 1e-20), ("int8", 1e-20, 1e-20), ("bf16", 1.0, 1e-40)])
def test_cross_attention(kv, k_scale, scale):
    b = _small(Cross([5, 1, 200, 2], [70, 1, 129, 700], 2, 4, 16, kv, seed=1), k_scale, scale)
    b.run()
    b.verify(f"{kv} {k_scale} {scale}")
    assert int(b.err) == 0


@pytest.mark.parametrize("kv,k_scale,scale", [("fp8", 2.0 ** -40, 0.09), ("fp8", 2.0 ** -18, 0.09),
                                              ("int8", 1e-30, 1e-20), ("bf16", 1.0, 1e-40)])
def test_shared_prefixes(kv, k_scale, scale):
    b = _small(Prefix([(48, [1, 17, 0, 300]), (80, [5, 9])], 2, 4, 16, kv, seed=2), k_scale, scale)
    out = b.run()
    torch.cuda.synchronize()
    assert int(b.err) == 0
    check(out, *b.reference(), f"{kv} {k_scale} {scale}")
