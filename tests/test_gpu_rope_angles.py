"""Angles of pkv_rope_and_cache at every size of position times frequency, against whole-number arithmetic.

The kernel's angle is off by less than 1.51 |p| 2^-64 turns (its fixed-point phase, at most 0.76 * 2^-32 of a turn) and 2^-32
of a turn (the half that is dropped), together 2 pi 1.76 * 2^-32 < 2^-28; then as in test_gpu_rope.py: pi 2^-25 for the
rounding to fp32, 2^-23 for sincospi, three products and sums of 2^-24.  In units of 2^-24 (|x| + |y|):
1.58 + 0.07 + 2 + 3 < 7.
"""
import random
from fractions import Fraction

import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B

pytestmark = pytest.mark.gpu
T, H, D = 48, 2, 128


def _per_radian(bits):
    """floor(2^bits / (2 pi)), within one: pi by Machin's formula, 16 arctan 1/5 - 4 arctan 1/239."""
    one = 1 << bits + 32

    def arctan(n):
        term, total, k = one // n, 0, 1
        while term:
            total += term // k if k % 4 == 1 else -(term // k)
            term //= n * n
            k += 2
        return total

    return (one << bits) // (2 * (16 * arctan(5) - 4 * arctan(239)))


def _turns(p, f, K):
    """p f / (2 pi) less whole turns, in [-1/2, 1/2); f exactly, as the fp32 number it is; K of 256 bits."""
    x = Fraction(p) * Fraction(f)
    t = x.numerator * K // x.denominator & (1 << 256) - 1
    return ((t + (1 << 255) & (1 << 256) - 1) - (1 << 255)) / (1 << 256)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("low,high", [(-20, 0), (0, 10), (10, 16), (16, 24)])
def test_large_frequencies_at_far_positions(low, high, interleaved):
    """Frequencies of 2^low to 2^high of either sign, positions over all of int32."""
    r = random.Random(low)
    inv = torch.tensor([r.choice((-1, 1)) * 2.0 ** r.uniform(low, high) for _ in range(D // 2)], dtype=torch.float32)
    inv[0], inv[1], inv[2] = 2.0 ** high, -(2.0 ** low), 2.0 ** high * (1 - 2.0 ** -24)
    inv = inv.clamp(-(2.0 ** 24 - 1), 2.0 ** 24 - 1)  # (promised below 2^24)
    pos = [2 ** 31 - 1, -2 ** 31, 1, -1, 0, 3 << 29] + [r.choice((-1, 1)) * int(2 ** r.uniform(0, 31)) for _ in range(T - 6)]
    K = _per_radian(256)
    angle = torch.tensor([[_turns(p, float(f), K) for f in inv] for p in pos], dtype=torch.float64) * 2 * torch.pi
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    q = torch.randn(T, H, D, generator=torch.Generator().manual_seed(high))
    out = torch.empty(T, H, D, device="cuda")
    desc = B.CacheDesc(num_blocks=4, block_size=16, num_kv_heads=1, head_dim=D, dtype=B.PKV_BF16, k_scale=1.0, v_scale=1.0)
    pkv.pkv_rope_and_cache(out, q.cuda(), None, None, torch.tensor(pos, dtype=torch.int32, device="cuda"), None, inv.cuda(), None, None,
                           desc, interleaved)
    a, b = (slice(0, D, 2), slice(1, D, 2)) if interleaved else (slice(0, D // 2), slice(D // 2, D))
    x, y, got = q[..., a].double(), q[..., b].double(), out.cpu().double()
    bound = 7 * 2.0 ** -24 * (x.abs() + y.abs())
    for part, ref in ((a, x * cos - y * sin), (b, y * cos + x * sin)):
        over = (got[..., part] - ref).abs() - bound * (1 + 2.0 ** -20) - 2.0 ** -24 * ref.abs()
        assert (over <= 0).all(), f"{int((over > 0).sum())} past the bound, worst by {float(over.max()):.3e}"
