"""Frequencies scaled as YaRN does (rotary_frequencies), against a ramp written out pair by pair."""
import math

import numpy as np
import pytest

import paged_kv_cache_71_gb300 as pkv


def _yarn(rot_dim, base, factor, length, fast, slow):
    def pair(turns):  # base^(-2 i / rot_dim) length / (2 pi) = turns, for i
        return rot_dim / 2 * math.log(length / (2 * math.pi * turns), base)

    lo, hi = max(0, math.floor(pair(fast))), math.ceil(pair(slow))
    out = []
    for i in range(rot_dim // 2):
        f = base ** (-2 * i / rot_dim)
        if i >= hi and i > lo or hi < 0:
            w = 1.0  # turns `slow` times or less often
        elif i <= lo:
            w = 0.0  # `fast` times or more often
        else:
            w = (i - lo) / (hi - lo)
        out.append((1 - w) * f + w * f / factor)
    return np.array(out)


@pytest.mark.parametrize("rot_dim", [8, 64, 128])
@pytest.mark.parametrize("base,length", [(10000.0, 4096), (10000.0, 32768), (10000.0, 65536), (10000.0, 131072), (10000.0, 1 << 20),
                                         (500000.0, 8192), (500000.0, 1 << 22), (150000.0, 4096), (10.0, 1000), (10000.0, 64),
                                         (10000.0, 4)])
@pytest.mark.parametrize("factor", [1.0, 4.0, 40.0])
def test_yarn_at_lengths_of_all_sizes(rot_dim, base, length, factor):
    """Lengths above 2 pi base, where the last pair turns more than beta_slow times and the ramp ends behind it; below 2 pi,
    where no pair turns once.  The tolerance: rounding to fp32 (2^-24), and 64-bit roundings."""
    f, s = pkv.rotary_frequencies(rot_dim, base, "yarn", factor, length)
    want = _yarn(rot_dim, base, factor, length, 32.0, 1.0)
    assert np.allclose(f, want, rtol=2.0 ** -23, atol=0)
    assert math.isclose(s, 0.1 * math.log(factor) + 1.0)


def test_yarn_with_other_turns():
    for fast, slow in ((64.0, 2.0), (33.0, 32.0), (100.0, 0.5), (5000.0, 1000.0)):
        f, _ = pkv.rotary_frequencies(64, 10000.0, "yarn", 8.0, 2048, beta_fast=fast, beta_slow=slow)
        assert np.allclose(f, _yarn(64, 10000.0, 8.0, 2048, fast, slow), rtol=2.0 ** -23, atol=0)


def test_yarn_leaves_every_pair_that_turns_beta_fast_times():
    f, _ = pkv.rotary_frequencies(64, 10000.0, "yarn", 16.0, 1 << 22)
    assert f.tolist() == pkv.rotary_frequencies(64, 10000.0)[0].tolist()
