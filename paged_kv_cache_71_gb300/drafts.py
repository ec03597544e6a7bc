"""What a program prepares on the host for the calls of a speculative decoding step: the masks of a draft tree of a fixed
shape (pkv_paged_attention_tree) and the rotary frequencies of a model (pkv_rope_and_cache).

A drafter that grows its trees on the GPU makes the masks there: a token's mask is its parent's with its own bit set.
"""
from __future__ import annotations

import math

import numpy as np


def draft_tree_masks(parents, words: int | None = None) -> tuple[np.ndarray, np.ndarray]:
    """(masks, depths) of one run of drafted tokens: parents[i] < i is the index in the run of the token that token i
    follows, -1 for none.  masks: int64 [tokens][words], bit j of a row: the token sees token j (its ancestors and itself),
    as pkv_paged_attention_tree takes it; words: 64-bit words of a row (default: as many as the run needs).  depths: int32,
    a token's position less the tokens before the run."""
    n = len(parents)
    need = max(1, -(-n // 64))
    words = need if words is None else int(words)
    if words < need:
        raise ValueError(f"{n} tokens need {need} words, {words} given")
    masks, depths = np.zeros((n, words), np.uint64), np.zeros(n, np.int32)
    for i, p in enumerate(parents):
        p = int(p)
        if not -1 <= p < i:
            raise ValueError(f"parents[{i}] is {p}, expected -1 or an earlier token")
        if p >= 0:
            masks[i], depths[i] = masks[p], depths[p] + 1
        masks[i, i // 64] |= np.uint64(1 << (i % 64))
    return masks.view(np.int64), depths


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       original_length: int = 8192, low_freq_factor: float = 1.0, high_freq_factor: float = 4.0,
                       beta_fast: float = 32.0, beta_slow: float = 1.0) -> tuple[np.ndarray, float]:
    """(inv_freq, rope_scale) as pkv_rope_and_cache takes them: fp32 [rot_dim / 2] angles per position, computed in 64 bits,
    and what the rotated elements are multiplied by.  With i-th frequency f_i = base^(-2 i / rot_dim) and s = factor:

    * "none":   f_i
    * "linear": f_i / s (positions interpolated)
    * "ntk":    the frequencies of base * s^(rot_dim / (rot_dim - 2)): the fastest as it is, the slowest f / s
    * "llama3": by wavelength against original_length L: f_i above L / high_freq_factor's frequency, f_i / s below
      L / low_freq_factor's, in between (1 - w) f_i / s + w f_i with w linear in L f_i / (2 pi)
    * "yarn":   f_i for pairs that turn beta_fast times or more within L, f_i / s for those below beta_slow turns, a ramp
      linear in i between the two pairs' indexes (rounded down, 0 at least, and up); rope_scale = 0.1 ln(s) + 1 for s > 1
    """
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim {rot_dim} is not a positive even number")
    if not (base > 1.0 and factor >= 1.0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError(f"base {base} must be above 1 and factor {factor} at least 1")
    if scaling == "ntk":
        if rot_dim <= 2:
            raise ValueError("ntk scaling needs rot_dim > 2")
        base = base * factor ** (rot_dim / (rot_dim - 2))
    half = rot_dim // 2
    i = np.arange(half, dtype=np.float64)
    f = base ** (-i / half)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "llama3":
        if not high_freq_factor > low_freq_factor > 0:
            raise ValueError("llama3 scaling needs high_freq_factor > low_freq_factor > 0")
        w = (original_length * f / (2 * math.pi) - low_freq_factor) / (high_freq_factor - low_freq_factor)
        w = np.clip(w, 0.0, 1.0)
        f = (1 - w) * f / factor + w * f
    elif scaling == "yarn":
        if not beta_fast > beta_slow > 0:
            raise ValueError("yarn scaling needs beta_fast > beta_slow > 0")

        def pair_of(turns):  # the pair (a real number) that turns that often within original_length
            return half * math.log(original_length / (turns * 2 * math.pi)) / math.log(base)

        # (hi may lie behind the last pair, where that one still turns more than beta_slow times, or before the first one)
        hi = math.ceil(pair_of(beta_slow))
        lo = min(max(0, math.floor(pair_of(beta_fast))), hi)
        w = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        f = (1 - w) * f + w * f / factor
        scale = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"scaling {scaling!r}: expected none, linear, ntk, llama3 or yarn")
    return f.astype(np.float32), scale
