"""Attention of drafted tokens in 64 bits over paged K/V, with the bound of attention_ref.py on the kernels' roundings (its
sums taken over the keys that a row sees)."""
from __future__ import annotations

import torch

from attention_ref import SCALE, gather  # noqa: F401  (SCALE for the callers)


def attend_masked(q, k, v, seen, scale, kv, k_scale, v_scale):
    """q [n][Hq][D] bf16 against codes k, v [L][Hkv][D] (64 bits); seen bool [n][L].  Returns (out, bound) [n][Hq][D]."""
    n, Hq, D = q.shape
    L, Hkv, _ = k.shape
    G = Hq // Hkv
    ks = torch.as_tensor(k_scale, dtype=torch.float64).expand(Hkv)
    vs = torch.as_tensor(v_scale, dtype=torch.float64).expand(Hkv)
    qd = q.double().reshape(n, Hkv, G, D)
    mask = seen[:, None, None, :]
    kd, vd = k * ks[None, :, None], v * vs[None, :, None]
    s = torch.einsum("nhgd,thd->nhgt", qd, kd.nan_to_num(0.0, 0.0, 0.0)) * scale
    s = s.masked_fill(~mask, float("-inf"))
    top = s.amax(-1, keepdim=True)
    e = torch.where(mask, torch.exp(s - torch.where(top == float("-inf"), torch.zeros_like(top), top)), torch.zeros_like(s))
    l = e.sum(-1, keepdim=True)
    w = e / torch.where(l == 0, torch.ones_like(l), l)
    vf = vd.nan_to_num(0.0, 0.0, 0.0)
    out = torch.einsum("nhgt,thd->nhgd", w, vf)
    A = torch.einsum("nhgt,thd->nhgd", w, vf.abs())
    d = torch.einsum("nhgd,thd->nhgt", qd.abs(), kd.abs().nan_to_num(0.0, 0.0, 0.0))
    d = d.masked_fill(~mask, 0.0).amax(-1, keepdim=True) * scale * 130 * 2.0 ** -24
    extra = 0.0
    u = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
    if kv == "fp8":
        u = 2.0 ** -8 + 2.0 ** -11
        kmax = kd.abs().nan_to_num(0.0, 0.0, 0.0).sum(-1).amax(0)
        d = d + 2.0 ** -18 * qd.abs().amax(-1, keepdim=True) * kmax[None, :, None, None] * scale
        part = torch.einsum("nt,thd->nhd", seen.double(), vf.abs())[:, :, None, :]
        extra = torch.where(l == 0, torch.zeros_like(part), 2.0 ** -14 * part / torch.where(l == 0, torch.ones_like(l), l))
    bound = A * (u + 2.0 ** -8 + 2 * d + 2.0 ** -12) + extra
    return out.reshape(n, Hq, D), bound.reshape(n, Hq, D)


def seen_keys(n, L, bits):
    """bool [n][L]: all keys before the run, and of its own those of `bits` (whole numbers; None: a chain)."""
    seen = torch.ones(n, L, dtype=torch.bool)
    for i in range(n):
        for j in range(n):
            seen[i, L - n + j] = j <= i if bits is None else bool(bits[i] >> j & 1)
    return seen


def mask_words(bits_of_runs, words):
    """int64 [tokens][words] of the runs' whole numbers."""
    rows = [[(b >> 64 * w) & (1 << 64) - 1 for w in range(words)] for run in bits_of_runs for b in run]
    rows = [[x - (1 << 64) if x >> 63 else x for x in r] for r in rows]
    return torch.tensor(rows, dtype=torch.int64).reshape(-1, words)


def random_tree(r, n):
    """Parents of a tree of n tokens, in breadth-first order."""
    return [-1] + sorted(min(i - 1, int(i * r.random() ** 2)) for i in range(1, n)) if n else []


def ancestors(parents):
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    return bits
