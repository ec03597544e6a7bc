"""Unmasked attention in 64 bits over paged K/V, with a bound on what the kernels' roundings can add up to.

For one query row with weights w_t = exp(s_t - max s) / sum and A = sum_t w_t |v_t| (per head dim), an output computed
with fp32 sums, the softmax weights rounded to a type of half-step u (relative) before P.V, and rounded to bf16 at the
end (half-step 2^-8) is off by at most

    A * (u + 2^-8 + 2 d) + e,        u = 2^-8 bf16 weights, 2^-11 f16 weights, 2^-8 + 2^-11 two E4M3 parts of an f16

* d bounds the error of a score: 130 roundings of 2^-24 on sums of at most scale * sum_d |q_d| (|k_d| + b), b = 1152
  code steps for INT8 keys, which the decode multiplies in the biased form 1152 + code; plus 2^-18 of the row's largest
  |q| for FP8 prefixes (the query rows' two E4M3 parts).  A relative error d of a weight moves numerator and
  denominator, hence 2 d.
* e, for two E4M3 parts: each weight is also off by up to 2^-10 (half a subnormal step) where the largest is at least
  2^4, so e = 2^-14 * sum_t |v_t| / sum_t exp(s_t - max s).
* 2^-12 A covers exp2's and the joins' fp32 roundings and f16's subnormal weights (2^-25 each).
"""
from __future__ import annotations

import torch

SCALE = {"bf16": 1.0, "fp8": 1.0 / 64, "int8": 1.0 / 32}
DTYPE = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


def make_cache(gen, shape, kv):
    x = torch.randn(shape, generator=gen)
    if kv == "bf16":
        return x.to(torch.bfloat16)
    x = x / SCALE[kv]
    return (x.clamp(-448, 448) if kv == "fp8" else x.round().clamp(-127, 127)).to(DTYPE[kv])


def gather(cache, table, length):
    """Tokens [0, length) of a table row, in 64 bits: [length][Hkv][D] (codes, unscaled)."""
    S = cache.shape[1]
    blocks = cache.view(torch.uint8)[table[: -(-length // S)].long()].view(cache.dtype)  # raw bytes index in every type
    return blocks.double().reshape(-1, *cache.shape[2:])[:length]


def attend(q, k, v, scale, kv, k_scale, v_scale, tile):
    """q [rows][Hq][D] bf16 against codes k, v [L][Hkv][D]; k_scale, v_scale floats or [Hkv] tensors; tile: the tensor-core
    tile's roundings (prefixes, cross attention), else the decode's.  Returns (out, bound), [rows][Hq][D] in 64 bits."""
    rows, Hq, D = q.shape
    L, Hkv, _ = k.shape
    if L == 0:
        return torch.zeros(rows, Hq, D, dtype=torch.float64), torch.zeros(rows, Hq, D, dtype=torch.float64)
    G = Hq // Hkv
    ks = torch.as_tensor(k_scale, dtype=torch.float64).expand(Hkv)
    vs = torch.as_tensor(v_scale, dtype=torch.float64).expand(Hkv)
    qd = q.double().reshape(rows, Hkv, G, D)
    kd, vd = k * ks[None, :, None], v * vs[None, :, None]
    s = torch.einsum("nhgd,thd->nhgt", qd, kd) * scale
    e = torch.exp(s - s.amax(-1, keepdim=True))
    l = e.sum(-1, keepdim=True)
    w = e / l
    out = torch.einsum("nhgt,thd->nhgd", w, vd)
    A = torch.einsum("nhgt,thd->nhgd", w, vd.abs())
    bias = 1152.0 * ks if kv == "int8" else torch.zeros(Hkv, dtype=torch.float64)
    d = torch.einsum("nhgd,thd->nhgt", qd.abs(), kd.abs() + bias[None, :, None]).amax(-1, keepdim=True)
    d = d * scale * 130 * 2.0 ** -24
    extra = 0.0
    u = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
    if kv == "fp8" and tile:
        u = 2.0 ** -8 + 2.0 ** -11
        kmax = kd.abs().sum(-1).amax(0)  # [Hkv] largest sum_d |k_d|
        d = d + 2.0 ** -18 * qd.abs().amax(-1, keepdim=True) * kmax[None, :, None, None] * scale
        extra = 2.0 ** -14 * vd.abs().sum(0)[None, :, None, :] / l
    bound = A * (u + 2.0 ** -8 + 2 * d + 2.0 ** -12) + extra
    return out.reshape(rows, Hq, D), bound.reshape(rows, Hq, D)


def check(got, ref, bound, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: non-finite output"
    over = (got - ref).abs() - bound
    assert (over <= 0).all(), (f"{what}: {int((over > 0).sum())} of {over.numel()} past the bound, worst by "
                               f"{float(over.max()):.3e} at {tuple(int(i) for i in torch.unravel_index(over.argmax(), over.shape))}")
