"""Rotary positions on the way into the cache (pkv_rope_and_cache) against the formula in 64 bits.

With a pair (x, y), a = rope_scale: the angle's fraction of a turn is rounded to fp32 (half a step of a half turn, pi 2^-25, plus
2^-32 turns of the fixed-point phase), sincospi is off by at most two steps below one (2^-23), its product with a by 2^-24, and
two products and a sum by 2^-24 each, so before the result's own rounding the error is at most
    (|x| + |y|) a (pi 2^-25 + 2^-29 + 2^-23 + 3 * 2^-24)  <  7 * 2^-24 a (|x| + |y|).
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_71_gb300 as pkv
from paged_kv_cache_71_gb300 import _binding as B

pytestmark = pytest.mark.gpu
SRC = {"f32": torch.float32, "bf16": torch.bfloat16}
DST = {**SRC, "fp8": torch.float8_e4m3fn, "int8": torch.int8}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp8": 2.0 ** -4}


def rotate(x, positions, inv_freq, scale, interleaved):
    """x [T][H][D] in 64 bits -> (rotated, |x| + |y| of each element's pair, 0 where nothing is rotated)."""
    half = inv_freq.numel()
    # the angle as two exact products (a position's 31 bits times 21 and 24 - 21), joined by the addition theorems
    f = inv_freq.double()
    m, e = torch.frexp(f)
    hi = torch.ldexp(torch.round(m * 2 ** 21) / 2 ** 21, e)
    t1, t2 = (torch.outer(positions.double(), x)[:, None, :] for x in (hi, f - hi))
    cos = torch.cos(t1) * torch.cos(t2) - torch.sin(t1) * torch.sin(t2)
    sin = torch.sin(t1) * torch.cos(t2) + torch.cos(t1) * torch.sin(t2)
    out, size = x.double().clone(), torch.zeros_like(x, dtype=torch.float64)
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    p, q = x[..., a].double(), x[..., b].double()
    out[..., a] = scale * (p * cos - q * sin)
    out[..., b] = scale * (q * cos + p * sin)
    size[..., a] = size[..., b] = scale * (p.abs() + q.abs())
    return out, size


def near(got, ref, size, kind, what, scale=1.0):
    """got: values or codes; ref: exact values; scale: of a code (a float or one per head)."""
    err = 7 * 2.0 ** -24 * size
    if kind == "int8":
        s = torch.as_tensor(scale, dtype=torch.float64).reshape(-1, 1)
        ref = torch.maximum(torch.minimum(ref, 127 * s), -127 * s)
        bound = 0.5 * s + err + 127 * s * 2.0 ** -23
        val = got.double() * s
    else:
        s = torch.as_tensor(scale, dtype=torch.float64).reshape(-1, 1)
        u = HALF_STEP[kind]
        if kind == "fp8":
            ref = torch.maximum(torch.minimum(ref, 448 * s), -448 * s)
        bound = u * (ref.abs() + err) + err + (s * 2.0 ** -10 + ref.abs() * 2.0 ** -23 if kind == "fp8" else 0.0)
        val = got.double() * s
    over = (val - ref).abs() - bound
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} past the bound, worst by {float(over.max()):.3e}"


class Call:
    def __init__(self, T, hq, hkv, D, rot, src, dst, seed, interleaved=False, far=4096, scale=1.0, fused=False, pads=0,
                 head_scales=False, S=16, base=10000.0):
        g = torch.Generator().manual_seed(seed)
        self.T, self.hq, self.hkv, self.D, self.src, self.dst, self.inter, self.scale = T, hq, hkv, D, src, dst, interleaved, scale
        self.inv = torch.from_numpy(pkv.rotary_frequencies(rot, base)[0])
        self.pos = torch.randint(0, far, (T,), generator=g).to(torch.int32)
        if fused:
            x = torch.randn(T, hq + 2 * hkv, D, generator=g).to(SRC[src])
            self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
            d = x.cuda()
            self.dq, self.dk, self.dv = d[:, :hq], d[:, hq:hq + hkv], d[:, hq + hkv:]
        else:
            self.q, self.k, self.v = (torch.randn(T, h, D, generator=g).to(SRC[src]) for h in (hq, hkv, hkv))
            self.dq, self.dk, self.dv = self.q.cuda(), self.k.cuda(), self.v.cuda()
        nb = -(-T // S) + 2
        self.slots = torch.randperm(nb * S, generator=g)[:T]
        self.slots[torch.randperm(T, generator=g)[:pads]] = -1
        self.kc = torch.zeros(nb, S, hkv, D, dtype=DST[dst], device="cuda")
        for c in (self.kc,):
            c.view(torch.uint8).fill_(0x3c)
        self.vc = self.kc.clone()
        self.sk = self.sv = {"int8": 1 / 32, "fp8": 0.25}.get(dst, 1.0)
        heads = {}
        if head_scales:
            self.sk = (torch.rand(hkv, generator=g) + 0.5) * self.sk
            self.sv = (torch.rand(hkv, generator=g) + 0.5) * self.sv
            self.keep = self.sk.cuda(), self.sv.cuda()
            heads = dict(k_head_scales=self.keep[0], v_head_scales=self.keep[1])
        self.desc = pkv.CacheDesc.for_cache(self.kc, 1.0 if heads else self.sk, 1.0 if heads else self.sv, **heads)
        self.out = torch.full((T, hq, D), 7.0, dtype=SRC[src], device="cuda")
        self.dp, self.ds, self.di = self.pos.cuda(), self.slots.cuda(), self.inv.cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, stream=None, out=None):
        pkv.pkv_rope_and_cache(self.out if out is None else out, self.dq, self.dk, self.dv, self.dp, self.ds, self.di, self.kc,
                               self.vc, self.desc, self.inter, self.scale, self.err, stream)
        return self

    def verify(self, what, out=None):
        torch.cuda.synchronize()
        live = self.slots >= 0
        out = (self.out if out is None else out).cpu()
        ref, size = rotate(self.q, self.pos, self.inv, self.scale, self.inter)
        near(out[live], ref[live], size[live], self.src, what + ", q")
        flat = self.kc.view(torch.uint8).cpu().reshape(-1, self.hkv, self.D * self.kc.element_size())
        k = flat[self.slots[live]].reshape(-1).view(DST[self.dst]).reshape(-1, self.hkv, self.D)
        ref, size = rotate(self.k, self.pos, self.inv, self.scale, self.inter)
        near(k, ref[live], size[live], self.dst, what + ", k", self.sk)
        untouched = torch.ones(flat.shape[0], dtype=torch.bool)
        untouched[self.slots[live]] = False
        assert (flat[untouched] == 0x3c).all(), what + ": slots of no token"
        # values, and keys that are not rotated: what the plain cache write stores
        kc, vc = torch.zeros_like(self.kc), torch.zeros_like(self.vc)
        for c in (kc, vc):
            c.view(torch.uint8).fill_(0x3c)
        pkv.pkv_reshape_and_cache(self.dk.contiguous(), self.dv.contiguous(), self.ds, kc, vc, self.desc)
        assert torch.equal(vc.view(torch.uint8), self.vc.view(torch.uint8)), what + ": values"
        rot, es = 2 * self.inv.numel(), self.kc.element_size()
        assert torch.equal(kc.view(torch.uint8)[..., rot * es:], self.kc.view(torch.uint8)[..., rot * es:]), what + ": past the rotated part"
        return self


TYPES = [(s, d) for s in ("f32", "bf16") for d in ("f32", "bf16", "fp8", "int8")]


@pytest.mark.parametrize("src,dst", TYPES)
@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (128, 128, True), (128, 24, False), (128, 8, True), (64, 64, False),
                                               (64, 40, True)])
def test_types_layouts_and_parts(src, dst, D, rot, interleaved):
    c = Call(37, 6, 2, D, rot, src, dst, seed=rot, interleaved=interleaved, pads=5, fused=True)
    c.run().verify(f"{src}->{dst} D={D} rot={rot}")
    assert int(c.err) == 0
    assert (c.out[c.slots < 0] == 7).all(), "padding tokens' rows stay"


@pytest.mark.parametrize("T", [1, 2, 3, 151, 1217, 2433, 5003])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (5, 3)])
def test_token_counts(T, hq, hkv):
    Call(T, hq, hkv, 128, 128, "bf16", "bf16", seed=T, fused=T % 2 == 1, pads=T // 10).run().verify(f"T={T}")


@pytest.mark.parametrize("hq,hkv", [(64, 8), (1, 1), (128, 128), (12, 3)])
def test_head_counts(hq, hkv):
    Call(19, hq, hkv, 128, 128, "bf16", "fp8", seed=hq).run().verify(f"{hq}/{hkv}")


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Up to 2^31 - 1 and negative ones: the angle is exact where an fp32 product would be off by many turns."""
    c = Call(64, 4, 2, 128, 128, "f32", "f32", seed=1, interleaved=interleaved, far=2 ** 31 - 1, scale=1.25)
    c.pos[:6] = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 1, 0, 1 << 24], dtype=torch.int32)
    c.dp.copy_(c.pos)
    c.run().verify("far")


def test_position_zero_and_frequencies_of_zero_leave_the_values():
    c = Call(9, 4, 2, 128, 64, "bf16", "bf16", seed=2)
    c.dp.zero_()
    c.run()
    assert torch.equal(c.out, c.dq)
    c.dp.copy_(c.pos)
    c.di.zero_()
    c.out.fill_(7.0)
    c.run()
    assert torch.equal(c.out, c.dq)


def test_frequencies_of_all_sizes():
    """Tiny, subnormal, negative, above one and huge frequencies at small positions."""
    c = Call(32, 2, 1, 64, 32, "f32", "f32", seed=3, far=100)
    vals = [1e-42, -1e-38, 2.0 ** -126, 1e-20, -1e-7, 0.3, -1.0, 1.5, 3.0, -6.25, 100.0, 1234.5, -65536.0, 2.0 ** 23, 8388607.0, 1e-3]
    c.inv = torch.tensor(vals, dtype=torch.float32)
    c.di.copy_(c.inv)
    c.run().verify("frequencies")


def test_frequencies_that_are_not_finite_give_nan():
    c = Call(5, 2, 1, 64, 16, "f32", "f32", seed=4)
    c.di[2], c.di[5] = float("inf"), float("nan")
    c.run()
    bad = torch.isnan(c.out).cpu()
    assert bad[..., [2, 5, 10, 13]].all() and not bad[..., [0, 1, 3, 4, 6, 7, 8, 9, 11, 12, 14, 15]].any() and not bad[..., 16:].any()


def test_in_place_and_inside_a_fused_projection():
    c = Call(77, 8, 2, 128, 128, "bf16", "bf16", seed=5, fused=True)
    k, v = c.dk.clone(), c.dv.clone()
    c.run(out=c.dq)
    c.verify("in place", out=c.dq)
    assert torch.equal(c.dk, k) and torch.equal(c.dv, v)


def test_queries_alone_and_keys_alone():
    c = Call(21, 8, 2, 128, 96, "bf16", "fp8", seed=6, pads=4)
    whole = Call(21, 8, 2, 128, 96, "bf16", "fp8", seed=6, pads=4).run()
    pkv.pkv_rope_and_cache(None, None, c.dk, c.dv, c.dp, c.ds, c.di, c.kc, c.vc, c.desc)
    assert (c.out == 7).all()
    pkv.pkv_rope_and_cache(c.out, c.dq, None, None, c.dp, c.ds, c.di, None, None, c.desc)
    for a, b in ((c.out, whole.out), (c.kc.view(torch.uint8), whole.kc.view(torch.uint8)), (c.vc.view(torch.uint8), whole.vc.view(torch.uint8))):
        assert torch.equal(a, b)
    c.out.fill_(7.0)  # without slots no token is padding
    pkv.pkv_rope_and_cache(c.out, c.dq, None, None, c.dp, None, c.di, None, None, c.desc)
    ref, size = rotate(c.q, c.pos, c.inv, 1.0, False)
    near(c.out.cpu(), ref, size, "bf16", "without slots")


@pytest.mark.parametrize("dst", ["fp8", "int8"])
def test_scales_per_head_and_saturation(dst):
    c = Call(40, 4, 3, 128, 128, "f32", dst, seed=7, head_scales=True, scale=30.0)
    c.run().verify(f"{dst} head scales")


@pytest.mark.parametrize("dst", ["fp8", "int8"])
@pytest.mark.parametrize("src", ["f32", "bf16"])
def test_codes_under_scales_of_all_sizes(src, dst):
    """At position 0 keys are not turned: codes as the plain cache write makes them, whatever the scale (powers of two are
    multiplied by their inverse, others divide).  Keys are compared as numbers: of a pair (-0, y) with y < 0 the turned first
    element is -0 * 1 - y * 0 = -0 - (-0) = +0; and only where both of a pair are finite: infinity * 0 is no number."""
    c = Call(33, 4, 2, 128, 128, src, dst, seed=11)
    c.dp.zero_()
    for scale in (2.0 ** -149, 2.0 ** -127, 2.0 ** -126, 2.0 ** -30, 0.3, 0.5, 1.0, 3.0, 2.0 ** 40, 2.0 ** 126, 2.0 ** 127, 1e38):
        desc = pkv.CacheDesc.for_cache(c.kc, scale, scale)
        kc, vc = torch.zeros_like(c.kc), torch.zeros_like(c.vc)
        kd, vd = torch.zeros_like(c.kc), torch.zeros_like(c.vc)
        x = torch.cat([c.dk[:16], c.dk[16:] * scale * 7]).to(c.dk.dtype)
        pkv.pkv_reshape_and_cache(x, c.dv, c.ds, kc, vc, desc)
        pkv.pkv_rope_and_cache(None, None, x, c.dv, c.dp, c.ds, c.di, kd, vd, desc)
        assert torch.equal(vc.view(torch.uint8), vd.view(torch.uint8)), scale
        finite = torch.isfinite(x) & torch.isfinite(x.roll(64, -1))
        ka, kb = (t.float().reshape(-1, 2, 128)[c.ds][finite] for t in (kc, kd))
        assert finite[:16].all() and torch.equal(ka, kb), scale


def test_slots_beyond_the_pool():
    c = Call(6, 4, 2, 128, 128, "bf16", "bf16", seed=8)
    c.slots[2] = c.kc.shape[0] * 16
    c.ds.copy_(c.slots)
    c.run()
    assert int(c.err) == B.DEVERR_BAD_SLOT and (c.out[2] == 7).all()
    c.slots[2] = -1
    c.ds.copy_(c.slots)
    c.verify("bad slot")


def test_streams_and_graphs():
    c = Call(50, 8, 2, 128, 128, "bf16", "bf16", seed=9).run()
    first = c.out.clone()
    s = torch.cuda.Stream()
    c.out.fill_(7.0)
    torch.cuda.synchronize()
    c.run(stream=s)
    s.synchronize()
    assert torch.equal(c.out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    c.pos = c.pos.flip(0).contiguous()
    c.dp.copy_(c.pos)
    g.replay()
    c.verify("replayed at other positions")


@pytest.mark.parametrize("scaling", ["linear", "ntk", "llama3", "yarn"])
def test_scaled_frequencies(scaling):
    c = Call(30, 2, 1, 128, 128, "f32", "f32", seed=10, far=100000)
    inv, c.scale = pkv.rotary_frequencies(128, 500000.0, scaling, factor=8.0)
    c.inv = torch.from_numpy(inv)
    c.di.copy_(c.inv)
    c.run().verify(scaling)


def test_rows_past_two_to_the_31_elements():
    """Token strides that put the last rows past 2^31 elements."""
    T, hq, D, wide = 9, 2, 128, 1 << 28
    x = torch.zeros((T - 1) * wide + hq * D, dtype=torch.bfloat16, device="cuda")
    q = x.as_strided((T, hq, D), (wide, D, 1))
    q.copy_(torch.randn(T, hq, D))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 1000
    inv = torch.from_numpy(pkv.rotary_frequencies(128)[0]).cuda()
    out = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda")
    desc = B.CacheDesc(num_blocks=4, block_size=16, num_kv_heads=1, head_dim=128, dtype=B.PKV_BF16, k_scale=1.0, v_scale=1.0)
    pkv.pkv_rope_and_cache(out, q, None, None, pos, None, inv, None, None, desc)
    ref, size = rotate(q.cpu(), pos.cpu(), inv.cpu(), 1.0, False)
    near(out.cpu(), ref, size, "bf16", "far rows")
