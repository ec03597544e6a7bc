"""What is measured of a speculative decoding step over the paged cache: rotating and appending, attention for trees
of drafted tokens, and committing the accepted path.

Three operators, each as the calls a serving program makes (``own``) and in a plain form of elementary torch
operations:

* ``rope``: rotary positions applied to queries and keys, keys and values appended to the paged cache;
* ``tree``: attention of runs of drafted tokens, masked by their tree, over paged K/V;
* ``commit``: the accepted path of each tree, its K/V moved to consecutive slots in every layer.

Sizes, tree shapes and accepted paths come from the case alone (``mix`` seeds them), so that ``work`` knows them; values,
token ids, physical block order and scattering come from the seed.
"""
import math
import random

import torch

own = False

CACHE_BYTES = {"f32": 4, "bf16": 2, "fp8": 1, "int8": 1}
KV_SCALE = {"f32": 1.0, "bf16": 1.0, "fp8": 1.0, "int8": 1.0 / 32}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode token of each of 8 requests (latency)
        {"name": "rope_decode_8", "op": "rope", "tokens": 8, "hq": 32, "hkv": 8, "D": 128, "rot": 128, "pairs": "halves",
         "src": "bf16", "kv": "bf16", "fused": True, "far": 2048, "base": 500000.0, "scaling": "none", "pad": 0, "mix": 1},
        # the drafted tokens of a batch at far positions, scaled for long contexts, one-byte cache
        {"name": "rope_drafts_fp8", "op": "rope", "tokens": 1013, "hq": 64, "hkv": 8, "D": 128, "rot": 128, "pairs": "halves",
         "src": "bf16", "kv": "fp8", "fused": False, "far": 131072, "base": 10000.0, "scaling": "yarn", "pad": 11, "mix": 2},
        # half of each small head rotated in neighbouring pairs, everything in 32 bits
        {"name": "rope_part_f32", "op": "rope", "tokens": 777, "hq": 16, "hkv": 8, "D": 64, "rot": 32, "pairs": "neighbours",
         "src": "f32", "kv": "f32", "fused": False, "far": 4096, "base": 10000.0, "scaling": "linear", "pad": 0, "mix": 3},
        # prompts, queries, keys and values as one projection leaves them
        {"name": "rope_prompt_8192", "op": "rope", "tokens": 8192, "hq": 32, "hkv": 8, "D": 128, "rot": 128,
         "pairs": "halves", "src": "bf16", "kv": "bf16", "fused": True, "far": 8192, "base": 500000.0, "scaling": "none",
         "pad": 0, "mix": 4},
        # a small tree for a single request (latency)
        {"name": "tree_one_8", "op": "tree", "n": 1, "nodes": -8, "past": 700, "hq": 32, "hkv": 8, "S": 16, "kv": "bf16",
         "shape": "tree", "mix": 5},
        # chains of four drafted tokens for a full batch, lengths as in the 256-sequence GQA batch
        {"name": "tree_chains_256", "op": "tree", "n": 256, "nodes": -5, "past": 1300, "hq": 32, "hkv": 8, "S": 16,
         "kv": "bf16", "shape": "chain", "mix": 6},
        # trees of all sizes, one-byte cache, ragged everywhere
        {"name": "tree_ragged_int8", "op": "tree", "n": 96, "nodes": 24, "past": 2048, "hq": 32, "hkv": 8, "S": 16,
         "kv": "int8", "shape": "tree", "mix": 7},
        # trees over long contexts, eight query heads a KV head, one-byte cache
        {"name": "tree_long_fp8", "op": "tree", "n": 48, "nodes": -16, "past": 14000, "hq": 64, "hkv": 8, "S": 16,
         "kv": "fp8", "shape": "tree", "mix": 8},
        # wide trees: where the products count as much as the reading
        {"name": "tree_wide_64", "op": "tree", "n": 32, "nodes": -64, "past": 6000, "hq": 64, "hkv": 8, "S": 16,
         "kv": "bf16", "shape": "tree", "mix": 9},
        # a few requests' trees committed in a 32-layer model (latency)
        {"name": "commit_8", "op": "commit", "n": 8, "nodes": -16, "layers": 32, "hkv": 8, "S": 16, "kv": "bf16",
         "shape": "tree", "mix": 10},
        # a full batch of ragged trees in the same model
        {"name": "commit_256", "op": "commit", "n": 256, "nodes": 32, "layers": 32, "hkv": 8, "S": 16, "kv": "bf16",
         "shape": "tree", "mix": 11},
        # wide trees, 80 layers, one-byte cache
        {"name": "commit_layers_fp8", "op": "commit", "n": 48, "nodes": -64, "layers": 80, "hkv": 8, "S": 16, "kv": "fp8",
         "shape": "tree", "mix": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "tree", "tree", "commit"))
    case = {"op": op, "mix": rng.randrange(1 << 30)}
    hq, hkv = rng.choice(((32, 8), (64, 8), (32, 32), (8, 8), (16, 8), (12, 3), (8, 1)))
    if op == "rope":
        D = rng.choice((64, 128, 128))
        src, kv = rng.choice((("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "fp8"), ("bf16", "int8"), ("f32", "f32"),
                              ("f32", "bf16"), ("f32", "fp8")))
        tokens = _log(rng, 1, 8192)
        case.update(tokens=tokens, hq=hq, hkv=hkv, D=D, rot=rng.choice((D, D, D // 2, 24)), src=src, kv=kv,
                    pairs=rng.choice(("halves", "neighbours")), fused=rng.random() < 0.5, far=_log(rng, 1, 1 << 20),
                    base=rng.choice((10000.0, 500000.0, 1000000.0)), scaling=rng.choice(("none", "linear", "yarn")),
                    pad=rng.choice((0, 0, tokens // 16, min(tokens // 2, 3))))
        top, keys = "rope_prompt_8192", ("tokens",)
    elif op == "tree":
        case.update(n=_log(rng, 1, 256), nodes=rng.choice((-1, 1, -1)) * _log(rng, 1, 96), past=rng.choice((0, _log(rng, 1, 16384),
                    _log(rng, 1, 16384), _log(rng, 1, 16384))), hq=hq, hkv=hkv, S=rng.choice((8, 16, 32)),
                    kv=rng.choice(("bf16", "fp8", "int8")), shape=rng.choice(("tree", "tree", "chain", "free")))
        top, keys = "tree_wide_64", ("n", "past", "nodes")
    else:
        case.update(n=_log(rng, 1, 256), nodes=rng.choice((-1, 1)) * _log(rng, 1, 96), layers=_log(rng, 1, 80), hkv=hkv,
                    S=rng.choice((4, 8, 16, 32)), kv=rng.choice(("f32", "bf16", "fp8", "int8")),
                    shape=rng.choice(("tree", "tree", "chain")))
        top, keys = "commit_256", ("n", "layers")
    tops = [work(c) for c in listed() if c["op"] == op]
    limit = {"bytes": max(w["bytes"] for w in tops), "flops": max(w["flops"] for w in tops)}
    pool = _pool_bytes(next(c for c in listed() if c["name"] == top)) if op == "commit" else 0
    while any(work(case)[k] > limit[k] for k in limit) or (op == "commit" and _pool_bytes(case) > pool):
        k = max(keys, key=lambda x: abs(case[x]))
        if abs(case[k]) <= 1:
            break
        case[k] = int(case[k] * 3 / 4)
        if op == "rope":
            case["pad"] = min(case["pad"], case["tokens"] // 2)
    return case


# ------------------------------------------------------------------ sizes and shapes

def _spread(r, mean, hi=8):
    """A length around ``mean``, lognormal, between 1 and ``hi`` times it."""
    return max(1, min(hi * mean, int(round(mean * math.exp(r.gauss(0.0, 0.7))))))


def _blocks(length, S):
    return -(-length // S)


def _runs(c):
    """Tokens of each run (nodes < 0: all alike) and tokens before it."""
    r = random.Random(c["mix"])
    nodes = [-c["nodes"] if c["nodes"] < 0 else min(128, _spread(r, c["nodes"], 3)) for _ in range(c["n"])]
    if c["op"] == "commit":  # only the ends of the sequences matter
        return nodes, [r.randrange(49) for _ in nodes]
    return nodes, [_spread(r, c["past"], 4) if c["past"] else 0 for _ in nodes]


def _parents(r, n, shape):
    """A tree's nodes in breadth-first order: node 0 the token that is already chosen, the others drafted."""
    if shape == "chain":
        return list(range(-1, n - 1))
    p = [-1] + [min(i - 1, int(i * r.random() ** 2)) for i in range(1, n)]
    return [-1] + sorted(p[1:])


def _trees(c):
    r = random.Random(c["mix"] + 1)
    return [_parents(r, n, c["shape"]) for n in _runs(c)[0]]


def _masks(c):
    """The run's tokens that each token sees, as whole numbers (bit j: token j); None for a chain."""
    if c["shape"] == "chain":
        return None
    out = []
    if c["shape"] == "free":  # any set of the run's tokens, none among them
        r = random.Random(c["mix"] + 2)
        for n in _runs(c)[0]:
            out += [0 if r.random() < 0.1 else r.getrandbits(n) for _ in range(n)]
        return out
    for p in _trees(c):
        m = []
        for i, up in enumerate(p):
            m.append((m[up] if up >= 0 else 0) | 1 << i)
        out += m
    return out


def _path(r, p):
    """An accepted path whose tokens' new places are none of the places that tokens leave (so that a pass can be repeated)."""
    kids = {}
    for i, up in enumerate(p):
        kids.setdefault(up, []).append(i)
    path = [0]
    while path[-1] in kids and r.random() < 0.8:
        path.append(r.choice(kids[path[-1]]))
    while not all(i == j or i >= len(path) for j, i in enumerate(path)):
        path.pop()
    return path


def _paths(c):
    r = random.Random(c["mix"] + 3)
    return [_path(r, p) for p in _trees(c)]


def _pool_blocks(c):
    nodes, past = _runs(c)
    return sum(_blocks(p + n, c["S"]) for p, n in zip(past, nodes)) + 2


def _pool_bytes(c):
    return _pool_blocks(c) * c["S"] * c["hkv"] * 128 * CACHE_BYTES[c["kv"]] * 2 * c["layers"]


def work(case):
    c = case
    if c["op"] == "rope":
        live = c["tokens"] - c["pad"]
        es, ec = CACHE_BYTES[c["src"]], CACHE_BYTES[c["kv"]]
        per = (2 * c["hq"] + 2 * c["hkv"]) * c["D"] * es + 2 * c["hkv"] * c["D"] * ec + 4
        return {"bytes": live * per + 8 * c["tokens"] + 2 * c["rot"], "flops": live * (c["hq"] + c["hkv"]) * c["rot"] * 3}
    nodes, past = _runs(c)
    if c["op"] == "tree":
        masks, S = _masks(c), c["S"]
        keys = sum(nodes) + sum(past)
        own_pairs = sum(n * (n + 1) // 2 for n in nodes) if masks is None else sum(bin(m).count("1") for m in masks)
        pairs = sum(n * p for n, p in zip(nodes, past)) + own_pairs
        words = 0 if masks is None else sum(nodes) * _blocks(max(nodes), 64)
        return {"bytes": keys * c["hkv"] * 256 * CACHE_BYTES[c["kv"]] + 4 * sum(nodes) * c["hq"] * 128 + 8 * words +
                4 * sum(_blocks(n + p, S) for n, p in zip(nodes, past)) + 8 * c["n"] + 4, "flops": 512 * c["hq"] * pairs}
    moved = sum(sum(i != j for j, i in enumerate(p)) for p in _paths(c))
    row = c["hkv"] * 128 * CACHE_BYTES[c["kv"]]
    return {"bytes": moved * c["layers"] * 4 * row + 16 * sum(nodes) + 28 * c["n"] + 8 * moved, "flops": sum(nodes)}


# ------------------------------------------------------------------ inputs

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _values(g, shape, kv):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16 if kv in ("bf16", "fp8") else torch.float32)
    return (x / KV_SCALE[kv]).round().clamp(-127, 127).to(torch.int8) if kv == "int8" else x.to(TYPES[kv])


def _frequencies(c):
    """Angles per position of each pair, and what cos and sin are multiplied by (positions scaled to eight times the length)."""
    half = c["rot"] // 2
    inv = [c["base"] ** (-i / half) for i in range(half)]
    if c["scaling"] == "linear":
        return [f / 8 for f in inv], 1.0
    if c["scaling"] == "yarn":  # fast pairs as they are, slow ones stretched, a ramp between
        def at(turns):
            return half * math.log(4096 / (turns * 2 * math.pi)) / math.log(c["base"])
        lo, hi = max(0, math.floor(at(32))), min(half - 1, math.ceil(at(1)))
        ramp = [min(1.0, max(0.0, (i - lo) / max(1e-3, hi - lo))) for i in range(half)]
        return [f * (1 - w) + f / 8 * w for f, w in zip(inv, ramp)], 0.1 * math.log(8) + 1
    return inv, 1.0


def _prepare_rope(c, g, hg):
    T, hq, hkv, D = c["tokens"], c["hq"], c["hkv"], c["D"]
    S, src = 16, TYPES[c["src"]]
    nb = _blocks(T, S) + 2
    if c["fused"]:
        x = torch.randn((T, hq + 2 * hkv, D), generator=g, device="cuda").to(src)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = (torch.randn((T, h, D), generator=g, device="cuda").to(src) for h in (hq, hkv, hkv))
    slots = torch.randperm(nb * S, generator=hg)[:T]
    slots[T - c["pad"]:] = -1
    inv, factor = _frequencies(c)
    return {"q": q, "k_new": k, "v_new": v, "slots": slots.cuda(), "interleaved": c["pairs"] == "neighbours",
            "positions": torch.randint(0, c["far"], (T,), generator=hg).to(torch.int32).cuda(), "factor": factor,
            "inv": torch.tensor(inv, dtype=torch.float32, device="cuda"),
            "q_out": torch.zeros((T, hq, D), dtype=src, device="cuda"), "kv_scale": KV_SCALE[c["kv"]],
            "k": _values(g, (nb, S, hkv, D), c["kv"]), "v": _values(g, (nb, S, hkv, D), c["kv"])}


def _prepare_runs(c, g, hg):
    S, (nodes, past) = c["S"], _runs(c)
    lens = [p + n for p, n in zip(past, nodes)]
    nb = _pool_blocks(c)
    perm, at = torch.randperm(nb, generator=hg).to(torch.int32), 0
    tables = torch.full((c["n"], max(_blocks(L, S) for L in lens)), -1, dtype=torch.int32)
    for i, L in enumerate(lens):
        tables[i, :_blocks(L, S)] = perm[at:at + _blocks(L, S)]
        at += _blocks(L, S)
    cu = [0]
    for n in nodes:
        cu.append(cu[-1] + n)
    return {"S": S, "nodes": nodes, "past_host": past, "lens_host": lens, "cu_host": cu, "tables": tables.cuda(),
            "past": _i32(past), "lens": _i32(lens), "cu": _i32(cu)}, nb


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    hg = torch.Generator().manual_seed(seed)
    if c["op"] == "rope":
        st = _prepare_rope(c, g, hg)
    else:
        st, nb = _prepare_runs(c, g, hg)
        T = st["cu_host"][-1]
    st.update(op=c["op"], err=_i32([0]))
    if c["op"] == "tree":
        st.update(hq=c["hq"], hkv=c["hkv"], scale=1.0 / math.sqrt(128), kv_scale=KV_SCALE[c["kv"]],
                  k=_values(g, (nb, c["S"], c["hkv"], 128), c["kv"]), v=_values(g, (nb, c["S"], c["hkv"], 128), c["kv"]),
                  q=torch.randn((T, c["hq"], 128), generator=g, device="cuda").to(torch.bfloat16))
        st["out"] = torch.zeros_like(st["q"])
        masks = _masks(c)
        st["mask"] = None
        if masks is not None:
            W = _blocks(max(st["nodes"]), 64)
            words = [[(m >> 64 * w & (1 << 64) - 1) for w in range(W)] for m in masks]
            st["mask"] = torch.tensor([[w - (1 << 64) if w >> 63 else w for w in row] for row in words], dtype=torch.int64,
                                      device="cuda")
    if c["op"] == "commit":
        r = random.Random(seed)
        parents, draft, target = [], [], []
        for p, path in zip(_trees(c), _paths(c)):
            d = r.sample(range(128000), len(p))
            t = [r.randrange(128000) for _ in p]
            for a, b in zip(path, path[1:]):
                t[a] = d[b]
            t[path[-1]] = 128000 + r.randrange(256)  # what no draft holds
            parents, draft, target = parents + p, draft + d, target + t
        shape = (c["layers"], nb, c["S"], c["hkv"], 128)
        st.update(parents=_i32(parents), draft=_i32(draft), target=_i32(target), longest=max(st["nodes"]),
                  ks=_values(g, shape, c["kv"]), vs=_values(g, shape, c["kv"]), accepted=_i32([0] * T),
                  **{k: _i32([0] * c["n"]) for k in ("count", "seq_lens", "next", "keep")})
    if own:
        import paged_kv_cache_71_gb300 as pkv
        if c["op"] == "commit":
            st["layers"] = pkv.LayerCaches(list(st["ks"]), list(st["vs"]))
        else:
            st["desc"] = pkv.CacheDesc.for_cache(st["k"], st["kv_scale"], st["kv_scale"])
        if c["op"] == "tree":
            ws = pkv.pkv_paged_attention_tree_workspace_size(st["desc"], T, c["n"], c["hq"])
            st["ws"] = torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _held(x, scale):
    """Cached 8-bit whole numbers as the values they stand for."""
    return x.float() * scale if x.dtype == torch.int8 else x


def _rotated(x, cos, sin, rot, interleaved):
    """x [T][heads][D] in 32 bits, cos and sin [T][rot / 2]."""
    c, s = cos[:, None], sin[:, None]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., : rot // 2], x[..., rot // 2:rot])
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _stored(x, like, scale):
    """Values as the cache holds them."""
    if like.dtype == torch.int8:
        return (x / scale).round().clamp(-127, 127).to(torch.int8)
    if like.dtype == torch.float8_e4m3fn:
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
    return x.to(like.dtype)


def _placed(cache, rows, slots):
    """The cache with rows [T][heads][D] at their slots, those of negative slots left out."""
    flat = cache.reshape(-1, *cache.shape[2:])
    raw = flat.view(torch.uint8).clone() if flat.dtype == torch.float8_e4m3fn else flat.clone()
    live = slots >= 0
    raw[slots[live]] = (rows.view(torch.uint8) if flat.dtype == torch.float8_e4m3fn else rows)[live]
    return raw.view(flat.dtype).reshape(cache.shape)


def _plain_rope(st):
    rot = 2 * st["inv"].numel()
    angle = st["positions"].double()[:, None] * st["inv"].double()
    cos, sin = (torch.cos(angle) * st["factor"]).float(), (torch.sin(angle) * st["factor"]).float()
    q = _rotated(st["q"].float(), cos, sin, rot, st["interleaved"])
    k = _rotated(st["k_new"].float(), cos, sin, rot, st["interleaved"])
    q_out = torch.where((st["slots"] >= 0)[:, None, None], q.to(st["q_out"].dtype), st["q_out"])
    kc = _placed(st["k"], _stored(k, st["k"], st["kv_scale"]), st["slots"])
    vc = _placed(st["v"], _stored(st["v_new"].float(), st["v"], st["kv_scale"]), st["slots"])
    return [q_out, _held(kc, st["kv_scale"]), _held(vc, st["kv_scale"])]


def _plain_tree(st):
    hq, hkv, S = st["hq"], st["hkv"], st["S"]
    G = hq // hkv
    out = torch.empty(st["q"].shape, dtype=torch.float32, device="cuda")
    for s, L in enumerate(st["lens_host"]):
        a, b = st["cu_host"][s], st["cu_host"][s + 1]
        n = b - a
        t = st["tables"][s, : _blocks(L, S)].long()
        k = (st["k"][t].float() * st["kv_scale"]).reshape(-1, hkv, 128)[:L]
        v = (st["v"][t].float() * st["kv_scale"]).reshape(-1, hkv, 128)[:L]
        j = torch.arange(n, device="cuda")
        if st["mask"] is None:
            seen = j[None, :] <= j[:, None]
        else:
            seen = (st["mask"][a:b][:, j // 64] >> (j % 64) & 1) != 0
        x = torch.einsum("nhgd,thd->nhgt", st["q"][a:b].float().reshape(n, hkv, G, 128), k) * st["scale"]
        x[..., L - n:] = x[..., L - n:].masked_fill(~seen[:, None, None, :], float("-inf"))
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - torch.where(m == float("-inf"), torch.zeros_like(m), m))
        l = e.sum(-1, keepdim=True)
        o = torch.einsum("nhgt,thd->nhgd", e, v) / torch.where(l == 0, torch.ones_like(l), l)
        out[a:b] = o.reshape(n, hq, 128)
    return out.to(torch.bfloat16)


def _plain_commit(st):
    S, n, longest = st["S"], len(st["nodes"]), st["longest"]
    cu, past = st["cu"].long(), st["past"].long()
    T, rows = st["parents"].numel(), torch.arange(n, device="cuda")
    at = (cu[:-1, None] + torch.arange(longest, device="cuda")).clamp(max=T - 1)
    inside = torch.arange(longest, device="cuda") < (cu[1:] - cu[:-1])[:, None]
    parents = torch.where(inside, st["parents"].long()[at], torch.full_like(at, -2))
    draft, target = st["draft"][at], st["target"][at]
    place = torch.full((n, longest), -1, dtype=torch.int64, device="cuda")
    place[:, 0] = 0
    cur, alive = torch.zeros(n, dtype=torch.int64, device="cuda"), torch.ones(n, dtype=torch.bool, device="cuda")
    for step in range(1, longest):
        fits = (parents == cur[:, None]) & (draft == target[rows, cur][:, None])
        alive = alive & fits.any(1)
        cur = torch.where(alive, fits.to(torch.uint8).argmax(1), cur)
        place[:, step] = torch.where(alive, cur, place[:, step])
    count = (place >= 0).sum(1)
    lens, nxt = past + count, target[rows, cur]
    accepted = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    accepted[at[inside]] = place[inside].to(torch.int32)
    moved = (place >= 0) & (place != torch.arange(longest, device="cuda"))
    r, j = moved.nonzero(as_tuple=True)
    src, dst = past[r] + place[r, j], past[r] + j
    src_b, dst_b = st["tables"][r, src // S].long(), st["tables"][r, dst // S].long()
    caches = []
    for c in (st["ks"], st["vs"]):
        raw = c.view(torch.uint8).clone() if c.dtype == torch.float8_e4m3fn else c.clone()
        raw[:, dst_b, dst % S] = raw[:, src_b, src % S]
        caches.append(raw.view(c.dtype))
    i32 = torch.int32
    return [accepted, count.to(i32), lens.to(i32), nxt, ((lens + S - 1) // S).to(i32), *caches]


def run(state):
    st = state
    if not own:
        return {"rope": _plain_rope, "tree": _plain_tree, "commit": _plain_commit}[st["op"]](st)
    import paged_kv_cache_71_gb300 as pkv
    if st["op"] == "rope":
        pkv.pkv_rope_and_cache(st["q_out"], st["q"], st["k_new"], st["v_new"], st["positions"], st["slots"], st["inv"],
                               st["k"], st["v"], st["desc"], st["interleaved"], st["factor"], st["err"])
        return [st["q_out"], _held(st["k"], st["kv_scale"]), _held(st["v"], st["kv_scale"])]
    if st["op"] == "tree":
        pkv.pkv_paged_attention_tree(st["out"], st["q"], st["cu"], st["lens"], st["mask"], st["k"], st["v"], st["desc"],
                                     st["tables"], st["scale"], st["ws"], st["err"])
        return st["out"]
    pkv.pkv_commit_tree(st["layers"], st["tables"], st["cu"], st["past"], st["parents"], st["draft"], st["target"],
                        st["accepted"], st["count"], st["seq_lens"], st["next"], st["keep"], st["err"])
    return [st["accepted"], st["count"], st["seq_lens"], st["next"], st["keep"], st["ks"], st["vs"]]


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_rope(case, st):
    T, rot, f = case["tokens"], case["rot"], st["factor"]
    half = rot // 2
    th = torch.outer(st["positions"].double(), st["inv"].double())[:, None, :]
    first = torch.arange(half, device="cuda") * (2 if st["interleaved"] else 1)
    second = first + (1 if st["interleaved"] else half)

    def turn(x):
        x = x.double().clone()
        a, b = x[..., first].clone(), x[..., second].clone()
        x[..., first] = f * (a * torch.cos(th) - b * torch.sin(th))
        x[..., second] = f * (a * torch.sin(th) + b * torch.cos(th))
        return x

    live = st["slots"] >= 0
    q = torch.zeros_like(st["q_out"], dtype=torch.float64)
    q[live] = turn(st["q"])[live]
    out, most = [q], {"int8": 127 * st["kv_scale"], "fp8": 448 * st["kv_scale"]}.get(case["kv"], math.inf)
    for cache, new in ((st["k"], turn(st["k_new"])), (st["v"], st["v_new"].double())):
        flat = cache.double().reshape(-1, *cache.shape[2:]) * st["kv_scale"]
        flat[st["slots"][live]] = new[live].clamp(-most, most)
        out.append(flat.reshape(cache.shape))
    return out


def _exact_tree(case, st):
    hkv, S, masks = case["hkv"], case["S"], _masks(case)
    G = case["hq"] // hkv
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, (n, p) in enumerate(zip(*_runs(case))):
        a, L = st["cu_host"][s], p + n
        pos = torch.arange(L, device="cuda")
        block = st["tables"][s].long()[pos // S]
        k = (st["k"][block, pos % S].double() * st["kv_scale"]).permute(1, 2, 0)  # [heads, D, L]
        v = (st["v"][block, pos % S].double() * st["kv_scale"]).permute(1, 0, 2)  # [heads, L, D]
        own_bits = torch.tensor([[(masks[a + i] >> j & 1) if masks is not None else int(j <= i) for j in range(n)]
                                 for i in range(n)], device="cuda").bool()
        seen = torch.cat([torch.ones(n, p, dtype=torch.bool, device="cuda"), own_bits], 1).repeat_interleave(G, 0)
        q = st["q"][a:a + n].double().reshape(n, hkv, G, 128).permute(1, 0, 2, 3).reshape(hkv, n * G, 128)
        w = torch.softmax((torch.bmm(q, k) * st["scale"]).masked_fill(~seen, -math.inf), dim=-1)
        w = w.masked_fill(~seen, 0.0)  # a row that sees nothing
        out[a:a + n] = torch.bmm(w, v).reshape(hkv, n, G, 128).permute(1, 0, 2, 3).reshape(n, -1, 128)
    return out


def _exact_commit(case, st):
    S, tables = case["S"], st["tables"].tolist()
    parents, draft, target = (st[k].tolist() for k in ("parents", "draft", "target"))
    accepted, counts, lens, nexts, keep, moves = [], [], [], [], [], []
    for s, (n, p) in enumerate(zip(*_runs(case))):
        a = st["cu_host"][s]
        path, more = [0], True
        while more:
            more = [i for i in range(n) if parents[a + i] == path[-1] and draft[a + i] == target[a + path[-1]]]
            path += more[:1]
        accepted += path + [-1] * (n - len(path))
        counts.append(len(path))
        lens.append(p + len(path))
        nexts.append(target[a + path[-1]])
        keep.append(_blocks(lens[-1], S))
        moves += [tuple(tables[s][q // S] * S + q % S for q in (p + i, p + j)) for j, i in enumerate(path) if i != j]
    caches = []
    src, dst = ([m[x] for m in moves] for x in (0, 1))
    for c in (st["ks"], st["vs"]):
        flat = (c.float() if c.element_size() == 1 else c.clone()).reshape(len(c), -1, *c.shape[3:])
        for a, b in zip(src, dst):  # the paths are such that no place is both left and taken
            flat[:, b] = flat[:, a]
        caches.append(flat.reshape(c.shape).to(c.dtype))
    return [_i32(accepted), _i32(counts), _i32(lens), _i32(nexts), _i32(keep), *caches]


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "tree": _exact_tree, "commit": _exact_commit}[case["op"]](case, st)
