"""What is measured of the step planning, shared-prefix decode and cross-attention calls.

Four operators, each as the calls a serving program makes (``own``) and in a plain form of elementary torch
operations:

* ``extend``: block tables, lengths and slot maps of a step from the request lengths;
* ``release``: finished sequences hand their blocks back to the free list;
* ``prefix``: one decode token per sequence, groups of sequences sharing a prompt prefix;
* ``cross``: decoder queries against paged encoder states of another length.

Lengths come from the case alone (``mix`` seeds them), so that ``work`` knows them; values, physical block order and
scattering come from the seed.
"""
import math
import random

import torch

own = False

D = 128  # head dimension
KV_BYTES = {"bf16": 2, "fp8": 1, "int8": 1}
KV_SCALE = {"bf16": 1.0, "fp8": 1.0 / 64, "int8": 1.0 / 32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # the smallest decode step of a lightly loaded server: 8 requests, one token each (latency)
        {"name": "extend_decode_8", "op": "extend", "n": 8, "past": 1024, "new": 1, "S": 16, "mix": 1},
        # the decode step of a full batch, lengths as in the 256-sequence GQA batch
        {"name": "extend_decode_256", "op": "extend", "n": 256, "past": 1024, "new": 1, "S": 16, "mix": 2},
        # admission of many prompts at once, some requests idle this step, some continuing a prompt
        {"name": "extend_prompts_512", "op": "extend", "n": 512, "past": 256, "new": 2048, "S": 16, "mix": 3},
        # a few of a full batch finish in this step
        {"name": "release_some_256", "op": "release", "n": 256, "past": 1024, "share": 0.05, "keep": 0, "S": 16,
         "mix": 4},
        # a drained batch of long sequences, each on a shared prefix that stays
        {"name": "release_most_2048", "op": "release", "n": 2048, "past": 4000, "share": 0.9, "keep": 8, "S": 16,
         "mix": 5},
        # four samples of one prompt, shortly after the fork (latency)
        {"name": "prefix_samples_4", "op": "prefix", "n": 4, "groups": 1, "prefix": 512, "suffix": 32, "hq": 32,
         "hkv": 8, "S": 16, "kv": "bf16", "mix": 6},
        # the prefix-sharing batch: 128 sequences over an 800-token prefix, 205 tokens of their own
        {"name": "prefix_shared_128", "op": "prefix", "n": 128, "groups": 1, "prefix": 800, "suffix": -205, "hq": 32,
         "hkv": 8, "S": 16, "kv": "bf16", "mix": 7},
        # several system prompts of different lengths in one batch, one-byte cache, ragged everywhere
        {"name": "prefix_groups_int8", "op": "prefix", "n": 96, "groups": 7, "prefix": 2048, "suffix": 700, "hq": 32,
         "hkv": 8, "S": 16, "kv": "int8", "mix": 8},
        # a long document that a large batch asks about
        {"name": "prefix_document_256", "op": "prefix", "n": 256, "groups": 1, "prefix": 32768, "suffix": 512,
         "hq": 64, "hkv": 8, "S": 16, "kv": "fp8", "mix": 9},
        # decoding over encoder states: one token a sequence, states of about 1500 positions
        {"name": "cross_decode_64", "op": "cross", "n": 64, "tokens": 0, "enc": 1500, "hq": 32, "hkv": 8, "S": 16,
         "kv": "bf16", "mix": 10},
        # beams over one-byte states: a few query tokens for each set of states
        {"name": "cross_beams_fp8", "op": "cross", "n": 24, "tokens": -5, "enc": 900, "hq": 64, "hkv": 8, "S": 16,
         "kv": "fp8", "mix": 11},
        # decoder prompts over long states, multi-head
        {"name": "cross_prompts_long", "op": "cross", "n": 12, "tokens": 700, "enc": 4096, "hq": 32, "hkv": 32,
         "S": 16, "kv": "bf16", "mix": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("extend", "release", "prefix", "cross"))
    case = {"op": op, "S": rng.choice((8, 16, 32)), "mix": rng.randrange(1 << 30)}
    if op == "extend":
        case.update(n=_log(rng, 1, 2048), past=_log(rng, 1, 4096), new=rng.choice((1, _log(rng, 1, 2048))))
    elif op == "release":
        case.update(n=_log(rng, 1, 2048), past=_log(rng, 1, 4000), share=rng.random(), keep=rng.choice((0, 0, 5, 8)))
    else:
        hq, hkv = rng.choice(((32, 8), (64, 8), (32, 32), (8, 8), (16, 8), (12, 3)))
        case.update(hq=hq, hkv=hkv, kv=rng.choice(("bf16", "fp8", "int8")))
        if op == "prefix":
            case.update(n=_log(rng, 1, 256), prefix=rng.choice((0, _log(rng, 16, 32768), _log(rng, 16, 32768))),
                        suffix=_log(rng, 1, 2048))
            case["groups"] = min(case["n"], _log(rng, 1, 12))
        else:
            case.update(n=_log(rng, 1, 64), tokens=rng.choice((0, -_log(rng, 1, 8), _log(rng, 1, 1024))),
                        enc=_log(rng, 1, 8192))
    top = {"extend": "extend_prompts_512", "release": "release_most_2048", "prefix": "prefix_document_256",
           "cross": "cross_prompts_long"}[op]
    limit = work(next(c for c in listed() if c["name"] == top))
    while case["n"] > 1 and any(work(case)[k] > limit[k] for k in limit):
        case["n"] = case["n"] * 3 // 4
        if op == "prefix":
            case["groups"] = min(case["n"], case["groups"])
    while any(work(case)[k] > limit[k] for k in limit):  # one sequence that is itself too much
        for k in ("past", "new", "prefix", "suffix", "tokens", "enc"):
            if case.get(k, 0) > 1:
                case[k] = case[k] * 3 // 4
    return case


# ------------------------------------------------------------------ lengths

def _spread(r, mean, hi=8):
    """A length around ``mean``, lognormal, between 1 and ``hi`` times it."""
    return max(1, min(hi * mean, int(round(mean * math.exp(r.gauss(0.0, 0.7))))))


def _blocks(length, S):
    return -(-length // S)


def _extend_lens(c):
    """past and new tokens of each request; some requests are new, some idle."""
    r = random.Random(c["mix"])
    past, new = [], []
    for _ in range(c["n"]):
        past.append(0 if c["new"] > 1 and r.random() < 0.5 else _spread(r, c["past"]))
        new.append(1 if c["new"] == 1 else 0 if r.random() < 0.1 else _spread(r, c["new"], 2))
    return past, new


def _release_lens(c):
    r = random.Random(c["mix"])
    past = [0 if r.random() < 0.02 else _spread(r, c["past"], 2) for _ in range(c["n"])]
    done = [int(r.random() < c["share"]) for _ in range(c["n"])]
    keep = [min(c["keep"], L // c["S"]) for L in past]
    return past, done, keep


def _prefix_lens(c):
    """group sizes, prefix length of each group (whole blocks), own tokens of each sequence."""
    r = random.Random(c["mix"])
    cuts = sorted(r.sample(range(1, c["n"]), c["groups"] - 1)) if c["groups"] > 1 else []
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [c["n"]])]
    pre = [c["prefix"] // c["S"] * c["S"] if c["groups"] == 1 else
           min(_spread(r, c["prefix"], 2), 2 * c["prefix"]) // c["S"] * c["S"] if c["prefix"] and r.random() < 0.9 else 0
           for _ in sizes]
    if c["suffix"] < 0:
        own_len = [-c["suffix"]] * c["n"]
    else:
        own_len = [_spread(r, c["suffix"], 4) for _ in range(c["n"])]
    return sizes, pre, own_len


def _cross_lens(c):
    """query tokens and encoder states of each sequence; some have no states."""
    r = random.Random(c["mix"])
    enc = [0 if c["n"] > 8 and r.random() < 0.04 else _spread(r, c["enc"], 2) for _ in range(c["n"])]
    if c["tokens"] == 0:
        tok = [1] * c["n"]
    elif c["tokens"] < 0:
        tok = [-c["tokens"]] * c["n"]
    else:
        tok = [_spread(r, c["tokens"], 3) for _ in range(c["n"])]
    return tok, enc


def work(case):
    c = case
    if c["op"] == "extend":
        past, new = _extend_lens(c)
        S, n = c["S"], c["n"]
        blocks = sum(_blocks(p + t, S) - _blocks(p, S) for p, t in zip(past, new))
        tails = sum(1 for p, t in zip(past, new) if p % S and t)
        cap = _capacity(sum(new))
        return {"bytes": 8 * n + 4 + 4 * blocks + 4 * tails + 4 * blocks + 8 * cap + 4 * (3 * n + 1) + 4,
                "flops": sum(new) + n}
    if c["op"] == "release":
        past, done, keep = _release_lens(c)
        S, n = c["S"], c["n"]
        blocks = sum(_blocks(p, S) - k for p, d, k in zip(past, done, keep) if d)
        return {"bytes": 9 * n + 4 + 8 * blocks + 4 * n + 4, "flops": blocks + n}
    es, hq, hkv = KV_BYTES[c["kv"]], c["hq"], c["hkv"]
    if c["op"] == "prefix":
        sizes, pre, own_len = _prefix_lens(c)
        keys = sum(pre) + sum(own_len)
        pairs = sum(n * p for n, p in zip(sizes, pre)) + sum(own_len)
        rows = c["n"]
        entries = (sum(pre) + sum(own_len)) // c["S"]
    else:
        tok, enc = _cross_lens(c)
        keys = sum(enc)
        pairs = sum(t * e for t, e in zip(tok, enc))
        rows = sum(tok)
        entries = keys // c["S"]
    return {"bytes": keys * hkv * D * 2 * es + 2 * rows * hq * D * 2 + 4 * entries + 8 * c["n"],
            "flops": 4 * D * hq * pairs}


def _capacity(tokens):
    """Slots that a program reserves for a step's tokens."""
    return (tokens + 63) // 64 * 64 + 64


# ------------------------------------------------------------------ inputs

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cache(g, nb, S, hkv, kv):
    x = torch.randn((nb, S, hkv, D), generator=g, device="cuda", dtype=torch.float32)
    if kv == "bf16":
        return x.to(torch.bfloat16)
    if kv == "fp8":
        return (x / KV_SCALE[kv]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return (x / KV_SCALE[kv]).round().clamp(-127, 127).to(torch.int8)


def _tables(rows, width, perm):
    """Block tables [len(rows)][width] from lists of indices into a permutation of the pool, -1 past the end."""
    t = torch.full((len(rows), width), -1, dtype=torch.int32)
    for i, r in enumerate(rows):
        t[i, : len(r)] = perm[torch.tensor(r, dtype=torch.int64)] if r else t[i, :0]
    return t.cuda()


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    hg = torch.Generator().manual_seed(seed)
    S = c["S"]
    if c["op"] in ("extend", "release"):
        if c["op"] == "extend":
            past, new = _extend_lens(c)
        else:
            past, done, keep = _release_lens(c)
            new = [0] * c["n"]
        used = sum(_blocks(p, S) for p in past)
        need = sum(_blocks(p + t, S) for p, t in zip(past, new))
        nb = need + max(8, need // 20)
        perm = torch.randperm(nb, generator=hg).to(torch.int32)
        rows, at = [], 0
        for p in past:
            rows.append(range(at, at + _blocks(p, S)))
            at += _blocks(p, S)
        width = max(_blocks(p + t, S) for p, t in zip(past, new)) + 4
        tables = torch.full((c["n"], width), -1, dtype=torch.int32)
        for i, r in enumerate(rows):
            tables[i, : len(r)] = perm[r.start:r.stop]
        free = torch.full((nb,), -1, dtype=torch.int32)
        free[: nb - used] = perm[used:]
        st = {"op": c["op"], "S": S, "num_blocks": nb, "tables": tables.cuda(), "past": _i32(past),
              "free": free.cuda(), "count": _i32([nb - used]), "seq_lens": _i32([0] * c["n"]),
              "count_out": _i32([0]), "err": _i32([0])}
        if c["op"] == "extend":
            cap = _capacity(sum(new))
            st.update(new=_i32(new), cap=cap, cu_q=_i32([0] * (c["n"] + 1)), q_starts=_i32([0] * c["n"]),
                      slots=torch.zeros(cap, dtype=torch.int64, device="cuda"))
        else:
            st.update(done=torch.tensor(done, dtype=torch.bool, device="cuda"), keep=_i32(keep))
        return st
    hq, hkv = c["hq"], c["hkv"]
    if c["op"] == "prefix":
        sizes, pre, own_len = _prefix_lens(c)
        rows, at, lens, s = [], 0, [], 0
        for n, p in zip(sizes, pre):
            head = list(range(at, at + p // S))
            at += p // S
            for _ in range(n):
                b = _blocks(own_len[s], S)
                rows.append(head + list(range(at, at + b)))
                lens.append(p + own_len[s])
                at += b
                s += 1
        n_rows = c["n"]
    else:
        tok, lens = _cross_lens(c)
        rows, at = [], 0
        for L in lens:
            rows.append(list(range(at, at + _blocks(L, S))))
            at += _blocks(L, S)
        n_rows = sum(tok)
    nb = at + max(2, at // 20)
    perm = torch.randperm(nb, generator=hg).to(torch.int32)
    st = {"op": c["op"], "S": S, "kv": c["kv"], "hq": hq, "hkv": hkv, "scale": 1.0 / math.sqrt(D),
          "kv_scale": KV_SCALE[c["kv"]], "k": _cache(g, nb, S, hkv, c["kv"]), "v": _cache(g, nb, S, hkv, c["kv"]),
          "q": torch.randn((n_rows, hq, D), generator=g, device="cuda").to(torch.bfloat16),
          "tables": _tables(rows, max(1, max(len(r) for r in rows)), perm), "lens_host": lens, "lens": _i32(lens),
          "err": _i32([0])}
    st["out"] = torch.zeros_like(st["q"])
    if c["op"] == "prefix":
        cu = [0]
        for n in sizes:
            cu.append(cu[-1] + n)
        st.update(cu_host=cu, pre_host=pre, cu=_i32(cu), pre=_i32(pre))
    else:
        cu = [0]
        for n in tok:
            cu.append(cu[-1] + n)
        st.update(cu_host=cu, single=c["tokens"] == 0, cu=None if c["tokens"] == 0 else _i32(cu))
    if own:
        import paged_kv_cache_71_gb300 as pkv
        st["desc"] = pkv.CacheDesc.for_cache(st["k"], st["kv_scale"], st["kv_scale"])
        if c["op"] == "prefix":
            ws = pkv.pkv_paged_attention_decode_prefix_workspace_size(st["desc"], c["n"], hq)
        else:
            ws = pkv.pkv_paged_cross_attention_workspace_size(st["desc"], n_rows, c["n"], hq)
        st["ws"] = torch.empty(max(ws, 16), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _plain_extend(st):
    S, past, new, tables, F = st["S"], st["past"].long(), st["new"].long(), st["tables"], st["count"].long()
    n, width = tables.shape
    nb0, nb1 = (past + S - 1) // S, (past + new + S - 1) // S
    taken = torch.cumsum(nb1 - nb0, 0)
    first = taken - (nb1 - nb0)
    j = torch.arange(width, device="cuda")[None, :]
    at = F - 1 - (first[:, None] + j - nb0[:, None])
    fresh = (j >= nb0[:, None]) & (j < nb1[:, None])
    table = torch.where(fresh, st["free"][at.clamp(0, st["num_blocks"] - 1)], tables)
    ends = torch.cumsum(new, 0)
    cu = torch.cat([ends.new_zeros(1), ends])
    t = torch.arange(st["cap"], device="cuda")
    s = torch.searchsorted(ends, t, right=True).clamp(max=n - 1)
    p = past[s] + t - cu[s]
    slots = table[s, (p // S).clamp(0, width - 1)].long() * S + p % S
    slots = torch.where(t < ends[-1], slots, torch.full_like(slots, -1))
    i32 = torch.int32
    return [table, (past + new).to(i32), (F - taken[-1]).to(i32), cu.to(i32), past.to(i32), slots]


def _plain_release(st):
    S, past, done, tables, F = st["S"], st["past"].long(), st["done"], st["tables"], st["count"].long()
    nb = (past + S - 1) // S
    gone = torch.where(done, (nb - st["keep"].long()).clamp(min=0), torch.zeros_like(nb))
    ends = torch.cumsum(gone, 0)
    i = torch.arange(st["num_blocks"], device="cuda") - F  # place on the stack past its old top
    s = torch.searchsorted(ends, i, right=True).clamp(max=len(past) - 1)
    j = st["keep"].long()[s] + i - (ends[s] - gone[s])
    freed = tables[s, j.clamp(0, tables.shape[1] - 1)]
    free = torch.where((i >= 0) & (i < ends[-1]), freed, st["free"])
    lens = torch.where(done, torch.zeros_like(past), past)
    return [free, lens.to(torch.int32), (F + ends[-1]).to(torch.int32)]


def _rows(cache, table, scale):
    """The tokens named by a row of block ids, in 32 bits: [..., blocks * S, heads, D]."""
    x = cache[table.long()]
    x = x.float() * scale
    return x.reshape(*table.shape[:-1], -1, *x.shape[-2:])


def _plain_prefix(st):
    S, hq, hkv = st["S"], st["hq"], st["hkv"]
    G = hq // hkv
    outs = []
    for g, p in enumerate(st["pre_host"]):
        a, b = st["cu_host"][g], st["cu_host"][g + 1]
        n = b - a
        q = st["q"][a:b].float().reshape(n, hkv, G, D)
        width = max(_blocks(L, S) for L in st["lens_host"][a:b])
        own_t = st["tables"][a:b, p // S:width].clamp(min=0)
        ko, vo = _rows(st["k"], own_t, st["kv_scale"]), _rows(st["v"], own_t, st["kv_scale"])
        so = torch.einsum("nhgd,nthd->nhgt", q, ko) * st["scale"]
        pos = p + torch.arange(so.shape[-1], device="cuda")
        so = so.masked_fill(pos >= st["lens"][a:b, None, None, None], float("-inf"))
        vo = vo.masked_fill((pos >= st["lens"][a:b, None])[..., None, None], 0.0)
        if p:
            pre_t = st["tables"][a, : p // S]
            kp, vp = _rows(st["k"], pre_t, st["kv_scale"]), _rows(st["v"], pre_t, st["kv_scale"])
            sp = torch.einsum("nhgd,thd->nhgt", q, kp) * st["scale"]
            m = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
            ep, eo = torch.exp(sp - m), torch.exp(so - m)
            o = torch.einsum("nhgt,thd->nhgd", ep, vp) + torch.einsum("nhgt,nthd->nhgd", eo, vo)
            o = o / (ep.sum(-1, keepdim=True) + eo.sum(-1, keepdim=True))
        else:
            eo = torch.exp(so - so.amax(-1, keepdim=True))
            o = torch.einsum("nhgt,nthd->nhgd", eo, vo) / eo.sum(-1, keepdim=True)
        outs.append(o.reshape(n, hq, D))
    return torch.cat(outs).to(torch.bfloat16)


def _plain_cross(st):
    hq, hkv, S = st["hq"], st["hkv"], st["S"]
    G = hq // hkv
    out = torch.zeros(st["q"].shape, dtype=torch.float32, device="cuda")
    for s, L in enumerate(st["lens_host"]):
        a, b = st["cu_host"][s], st["cu_host"][s + 1]
        if L == 0 or a == b:
            continue
        t = st["tables"][s, : _blocks(L, S)]
        k, v = _rows(st["k"], t, st["kv_scale"])[:L], _rows(st["v"], t, st["kv_scale"])[:L]
        q = st["q"][a:b].float().reshape(b - a, hkv, G, D)
        x = torch.einsum("nhgd,thd->nhgt", q, k) * st["scale"]
        e = torch.exp(x - x.amax(-1, keepdim=True))
        out[a:b] = (torch.einsum("nhgt,thd->nhgd", e, v) / e.sum(-1, keepdim=True)).reshape(b - a, hq, D)
    return out.to(torch.bfloat16)


def run(state):
    st = state
    if not own:
        return {"extend": _plain_extend, "release": _plain_release, "prefix": _plain_prefix,
                "cross": _plain_cross}[st["op"]](st)
    import paged_kv_cache_71_gb300 as pkv
    if st["op"] == "extend":
        pkv.pkv_extend_sequences(st["tables"], st["past"], st["new"], st["S"], st["free"], st["count"],
                                 st["seq_lens"], st["count_out"], st["slots"], st["cu_q"], st["q_starts"], st["err"])
        return [st["tables"], st["seq_lens"], st["count_out"], st["cu_q"], st["q_starts"], st["slots"]]
    if st["op"] == "release":
        pkv.pkv_release_sequences(st["tables"], st["past"], st["done"], st["S"], st["free"], st["count"],
                                  st["seq_lens"], st["count_out"], st["keep"], st["err"])
        return [st["free"], st["seq_lens"], st["count_out"]]
    if st["op"] == "prefix":
        pkv.pkv_paged_attention_decode_prefix(st["out"], st["q"], st["k"], st["v"], st["desc"], st["tables"],
                                              st["lens"], st["cu"], st["pre"], st["scale"], st["ws"], st["err"])
    else:
        pkv.pkv_paged_cross_attention(st["out"], st["q"], st["cu"], st["lens"], st["k"], st["v"], st["desc"],
                                      st["tables"], st["scale"], st["ws"], st["err"])
    return st["out"]


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    S = st["S"]
    if st["op"] == "extend":
        table, past, new = st["tables"].tolist(), st["past"].tolist(), st["new"].tolist()
        stack = st["free"].tolist()
        top, cu, slots = int(st["count"]), [0], []
        for s, (p, t) in enumerate(zip(past, new)):
            for pos in range(p, p + t):
                if pos % S == 0:
                    top -= 1
                    table[s][pos // S] = stack[top]
                slots.append(table[s][pos // S] * S + pos % S)
            cu.append(cu[-1] + t)
        slots += [-1] * (st["cap"] - len(slots))
        return [_i32(table), _i32([p + t for p, t in zip(past, new)]), _i32([top]), _i32(cu), _i32(past),
                torch.tensor(slots, dtype=torch.int64, device="cuda")]
    if st["op"] == "release":
        table, past, done, keep = (st[k].tolist() for k in ("tables", "past", "done", "keep"))
        stack, top = st["free"].tolist(), int(st["count"])
        for s, p in enumerate(past):
            for b in table[s][keep[s]:_blocks(p, S)] if done[s] else []:
                stack[top] = b
                top += 1
        return [_i32(stack), _i32([0 if d else p for p, d in zip(past, done)]), _i32([top])]
    # attention: every sequence by itself over all of its keys
    G = st["hq"] // st["hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, L in enumerate(st["lens_host"]):
        a, b = (s, s + 1) if st["op"] == "prefix" else (st["cu_host"][s], st["cu_host"][s + 1])
        if L == 0 or a == b:
            continue
        pos = torch.arange(L, device="cuda")
        blk = st["tables"][s].long()[pos // S]
        k = (st["k"][blk, pos % S].double() * st["kv_scale"]).permute(1, 2, 0)  # [heads, D, L]
        v = (st["v"][blk, pos % S].double() * st["kv_scale"]).permute(1, 0, 2)  # [heads, L, D]
        q = st["q"][a:b].double().reshape(b - a, st["hkv"], G, D).permute(1, 0, 2, 3).reshape(st["hkv"], -1, D)
        w = torch.softmax(torch.bmm(q, k) * st["scale"], dim=-1)
        o = torch.bmm(w, v).reshape(st["hkv"], b - a, G, D).permute(1, 0, 2, 3)
        out[a:b] = o.reshape(b - a, st["hq"], D)
    return out
