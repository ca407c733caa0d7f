"""Workloads of the operators of a serving step that never waits for the host:
block tables on the device, a cache of 8-bit codes with a scale for each block
and KV head, and the verification of drafted tokens. Each in a plain form
(elementary torch operations) and as a call of this library.

Five entry points of ``paged_kv_cache_141_gb300.binding``:

``extend_tables``    gives every request the blocks that its new tokens need from
    a stack of free blocks, and builds the slots and positions of those tokens.
``trim_tables``      takes a number of newest tokens from every request and puts the
    blocks that fall empty back on the stack.
``scaled_append``    writes new keys and values as E4M3 or 8-bit integer codes; each
    (block, KV head) has a scale of its own, which grows with its tokens.
``scaled_attention`` causal attention of one or several query tokens per sequence
    over such a cache.
``verify_drafts``    accepts drafted tokens against the target's probabilities, and
    draws the token after the last accepted one, from given random numbers.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
LEAST_SCALE = 2.0 ** -96


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # a handful of requests being generated: the smallest call, where launch latency is all
        _extend("tables: 4 requests, a token each", seqs=4, hi=1000, new=1),
        # a large batch with drafted tokens: five slots to each request
        _extend("tables: 512 requests, 5 tokens each", seqs=512, hi=8000, new=5),
        # a prompt step, ragged
        _extend("tables: 64 prompts of up to 4096", seqs=64, hi=0, new=4096, ragged=True),
        # the end of a step: rejected drafts given back, and every eighth request is done
        _trim("trim: 512 requests, contexts to 32k", seqs=512, hi=32768),
        # a decode step's append
        _append("append: 128 decode tokens, E4M3 codes", seqs=128, new=1, hi=512),
        # a prompt step's append; an odd chunk length ends inside blocks
        _append("append: 32 chunks of 1001, E4M3 codes", seqs=32, new=1001, hi=1400),
        # one long conversation: few rows, a long axis
        _attend("attend: one context of 131072, int8", seqs=1, lo=131072, hi=131072),
        # a decode step of a batch
        _attend("attend: 64 contexts of 512-8192, int8", seqs=64, lo=512, hi=8192),
        # four drafted tokens and the one before them, a larger group, binary16
        _attend("attend: 5 tokens, 64 contexts of 512-4096, E4M3", seqs=64, lo=512, hi=4096, new=5, q_heads=64, dtype="f16",
                cache="e4m3"),
        # prompt chunks over what the earlier chunks left
        _attend("attend: 8 chunks of 512 in contexts to 8k, int8", seqs=8, lo=1024, hi=8192, new=512),
        # one request's drafts
        _verify("verify: one request, 4 drafts of 32000", seqs=1, drafts=4, vocab=32000),
        # a batch's drafts over a large vocabulary
        _verify("verify: 256 requests, 4 drafts of 128256", seqs=256, drafts=4, vocab=128256),
    ]


def _extend(name, seqs, hi, new, ragged=False, block_size=16):
    return {"name": name, "op": "extend", "seqs": seqs, "hi": hi, "new": new, "ragged": ragged, "block_size": block_size}


def _trim(name, seqs, hi, block_size=16):
    return {"name": name, "op": "trim", "seqs": seqs, "hi": hi, "block_size": block_size}


def _append(name, seqs, new, hi, kv_heads=8, head_size=128, block_size=16, dtype="bf16", cache="e4m3"):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "hi": hi, "kv_heads": kv_heads,
            "head_size": head_size, "block_size": block_size, "dtype": dtype, "cache": cache}


def _attend(name, seqs, lo, hi, new=1, q_heads=32, kv_heads=8, head_size=128, block_size=16, dtype="bf16", cache="int8"):
    return {"name": name, "op": "attend", "seqs": seqs, "lo": lo, "hi": hi, "new": new, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_size": head_size, "block_size": block_size, "dtype": dtype, "cache": cache}


def _verify(name, seqs, drafts, vocab, sampled=True):
    return {"name": name, "op": "verify", "seqs": seqs, "drafts": drafts, "vocab": vocab, "sampled": sampled}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("extend", "trim", "append", "append", "attend", "attend", "attend", "verify"))
    block_size = rng.choice((8, 16, 16, 32, 64, 24))
    kv = {"head_size": rng.choice((64, 128, 128, 256)), "block_size": block_size, "dtype": rng.choice(("bf16", "bf16", "f16")),
          "cache": rng.choice(("int8", "e4m3"))}
    q_heads, kv_heads = rng.choice(((32, 8), (32, 32), (64, 8), (16, 4), (8, 1), (12, 2), (40, 8)))
    if op == "extend":
        seqs = _log(rng, 1, 512)
        c = _extend(None, seqs, _log(rng, 1, 16384), _log(rng, 1, min(4096, 131072 // seqs)), rng.random() < 0.5, block_size)
    elif op == "trim":
        c = _trim(None, _log(rng, 1, 512), _log(rng, 16, 32768), block_size)
    elif op == "append":
        seqs = _log(rng, 1, 128)
        budget = 32 * 1001 * 8 * 128 // (kv_heads * kv["head_size"])
        new = rng.choice((1, _log(rng, 1, max(1, min(1001, budget // seqs)))))
        c = _append(None, seqs, new, new + _log(rng, 1, 400), kv_heads, **kv)
    elif op == "attend":
        new = rng.choice((1, 1, rng.randint(2, 8), _log(rng, 9, 512)))
        hi = max(new, _log(rng, 16, 131072 if new < 9 else 8192))
        c = _attend(None, _log(rng, 1, 64), min(hi, max(new if new > 1 else 0, hi // rng.choice((1, 2, 8, 1 << 20)))), hi, new, q_heads,
                    kv_heads, **kv)
    else:
        c = _verify(None, _log(rng, 1, 256), rng.randint(0, 8), _log(rng, 1000, 128256), rng.random() < 0.8)
    # no costlier than the largest listed case, in bytes, in products, or in what the plain form holds at a time
    while c["seqs"] > 1 and (work(c)["bytes"] > 6e8 or work(c)["flops"] > 5e11
                             or (op == "attend" and c["seqs"] * c["hi"] * max(c["q_heads"] * c["new"], 2 * c["kv_heads"] * c["head_size"]) > 1.2e9)):
        c["seqs"] //= 2
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    return {"extend": _prepare_extend, "trim": _prepare_trim, "append": _prepare_append, "attend": _prepare_attend,
            "verify": _prepare_verify}[case["op"]](case, seed)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, device="cuda", dtype=dtype)


def _prepare_tables(c, seed, lens, room):
    """Requests of the given lengths in scattered blocks, and the stack of the blocks that none of them holds."""
    B, S, g = c["block_size"], c["seqs"], _gen(seed)
    most = -(-room // B)
    held = (lens + B - 1) // B
    perm = (torch.randperm(S * most, generator=g, device="cuda") + 1).to(torch.int32)
    table = perm.view(S, most).clone()
    taken = torch.arange(most, device="cuda") < held.view(S, 1)
    stack = torch.cat((perm[~taken.view(-1)], perm[taken.view(-1)]))         # above the free ones: stale entries
    return {"case": c, "block_tables": torch.where(taken, table, -1), "context_lens": lens.to(torch.int32), "free_blocks": stack,
            "num_free": _ints([int((~taken).sum())]), "new_lens": torch.empty(S, device="cuda", dtype=torch.int32),
            "new_num_free": _ints([0])}


def _prepare_extend(c, seed):
    r, S = random.Random(seed), c["seqs"]
    lens = _ints([r.randint(0, c["hi"]) for _ in range(S)], torch.int64)
    s = _prepare_tables(c, seed, lens, c["hi"] + c["new"])
    s["new_tokens"] = _ints([r.randint(0, c["new"]) if c["ragged"] else c["new"] for _ in range(S)])
    s["slots"] = torch.empty(S * c["new"], device="cuda", dtype=torch.int64)
    s["positions"] = torch.empty_like(s["slots"])
    s["query_start"] = torch.empty(S + 1, device="cuda", dtype=torch.int32)
    return s


def _prepare_trim(c, seed):
    r, S = random.Random(seed), c["seqs"]
    lens = [r.randint(1, c["hi"]) for _ in range(S)]
    s = _prepare_tables(c, seed, _ints(lens, torch.int64), c["hi"])
    s["drop"] = _ints([n if r.random() < 0.125 else min(n, r.randint(0, 4)) for n in lens])
    return s


def _heads_like(shape, dtype, g):
    """New or cached keys or values: unit variance with a few channels of larger spread, and tokens of different size."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    x.mul_(1 + 3 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.06).to(dtype))
    return x


def _fresh_scale(most, cache):
    """A block's scale for a largest magnitude: the largest code stands for it (integers), or the smallest power of two
    under which it does not pass the largest code (E4M3, whose codes then only move their exponents when a scale grows)."""
    if cache == "int8":
        scale = most / torch.full_like(most, 127)
    else:
        m, e = torch.frexp(most)                                             # 448 is 0.875 * 2^9
        scale = torch.ldexp(torch.ones_like(most), torch.where(m <= 0.875, e - 9, e - 8))
        scale = torch.where(most > 0, scale, 0.0)
    return scale.clamp(min=LEAST_SCALE)


def _coded(x, scale, cache):
    """Codes of x (32 bits) under a scale."""
    x = x / scale
    if cache == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _scaled_pool(shape, c, g):
    """A cache of codes and its scales [num_blocks, kv_heads]; blocks differ in size."""
    cache = torch.empty(shape, device="cuda", dtype=CODES[c["cache"]])
    scales = torch.empty(shape[:2], device="cuda")
    for at in range(0, shape[0], 16384):                                     # in parts, to bound the temporaries
        part = _heads_like((min(16384, shape[0] - at),) + shape[1:], torch.float32, g)
        part.mul_(torch.rand((part.shape[0], 1, 1, 1), generator=g, device="cuda") + 0.5)
        scale = _fresh_scale(part.abs().amax((2, 3)), c["cache"])
        scales[at:at + 16384] = scale
        cache[at:at + 16384] = _coded(part, scale.view(*scale.shape, 1, 1), c["cache"])
    return cache, scales


def _blocks(seqs, most, g):
    """A block table whose entries are scattered over the pool; block 0 stays reserved."""
    return (torch.randperm(seqs * most, generator=g, device="cuda") + 1).view(seqs, most).to(torch.int32), seqs * most + 1


def _prepare_append(c, seed):
    g, r, S = _gen(seed), random.Random(seed), c["seqs"]
    B, Q = c["block_size"], c["new"]
    lens = _ints([r.randint(Q, c["hi"]) for _ in range(S)])
    table, num_blocks = _blocks(S, -(-c["hi"] // B), g)
    shape = (num_blocks, c["kv_heads"], B, c["head_size"])
    (k_cache, k_scales), (v_cache, v_scales) = _scaled_pool(shape, c, g), _scaled_pool(shape, c, g)
    # one projection's output holds keys and values of every head; the two are views of it
    kv = _heads_like((S * Q, 2 * c["kv_heads"], c["head_size"]), DTYPES[c["dtype"]], g)
    k, v = kv.split(c["kv_heads"], dim=1)
    return {"case": c, "k": k, "v": v, "k_cache": k_cache, "v_cache": v_cache, "k_scales": k_scales, "v_scales": v_scales,
            "block_tables": table, "context_lens": lens, "query_start": torch.arange(S + 1, device="cuda", dtype=torch.int32) * Q}


def _prepare_attend(c, seed):
    g, r, S, Q = _gen(seed), random.Random(seed), c["seqs"], c["new"]
    B, D = c["block_size"], c["head_size"]
    lens = _ints([r.randint(c["lo"], c["hi"]) for _ in range(S)])
    table, num_blocks = _blocks(S, -(-c["hi"] // B), g)
    shape = (num_blocks, c["kv_heads"], B, D)
    (k_cache, k_scales), (v_cache, v_scales) = _scaled_pool(shape, c, g), _scaled_pool(shape, c, g)
    if c["cache"] == "e4m3":                # past each context's end lie an earlier request's codes, here E4M3's NaN
        full = lens > 0
        at = (lens.long() - 1).clamp(min=0)
        last = table.gather(1, (at // B).view(-1, 1)).view(-1).long()
        stale = (torch.arange(B, device="cuda").view(1, -1) > (at % B).view(-1, 1)) & full.view(-1, 1)
        for cache in (k_cache, v_cache):
            bits = cache.view(torch.uint8)
            bits[last] = bits[last].masked_fill(stale.view(S, 1, B, 1), 0x7F)
    query = torch.randn((S * Q, c["q_heads"], D), generator=g, device="cuda").to(DTYPES[c["dtype"]])
    return {"case": c, "query": query, "k_cache": k_cache, "v_cache": v_cache, "k_scales": k_scales, "v_scales": v_scales,
            "block_tables": table, "context_lens": lens, "scale": D ** -0.5, "out": torch.empty_like(query),
            "query_start": None if Q == 1 else torch.arange(S + 1, device="cuda", dtype=torch.int32) * Q}


def _prepare_verify(c, seed):
    g, S, K, V = _gen(seed), c["seqs"], c["drafts"], c["vocab"]
    # every request of a batch has drafts of its own number: the last is the fixed one, others may have fewer
    r = random.Random(seed)
    rows = [1 + (K if s == S - 1 else r.randint(max(0, K - 2), K)) for s in range(S)]
    start = _ints([0] + rows).cumsum(0).to(torch.int32)
    T = sum(rows)
    logits = torch.randn((T, V), generator=g, device="cuda") * 2.5
    target = torch.softmax(logits, -1)
    draft = None
    inside = (torch.arange(K, device="cuda").view(1, K) < _ints(rows).view(S, 1) - 1)
    tokens = torch.zeros((S, K), device="cuda", dtype=torch.int64)
    if K:
        at = start[:-1].long().view(S, 1) + torch.arange(K, device="cuda")
        draft = torch.empty((S, K, V), device="cuda")
        for i in range(K):                  # the drafter: the target's logits and some noise
            part = logits[at[:, i].clamp(max=T - 1)]
            draft[:, i] = torch.softmax(part + 0.8 * torch.randn(part.shape, generator=g, device="cuda"), -1)
        tokens = torch.multinomial(draft.view(S * K, V), 1, generator=g).view(S, K)
        tokens = torch.where(inside, tokens, -1)
    uniforms = torch.rand((S, K + 1), generator=g, device="cuda")
    return {"case": c, "target": target, "draft": draft if c["sampled"] else None, "drafted": tokens, "uniforms": uniforms,
            "query_start": start, "tokens": torch.empty((S, K + 1), device="cuda", dtype=torch.int64),
            "accepted": torch.empty(S, device="cuda", dtype=torch.int32)}


# ---------------------------------------------------------------- one pass

def run(state):
    return {"extend": _run_extend, "trim": _run_trim, "append": _run_append, "attend": _run_attend,
            "verify": _run_verify}[state["case"]["op"]](state)


def _run_extend(s):
    B = s["case"]["block_size"]
    if own:
        from paged_kv_cache_141_gb300 import binding as pk
        pk.extend_tables(s["block_tables"], s["context_lens"], s["new_tokens"], s["free_blocks"], s["num_free"], s["slots"],
                         s["query_start"], B, positions=s["positions"], new_lens=s["new_lens"], new_num_free=s["new_num_free"])
        return {k: s[k] for k in ("block_tables", "slots", "positions", "query_start", "new_lens", "new_num_free")}
    S, most = s["block_tables"].shape
    L, n, F = s["context_lens"].long(), s["new_tokens"].long(), s["num_free"].long()
    T = s["slots"].numel()
    n = torch.where((n >= 0) & (L + n <= most * B), n, 0)
    held = (L + B - 1) // B
    need = (L + n + B - 1) // B - held
    before = need.cumsum(0) - need
    n = torch.where(((before + need <= F) | (need == 0)) & (n.cumsum(0) <= T), n, 0)
    need = torch.where(n > 0, need, 0)
    s["query_start"][0] = 0
    s["query_start"][1:] = n.cumsum(0)
    # the blocks: request s takes the stack's topmost after those before it
    j = torch.arange(most, device="cuda")
    fresh = (j >= held.view(S, 1)) & (j < (held + need).view(S, 1))
    top = F - 1 - before.view(S, 1) - (j - held.view(S, 1))
    s["block_tables"].copy_(torch.where(fresh, s["free_blocks"][top.clamp(0, s["free_blocks"].numel() - 1)], s["block_tables"]))
    # every token's request, position and slot
    t = torch.arange(T, device="cuda")
    ends = s["query_start"][1:].long()
    mine = torch.searchsorted(ends, t, right=True).clamp(max=S - 1)
    there = t < ends[-1]
    at = torch.where(there, L[mine] + t - (ends[mine] - n[mine]), 0)
    slot = s["block_tables"][mine, at // B].long() * B + at % B
    s["slots"].copy_(torch.where(there, slot, -1))
    s["positions"].copy_(at)
    s["new_lens"].copy_(L + n)
    s["new_num_free"].copy_(F - need.sum())
    return {k: s[k] for k in ("block_tables", "slots", "positions", "query_start", "new_lens", "new_num_free")}


def _run_trim(s):
    B = s["case"]["block_size"]
    if own:
        from paged_kv_cache_141_gb300 import binding as pk
        pk.trim_tables(s["block_tables"], s["context_lens"], s["drop"], s["free_blocks"], s["num_free"], B, new_lens=s["new_lens"],
                       new_num_free=s["new_num_free"])
        return {k: s[k] for k in ("free_blocks", "new_lens", "new_num_free")}
    S, most = s["block_tables"].shape
    L, d, F = s["context_lens"].long(), s["drop"].long(), s["num_free"].long()
    kept = (L - d + B - 1) // B
    count = (L + B - 1) // B - kept
    before = count.cumsum(0) - count
    total = count.sum()
    # the first request's first block comes to lie on top, as extend_tables would take them again
    j = torch.arange(most, device="cuda")
    freed = (j >= kept.view(S, 1)) & (j < (kept + count).view(S, 1))
    place = F + total - 1 - before.view(S, 1) - (j - kept.view(S, 1))
    spare = s["free_blocks"].numel()
    stack = torch.cat((s["free_blocks"], s["free_blocks"][:1]))              # what is not freed goes to one place more
    stack[torch.where(freed, place, spare)] = s["block_tables"]
    s["free_blocks"].copy_(stack[:spare])
    s["new_lens"].copy_(L - d)
    s["new_num_free"].copy_(F + total)
    return {k: s[k] for k in ("free_blocks", "new_lens", "new_num_free")}


def _append_out(s):
    names = ("k_cache", "v_cache")
    scales = {"k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    if s["case"]["cache"] == "e4m3":
        return {**{k: s[k] for k in names}, **scales}
    dt = DTYPES[s["case"]["dtype"]]                                          # the values that the integers stand for
    return {**{k: (s[k].float() * s[k[0] + "_scales"].view(*s[k].shape[:2], 1, 1)).to(dt) for k in names}, **scales}


def _run_append(s):
    c = s["case"]
    if own:
        from paged_kv_cache_141_gb300 import binding as pk
        pk.scaled_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["block_tables"],
                         s["context_lens"], max_new_tokens=c["new"], query_start=s["query_start"])
        return _append_out(s)
    B, Q = c["block_size"], c["new"]
    L = s["context_lens"].long().view(-1, 1)
    first = L - Q                                                            # the first new position
    j = first // B + torch.arange((Q + B - 2) // B + 1, device="cuda")      # [S, J] touched blocks
    touched = j * B < L
    block = torch.where(touched, s["block_tables"].long().gather(1, j.clamp(max=s["block_tables"].shape[1] - 1)), 0)
    at = j.unsqueeze(-1) * B + torch.arange(B, device="cuda")               # [S, J, B] positions
    new = ((at >= first.unsqueeze(-1)) & (at < L.unsqueeze(-1))).view(*at.shape, 1, 1)
    old = (touched & (j * B < first)).unsqueeze(-1)                          # holds older tokens
    row = s["query_start"][:-1].long().view(-1, 1, 1) + (at - first.unsqueeze(-1)).clamp(0, Q - 1)
    for x, cache, scales in ((s["k"], s["k_cache"], s["k_scales"]), (s["v"], s["v_cache"], s["v_scales"])):
        x = x[row].float()                                                   # [S, J, B, H, D]
        fresh = _fresh_scale(torch.where(new, x.abs(), 0.0).amax((2, 4)), c["cache"])
        before = scales[block]
        scale = torch.where(old, torch.maximum(before, fresh), fresh)
        codes = cache[block].transpose(2, 3)
        wide = scale.unsqueeze(2).unsqueeze(-1)
        ratio = (before / scale).unsqueeze(2).unsqueeze(-1)
        older = codes.float() * ratio                                        # what was there, under the new scale
        older = older.round().to(torch.int8) if c["cache"] == "int8" else older.to(torch.float8_e4m3fn)
        there = old.unsqueeze(-1).unsqueeze(-1) & (at < first.unsqueeze(-1)).view(new.shape)
        bits = torch.where(there, older.view(torch.uint8), codes.view(torch.uint8))
        bits = torch.where(new, _coded(x, wide, c["cache"]).view(torch.uint8), bits)
        cache.view(torch.uint8)[block] = torch.where(touched.view(*j.shape, 1, 1, 1), bits.transpose(2, 3), cache.view(torch.uint8)[0])
        scales[block] = torch.where(touched.unsqueeze(-1), scale, scales[0])
    return _append_out(s)


def _run_attend(s):
    c = s["case"]
    S, Q, Hq, H, D, B = c["seqs"], c["new"], c["q_heads"], c["kv_heads"], c["head_size"], c["block_size"]
    if own:
        from paged_kv_cache_141_gb300 import binding as pk
        if "workspace" not in s:                                             # a serving loop keeps it from step to step
            s["workspace"] = pk.alloc_scaled_workspace(S, S * Q, Hq, H, D, Q, c["hi"])
        pk.scaled_attention(s["out"], s["query"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["block_tables"],
                            s["context_lens"], c["hi"], s["scale"], s["workspace"], query_start=s["query_start"],
                            max_queries_per_seq=Q)
        return {"out": s["out"]}
    G = Hq // H
    block, L = s["block_tables"].long(), s["context_lens"].long()
    at = torch.arange(block.shape[1] * B, device="cuda")
    inside = (at < L.view(S, 1)).view(S, 1, -1, 1)

    def values(cache, scales):
        x = cache[block].float() * scales[block].unsqueeze(-1).unsqueeze(-1)             # [S, J, H, B, D]
        return x.transpose(1, 2).flatten(2, 3).masked_fill_(~inside, 0.0)               # [S, H, J B, D]

    q = s["query"].float().view(S, Q, H, G, D).permute(0, 2, 1, 3, 4).reshape(S, H, Q * G, D)
    logits = q @ values(s["k_cache"], s["k_scales"]).transpose(2, 3)
    logits.mul_(s["scale"])
    seen = (L.view(S, 1) - Q + torch.arange(Q, device="cuda")).repeat_interleave(G, 1)   # [S, Q G]: a row's last key
    logits.masked_fill_((at > seen.unsqueeze(-1)).unsqueeze(1), -math.inf)
    logits.sub_(logits.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    total = logits.sum(-1, keepdim=True)
    out = logits @ values(s["v_cache"], s["v_scales"]) / torch.where(total > 0, total, 1.0)
    s["out"].copy_(out.view(S, H, Q, G, D).transpose(1, 2).reshape(S * Q, Hq, D))
    return {"out": s["out"]}


def _run_verify(s):
    c = s["case"]
    if own:
        from paged_kv_cache_141_gb300 import binding as pk
        pk.verify_drafts(s["tokens"], s["accepted"], s["target"], s["drafted"], s["uniforms"], s["query_start"],
                         draft_probs=s["draft"])
        return {"tokens": s["tokens"], "accepted": s["accepted"]}
    S, K, V = c["seqs"], c["drafts"], c["vocab"]
    start = s["query_start"].long()
    rows = start[1:] - start[:-1]
    i = torch.arange(K, device="cuda")
    token = s["drafted"].clamp(min=0)
    p = s["target"][(start[:-1].view(S, 1) + i).clamp(max=s["target"].shape[0] - 1), token].double()      # [S, K]
    q = s["draft"].gather(2, token.unsqueeze(-1)).squeeze(-1).double() if s["draft"] is not None else torch.ones_like(p)
    fine = (s["uniforms"][:, :K].double() * q < p) & (i < (rows - 1).view(S, 1))
    taken = fine.long().cumprod(1).sum(1)
    # the token after them: from the target's probabilities beyond the drafter's, or the target's own after the last draft
    left = s["target"][start[:-1] + taken].double()
    rejected = (taken < rows - 1).view(S, 1)
    if K:
        last = taken.clamp(max=K - 1)
        mine = torch.arange(S, device="cuda")
        if s["draft"] is not None:
            beyond = (left - s["draft"][mine, last].double()).clamp(min=0)
        else:
            beyond = left.scatter(1, token.gather(1, last.view(S, 1)), 0.0)
        left = torch.where(rejected & (beyond.sum(1, keepdim=True) > 0), beyond, left)
    sums = left.cumsum(1)
    goal = s["uniforms"][:, K:].double() * sums[:, -1:]
    drawn = torch.searchsorted(sums, goal, right=True).clamp(max=V - 1)
    at = torch.arange(K + 1, device="cuda")
    drafted = torch.cat((s["drafted"], drawn), 1)
    s["tokens"].copy_(torch.where(at < taken.view(S, 1), drafted, torch.where(at == taken.view(S, 1), drawn, -1)))
    s["accepted"].copy_(taken)
    return {"tokens": s["tokens"], "accepted": s["accepted"]}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    B, S = c["block_size"] if "block_size" in c else 0, c["seqs"]
    if c["op"] == "extend":
        tokens = S * c["new"] / (2 if c["ragged"] else 1)
        blocks = tokens / B
        return {"bytes": 16 * tokens + 8 * blocks + 8 * S * c["new"] * (2 if c["ragged"] else 0) / 2 + 20 * S, "flops": 4 * tokens}
    if c["op"] == "trim":
        return {"bytes": 8 * S * c["hi"] / 2 / B / 8 + 12 * S, "flops": S * c["hi"] / 2 / B / 8}
    if c["op"] == "append":
        w = 4 if c["dtype"] == "f32" else 2
        rows = S * c["kv_heads"] * c["head_size"]
        return {"bytes": 2 * rows * c["new"] * (w + 1) + 16 * S * c["kv_heads"] * (c["new"] / B + 1), "flops": 2 * rows * c["new"] * 2}
    if c["op"] == "attend":
        mean = (c["lo"] + c["hi"]) / 2
        rows = S * c["kv_heads"]
        Q, G = c["new"], c["q_heads"] // c["kv_heads"]
        seen = mean - (Q - 1) / 2
        return {"bytes": rows * (2 * mean * (c["head_size"] + 4 / B) + 4 * Q * G * c["head_size"]),
                "flops": 4 * rows * Q * G * max(1, seen) * c["head_size"]}
    # the accept test reads single values; one row of each request is drawn from
    V = c["vocab"]
    return {"bytes": S * V * 4 * (2 if c["sampled"] and c["drafts"] else 1) + 20 * S * (c["drafts"] + 1), "flops": 3 * S * V}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"extend": _exact_extend, "trim": _exact_trim, "append": _exact_append, "attend": _exact_attend,
            "verify": _exact_verify}[case["op"]](s, case)


def _exact_extend(s, c):
    B, table = c["block_size"], s["block_tables"].cpu()
    stack = s["free_blocks"].tolist()[:int(s["num_free"])]
    slots, positions, start, lens = [], [], [0], []
    for r, (L, n) in enumerate(zip(s["context_lens"].tolist(), s["new_tokens"].tolist())):
        for at in range(L, L + n):
            if at % B == 0:
                table[r, at // B] = stack.pop()
            positions.append(at)
            slots.append(int(table[r, at // B]) * B + at % B)
        start.append(len(slots))
        lens.append(L + n)
    pad = s["slots"].numel() - len(slots)
    return {"block_tables": table, "slots": torch.tensor(slots + [-1] * pad), "positions": torch.tensor(positions + [0] * pad),
            "query_start": torch.tensor(start, dtype=torch.int32), "new_lens": torch.tensor(lens, dtype=torch.int32),
            "new_num_free": torch.tensor([len(stack)], dtype=torch.int32)}


def _exact_trim(s, c):
    B, table = c["block_size"], s["block_tables"].tolist()
    stack, free = s["free_blocks"].tolist(), int(s["num_free"])
    back, lens = [], []
    for row, L, d in zip(table, s["context_lens"].tolist(), s["drop"].tolist()):
        back += row[-(-(L - d) // B):-(-L // B)]
        lens.append(L - d)
    stack[free:free + len(back)] = back[::-1]
    return {"free_blocks": torch.tensor(stack, dtype=torch.int32), "new_lens": torch.tensor(lens, dtype=torch.int32),
            "new_num_free": torch.tensor([free + len(back)], dtype=torch.int32)}


def _exact_append(s, c):
    """E4M3: what the codes are nearest to, before any rounding. Integers: the values that they stand for."""
    B, Q, code = c["block_size"], c["new"], c["cache"]
    out = {}
    tables, lens = s["block_tables"].tolist(), s["context_lens"].tolist()
    for name, x in (("k", s["k"]), ("v", s["v"])):
        pool, scales = s[name + "_cache"].double(), s[name + "_scales"].double()
        x = x.double()
        for r, (table, L) in enumerate(zip(tables, lens)):
            for b in range((L - Q) // B, (L - 1) // B + 1):
                lo, hi = max(L - Q, b * B), min(L, (b + 1) * B)
                rows = x[r * Q + lo - (L - Q):r * Q + hi - (L - Q)].transpose(0, 1)      # [H, tokens, D]
                most = rows.abs().amax((1, 2))
                if code == "int8":
                    scale = most / 127
                else:
                    scale = torch.exp2(torch.ceil(torch.log2(most / 448)))
                    scale = torch.where(most <= 224 * scale, scale / 2, scale)           # the logarithm rounds
                scale = scale.clamp(min=LEAST_SCALE)
                id_ = table[b]
                if lo > b * B:
                    scale = torch.maximum(scale, scales[id_])
                    pool[id_, :, :lo - b * B] *= (scales[id_] / scale).view(-1, 1, 1)
                pool[id_, :, lo - b * B:hi - b * B] = rows / scale.view(-1, 1, 1)
                if code == "int8":
                    pool[id_] = pool[id_].round()
                scales[id_] = scale
        out[name + "_cache"] = pool if code == "e4m3" else pool * scales.view(*scales.shape, 1, 1)
        out[name + "_scales"] = scales
    return out


def _exact_attend(s, c):
    Q, H, B, D = c["new"], c["kv_heads"], c["block_size"], c["head_size"]
    G, lens = c["q_heads"] // H, s["context_lens"].tolist()
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device="cuda")
    for r, L in enumerate(lens):
        if L == 0:
            continue
        ids = s["block_tables"][r, :-(-L // B)].long()
        k, v = ((cache[ids].double() * scales[ids].double().view(-1, H, 1, 1)).permute(1, 0, 2, 3).reshape(H, -1, D)[:, :L]
                for cache, scales in ((s["k_cache"], s["k_scales"]), (s["v_cache"], s["v_scales"])))
        hidden = torch.ones((Q, L), dtype=torch.bool, device="cuda").triu(L - Q + 1)
        for g in range(G):
            q = s["query"][r * Q:(r + 1) * Q, g::G].double().transpose(0, 1)             # [H, Q, D]
            score = torch.einsum("hqd,hkd->hqk", q, k) * s["scale"]
            p = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            out[r * Q:(r + 1) * Q, g::G] = torch.einsum("hqk,hkd->qhd", p, v)
    return {"out": out}


def _exact_verify(s, c):
    K, V = c["drafts"], c["vocab"]
    start, drafted, u = s["query_start"].tolist(), s["drafted"].tolist(), s["uniforms"].double().tolist()
    tokens, accepted = [], []
    for r in range(c["seqs"]):
        n = start[r + 1] - start[r] - 1
        row, got = start[r], []
        while len(got) < n:
            t = drafted[r][len(got)]
            q = 1.0 if s["draft"] is None else float(s["draft"][r, len(got), t])
            if not u[r][len(got)] * q < float(s["target"][row + len(got), t]):
                break
            got.append(t)
        p = s["target"][row + len(got)].double()
        if len(got) < n:
            other = torch.zeros_like(p)
            if s["draft"] is None:
                other[drafted[r][len(got)]] = math.inf
            else:
                other = s["draft"][r, len(got)].double()
            beyond = torch.relu(p - other)
            p = beyond if bool(beyond.any()) else p
        sums = torch.cumsum(p, 0)
        drawn = min(V - 1, int((sums <= u[r][K] * sums[-1]).sum()))
        accepted.append(len(got))
        tokens.append(got + [drawn] + [-1] * (K - len(got)))
    return {"tokens": torch.tensor(tokens), "accepted": torch.tensor(accepted, dtype=torch.int32)}
