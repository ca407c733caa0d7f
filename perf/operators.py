"""Workloads of the position-rotating KV append, the key-bound summaries and
the block-sparse decode, each in a plain form (elementary torch operations)
and as a call of this library.

Three entry points of ``paged_kv_cache_141_gb300.binding``:

``rope_and_cache``  rotates the new tokens' queries and keys by their
    positions (one axis, or several with an axis for each frequency),
    optionally after an RMS norm of each head, writes the queries out and
    appends the keys and values to the paged cache.
``key_bounds``      the elementwise minimum and maximum of the keys of every
    cache block that holds a new token.
``sparse_decode``   scores every block of a context by the largest value that
    q.k can take within its bounds, selects the best ones for each (sequence,
    KV head) beside the first and the newest, and attends to those.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def _bytes(dtype):
    return {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}[dtype]


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one request being generated: the smallest call, where launch latency is all
        _append("append: one token, GQA bf16", seqs=1, chunk=1, q_heads=32, kv_heads=8),
        # one decode step of a large batch
        _append("append: 256 decode tokens, GQA bf16", seqs=256, chunk=1, q_heads=32, kv_heads=8),
        # a step of prompt chunks, multi-head attention in binary16
        _append("append: 16 chunks of 512, MHA fp16", seqs=16, chunk=512, q_heads=32, kv_heads=32, dtype="f16"),
        # decode step of a model with query/key norms on an E4M3 pool
        _append("append+norm: 128 decode tokens, E4M3 pool", seqs=128, chunk=1, q_heads=64, kv_heads=8, cache="e4m3",
                norm=True),
        # a large prompt step with norms; an odd chunk length ends inside blocks
        _append("append+norm: 32 chunks of 1001, GQA bf16", seqs=32, chunk=1001, q_heads=32, kv_heads=8, norm=True),
        # one image-and-text prompt, three position axes, odd length
        _append("append, 3 axes: one prompt of 1373, bf16", seqs=1, chunk=1373, q_heads=32, kv_heads=8, axes=3),
        # a batch of video prompts: norms, three axes, neighbouring pairs, half of each head rotated
        _append("append+norm, 3 axes: 8 x 2048, pairs, fp16", seqs=8, chunk=2048, q_heads=32, kv_heads=8, dtype="f16",
                norm=True, axes=3, adjacent=True, rotary=64),
        # one decode step: only the newest block of each sequence changes
        _bounds("bounds: 64 sequences, newest block, bf16", seqs=64, new=1, lo=512, hi=4096),
        # after a prompt step of an E4M3 pool
        _bounds("bounds: 32 chunks of 1000, E4M3 pool", seqs=32, new=1000, lo=1000, hi=4096, cache="e4m3"),
        # one long conversation: few rows, a long axis
        _sparse("sparse: one context of 131072, bf16", seqs=1, lo=131072, hi=131072, select=128),
        # a batch of long contexts
        _sparse("sparse: 64 contexts of 8k-32k, bf16", seqs=64, lo=8192, hi=32768, select=64, first=1, recent=4),
        # larger groups on an E4M3 pool, ragged contexts, some shorter than the selection
        _sparse("sparse: 128 contexts of 100-8k, E4M3 pool", seqs=128, lo=100, hi=8192, q_heads=64, select=96,
                cache="e4m3", recent=2),
    ]


def _append(name, seqs, chunk, q_heads, kv_heads, head_size=128, rotary=None, block_size=16, dtype="bf16",
            cache="same", norm=False, axes=1, adjacent=False, max_position=16384):
    return {"name": name, "op": "append", "seqs": seqs, "chunk": chunk, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_size": head_size, "rotary": rotary or head_size, "block_size": block_size, "dtype": dtype,
            "cache": cache, "norm": norm, "axes": axes, "adjacent": adjacent, "max_position": max_position}


def _bounds(name, seqs, new, lo, hi, kv_heads=8, head_size=128, block_size=16, dtype="bf16", cache="same"):
    return {"name": name, "op": "bounds", "seqs": seqs, "new": new, "lo": lo, "hi": hi, "kv_heads": kv_heads,
            "head_size": head_size, "block_size": block_size, "dtype": dtype, "cache": cache}


def _sparse(name, seqs, lo, hi, select, q_heads=32, kv_heads=8, head_size=128, block_size=16, dtype="bf16",
            cache="same", first=1, recent=1):
    return {"name": name, "op": "sparse", "seqs": seqs, "lo": lo, "hi": hi, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_size": head_size, "block_size": block_size, "dtype": dtype, "cache": cache, "select": select,
            "first": first, "recent": recent}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "append", "append", "bounds", "sparse", "sparse"))
    dtype = rng.choice(("bf16", "bf16", "f16"))
    cache = rng.choice(("same", "same", "e4m3"))
    head_size = rng.choice((64, 128, 128, 256))
    block_size = rng.choice((16, 16, 32))
    q_heads, kv_heads = rng.choice(((32, 8), (32, 32), (64, 8), (16, 4), (8, 1), (12, 2)))
    if op == "append":
        seqs = _log(rng, 1, 256)
        budget = 32 * 1001 * 48 * 128 // ((q_heads + 2 * kv_heads) * head_size)
        c = _append(None, seqs, _log(rng, 1, max(1, min(2048, budget // seqs))), q_heads, kv_heads, head_size,
                    rng.choice((head_size, head_size, head_size // 2)), block_size, dtype, cache,
                    rng.random() < 0.5, rng.choice((1, 1, 3)), rng.random() < 0.3)
    elif op == "bounds":
        hi = _log(rng, 64, 4096)
        c = _bounds(None, _log(rng, 1, 128), rng.choice((1, _log(rng, 1, min(1000, hi // 2)))), hi // 2, hi, kv_heads,
                    head_size, block_size, dtype, cache)
    else:
        hi = _log(rng, 256, 131072)
        most = 64 * 32768 * 8 * 128 // (hi * kv_heads * head_size)
        first, recent = rng.choice((0, 1, 2)), rng.choice((1, 2, 4))
        c = _sparse(None, _log(rng, 1, max(1, min(128, most))), max(1, hi // rng.choice((2, 4, 8))), hi,
                    _log(rng, 8, 128), q_heads, kv_heads, head_size, block_size, dtype, cache, first, recent)
    while c["seqs"] > 1 and work(c)["bytes"] > 6e8:               # no costlier than the largest listed case
        c["seqs"] //= 2
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _blocks(per_seq, g):
    """A block table [seqs, most] whose entries are scattered over the pool; block 0 stays reserved."""
    seqs, most = len(per_seq), max(per_seq)
    perm = torch.randperm(seqs * most, generator=g, device="cuda") + 1
    return perm.view(seqs, most).to(torch.int32), seqs * most + 1


def _keys(shape, dtype, cache, g):
    """Cached keys or values: unit variance with a few channels of larger mean and spread, as rotated keys have."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16 if dtype == "bf16" or cache == "e4m3" else DTYPES[dtype])
    gain = 1 + 2 * (torch.rand(shape[-1], generator=g, device="cuda") < 0.06).to(x.dtype)
    x.mul_(gain)
    if cache == "e4m3":
        return x.mul_(30).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return x


def prepare(case, seed):
    return {"append": _prepare_append, "bounds": _prepare_bounds, "sparse": _prepare_sparse}[case["op"]](case, seed)


def _prepare_append(c, seed):
    g, r = _gen(seed), random.Random(seed)
    B, D, T = c["block_size"], c["head_size"], c["seqs"] * c["chunk"]
    dt = DTYPES[c["dtype"]]
    start = [r.randrange(0, c["max_position"] - c["chunk"] + 1) for _ in range(c["seqs"])]
    table, num_blocks = _blocks([-(-(c["chunk"] + B) // B)] * c["seqs"], g)
    at = torch.tensor(start, device="cuda").view(-1, 1)
    step = torch.arange(c["chunk"], device="cuda").view(1, -1)
    inside = at % B + step
    slots = table.gather(1, inside // B).long() * B + inside % B
    if c["chunk"] > 1:                      # the last prompt's last token is padding
        slots[-1, -1] = -1
    positions = (at + step).view(-1)
    freq_axes = None
    if c["axes"] > 1:                       # an image of rows of 37 patches: time stands still, height and width run
        wide = step.expand(c["seqs"], -1)
        positions = torch.stack(((at + 0 * wide).reshape(-1), (wide // 37).reshape(-1), (wide % 37).reshape(-1)))
        half = c["rotary"] // 2
        freq_axes = [0] * (half // 4) + [1] * (half * 3 // 8)
        freq_axes += [2] * (half - len(freq_axes))
    inv = 500000.0 ** (-torch.arange(0, c["rotary"], 2, device="cuda", dtype=torch.float64) / c["rotary"])
    angle = torch.arange(c["max_position"], device="cuda", dtype=torch.float64).view(-1, 1) * inv
    cos_sin = torch.cat((angle.cos(), angle.sin()), 1).float()
    # one projection's output holds every head of queries, keys and values; the three are views of it
    heads = c["q_heads"] + 2 * c["kv_heads"]
    qkv = torch.randn((T, heads, D), generator=g, device="cuda").to(dt)
    q, k, v = qkv.split((c["q_heads"], c["kv_heads"], c["kv_heads"]), dim=1)
    weight = [1 + 0.2 * torch.randn(D, generator=g, device="cuda") if c["norm"] else None for _ in range(2)]
    shape = (num_blocks, c["kv_heads"], B, D)
    return {"case": c, "q": q, "k": k, "v": v, "q_out": torch.empty((T, c["q_heads"], D), device="cuda", dtype=dt),
            "k_cache": _keys(shape, c["dtype"], c["cache"], g), "v_cache": _keys(shape, c["dtype"], c["cache"], g),
            "cos_sin": cos_sin, "positions": positions.contiguous(), "freq_axes": freq_axes,
            "axis": torch.tensor(freq_axes or [0] * (c["rotary"] // 2), device="cuda"),
            "slots": slots.view(-1).contiguous(), "q_weight": weight[0], "k_weight": weight[1],
            "k_scale": 0.011, "v_scale": 0.013}


def _lengths(c, seed):
    r = random.Random(seed)
    return [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]


def _pool(c, seed, g):
    B, lens = c["block_size"], _lengths(c, seed)
    table, num_blocks = _blocks([-(-c["hi"] // B)] * c["seqs"], g)
    context = torch.tensor(lens, device="cuda", dtype=torch.int32)
    return table, context, (num_blocks, c["kv_heads"], B, c["head_size"])


def _prepare_bounds(c, seed):
    g = _gen(seed)
    table, context, shape = _pool(c, seed, g)
    new = None if c["new"] == 1 else torch.minimum(torch.full_like(context, c["new"]), context)
    k_cache = _keys(shape, c["dtype"], c["cache"], g)
    k_bounds = torch.randn((shape[0], shape[1], 2, shape[3]), generator=g, device="cuda").to(DTYPES[c["dtype"]])
    return {"case": c, "k_cache": k_cache, "k_bounds": k_bounds, "block_tables": table, "context_lens": context,
            "new_tokens": new}


def _prepare_sparse(c, seed):
    g = _gen(seed)
    table, context, shape = _pool(c, seed, g)
    S, B, D = c["seqs"], c["block_size"], c["head_size"]
    k_cache, v_cache = (_keys(shape, c["dtype"], c["cache"], g) for _ in range(2))
    dt = DTYPES[c["dtype"]]
    k_bounds = torch.empty((shape[0], shape[1], 2, D), device="cuda", dtype=dt)
    for at in range(0, shape[0], 65536):    # in parts, to bound the temporary
        part = k_cache[at:at + 65536].to(dt)
        k_bounds[at:at + 65536, :, 0] = part.amin(2)
        k_bounds[at:at + 65536, :, 1] = part.amax(2)
    # the slots past each context's end hold what an earlier request left, here NaN
    last = table.gather(1, ((context.long() - 1) // B).view(-1, 1)).view(-1).long()
    stale = torch.arange(B, device="cuda").view(1, -1) > ((context.long() - 1) % B).view(-1, 1)
    for cache in (k_cache, v_cache):
        bits = cache.view(torch.uint8) if c["cache"] == "e4m3" else cache
        nan = 0x7F if c["cache"] == "e4m3" else float("nan")
        bits[last] = bits[last].masked_fill(stale.view(S, 1, B, 1), nan)
    query = torch.randn((S, c["q_heads"], D), generator=g, device="cuda").to(dt)
    state = {"case": c, "query": query, "k_cache": k_cache, "v_cache": v_cache, "k_bounds": k_bounds,
             "block_tables": table, "context_lens": context, "scale": D ** -0.5, "out": torch.empty_like(query),
             "selected": torch.empty((S, c["kv_heads"], c["select"]), device="cuda", dtype=torch.int32),
             "k_scale": 0.033 if c["cache"] == "e4m3" else 1.0, "v_scale": 0.033 if c["cache"] == "e4m3" else 1.0}
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    return {"append": _run_append, "bounds": _run_bounds, "sparse": _run_sparse}[state["case"]["op"]](state)


def _run_append(s):
    c = s["case"]
    if own:
        from paged_kv_cache_141_gb300 import binding as pk
        pk.rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["cos_sin"], s["positions"],
                          s["slots"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                          freq_axes=s["freq_axes"], adjacent_pairs=c["adjacent"], k_scale=s["k_scale"],
                          v_scale=s["v_scale"])
        return {"query": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    R, half = c["rotary"], c["rotary"] // 2
    if c["axes"] > 1:
        rows = s["positions"][s["axis"]].t()                       # [T, R/2]: each frequency's position
        columns = torch.arange(half, device="cuda")
        cos, sin = s["cos_sin"][rows, columns], s["cos_sin"][rows, columns + half]
    else:
        cos, sin = s["cos_sin"][s["positions"]].split(half, dim=1)
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
        if c["adjacent"]:
            a, b = x[..., 0:R:2], x[..., 1:R:2]
            pair = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = x[..., :half], x[..., half:R]
            pair = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((pair, x[..., R:]), -1)

    s["q_out"].copy_(turned(s["q"], s["q_weight"]))
    B, kept = c["block_size"], s["slots"] >= 0
    slots = s["slots"].clamp(min=0)                                # padding rewrites the reserved block's first slot
    for cache, x, scale in ((s["k_cache"], turned(s["k"], s["k_weight"]), s["k_scale"]),
                            (s["v_cache"], s["v"].float(), s["v_scale"])):
        if c["cache"] == "e4m3":
            x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            cache = cache.view(torch.uint8)
        else:
            x = x.to(cache.dtype)
        cache[slots // B, :, slots % B] = torch.where(kept.view(-1, 1, 1), x, cache[0, :, 0])
    return {"query": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _run_bounds(s):
    c = s["case"]
    if own:
        from paged_kv_cache_141_gb300 import binding as pk
        pk.key_bounds(s["k_bounds"], s["k_cache"], s["block_tables"], s["context_lens"], c["hi"],
                      new_tokens=s["new_tokens"], max_new_tokens=c["new"])
        return {"k_bounds": s["k_bounds"]}
    B = c["block_size"]
    L = s["context_lens"].long().view(-1, 1)
    new = 1 if s["new_tokens"] is None else s["new_tokens"].long().view(-1, 1)
    j = (L - new) // B + torch.arange((c["new"] + B - 2) // B + 1, device="cuda")
    touched = j * B < L
    block = torch.where(touched, s["block_tables"].long().gather(1, j.clamp(max=s["block_tables"].shape[1] - 1)), 0)
    keys = s["k_cache"][block].float()                             # [S, J, Hkv, B, D]
    there = (j.unsqueeze(-1) * B + torch.arange(B, device="cuda") < L.unsqueeze(-1)).view(*j.shape, 1, B, 1)
    low = keys.masked_fill(~there, math.inf).amin(3)
    high = keys.masked_fill(~there, -math.inf).amax(3)
    both = torch.stack((low, high), 3).to(s["k_bounds"].dtype)
    s["k_bounds"][block] = torch.where(touched.view(*j.shape, 1, 1, 1), both, s["k_bounds"][0])
    return {"k_bounds": s["k_bounds"]}


def _run_sparse(s):
    c = s["case"]
    if own:
        from paged_kv_cache_141_gb300 import binding as pk
        if "workspace" not in s:                                   # a serving loop keeps it from step to step
            s["workspace"] = pk.alloc_sparse_workspace(c["seqs"], c["q_heads"], c["kv_heads"], c["head_size"],
                                                       c["block_size"], c["hi"], c["select"])
        pk.sparse_decode(s["out"], s["query"], s["k_cache"], s["v_cache"], s["k_bounds"], s["block_tables"],
                         s["context_lens"], c["hi"], s["scale"], c["select"], s["workspace"],
                         first_blocks=c["first"], recent_blocks=c["recent"], selected=s["selected"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"out": s["out"], "selected": s["selected"]}
    S, H, D, B, K = c["seqs"], c["kv_heads"], c["head_size"], c["block_size"], c["select"]
    G = c["q_heads"] // H
    table, L = s["block_tables"].long(), s["context_lens"].long()
    n, j = ((L + B - 1) // B).view(S, 1, 1), torch.arange(table.shape[1], device="cuda")
    # the scores in 64 bits: two blocks next to the border may be closer than 32 bits tell apart
    q = s["query"].double().view(S, H, G, D)
    sides = torch.cat((q.clamp(max=0), q.clamp(min=0)), -1)        # negative parts meet the minimum, others the maximum
    bounds = s["k_bounds"][table].flatten(3).permute(0, 2, 3, 1).double()          # [S, H, 2 D, blocks]
    score = (sides @ bounds).amax(2)
    score = score.masked_fill((j < c["first"]) | (j >= n - c["recent"]), math.inf).masked_fill(j >= n, -math.inf)
    best = score.sort(dim=-1, descending=True, stable=True).indices[..., :K]
    if best.shape[-1] < K:
        best = torch.nn.functional.pad(best, (0, K - best.shape[-1]), value=table.shape[1])
    best = torch.where(torch.arange(K, device="cuda") < n, best, table.shape[1]).sort(-1).values
    s["selected"].copy_(torch.where(best < table.shape[1], best, -1))
    # attention over the selected blocks
    block = table.unsqueeze(1).expand(S, H, -1).gather(2, best.clamp(max=table.shape[1] - 1))
    head = torch.arange(H, device="cuda").view(1, H, 1)
    there = (best.unsqueeze(-1) * B + torch.arange(B, device="cuda") < L.view(S, 1, 1, 1)).flatten(2)   # [S, H, K B]
    k, v = (x[block, head].flatten(2, 3).float().masked_fill(~there.unsqueeze(-1), 0.0) for x in (s["k_cache"], s["v_cache"]))
    logits = s["query"].float().view(S, H, G, D) @ k.transpose(2, 3) * (s["scale"] * s["k_scale"])
    logits = logits.masked_fill(~there.unsqueeze(2), -math.inf)
    p = (logits - logits.amax(-1, keepdim=True)).exp()
    out = (p @ v) / p.sum(-1, keepdim=True) * s["v_scale"]
    s["out"].copy_(out.view(S, c["q_heads"], D))
    return {"out": s["out"], "selected": s["selected"]}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    w = _bytes(c["dtype"])
    kept = _bytes("e4m3") if c["cache"] == "e4m3" else w
    D = c["head_size"]
    if c["op"] == "append":
        T = c["seqs"] * c["chunk"]
        rows = 2 * c["q_heads"] * w + 2 * c["kv_heads"] * (w + kept)
        table = min(T, c["max_position"]) * c["rotary"] * 4
        return {"bytes": T * (rows * D + 8 + 8 * c["axes"]) + table,
                "flops": T * (c["q_heads"] + c["kv_heads"]) * (3 * c["rotary"] + (4 * D if c["norm"] else 0))}
    B = c["block_size"]
    mean = (c["lo"] + c["hi"]) / 2
    if c["op"] == "bounds":
        tokens = min(c["new"], mean) + B / 2                       # the touched blocks' tokens, on average
        blocks = (tokens + B - 1) // B
        rows = c["seqs"] * c["kv_heads"] * D
        return {"bytes": rows * (tokens * kept + 2 * blocks * w), "flops": 2 * rows * tokens}
    blocks = mean / B
    picked = min(blocks, c["select"])
    rows = c["seqs"] * c["kv_heads"] * D
    G = c["q_heads"] // c["kv_heads"]
    scored = blocks if c["select"] < blocks else 0
    return {"bytes": rows * (2 * scored * w + 2 * picked * B * kept + 2 * G * w) + 4 * c["seqs"] * (blocks + c["kv_heads"] * c["select"]),
            "flops": rows * G * (2 * scored + 4 * picked * B)}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "bounds": _exact_bounds, "sparse": _exact_sparse}[case["op"]](s, case)


def _exact_append(s, c):
    R, half, T = c["rotary"], c["rotary"] // 2, s["q"].shape[0]
    # frequency i of token t as one complex number
    positions = s["positions"].view(c["axes"], T)
    turn = torch.empty((T, half), dtype=torch.complex128, device="cuda")
    for i in range(half):
        row = s["cos_sin"][positions[int(s["axis"][i])]].double()
        turn[:, i] = torch.complex(row[:, i], row[:, half + i])

    def rows(x, weight):
        x = x.double()
        if weight is not None:
            norm = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
            x = x / (norm * norm / c["head_size"] + EPS).sqrt() * weight.double()
        y = x.clone()
        first = slice(0, R, 2) if c["adjacent"] else slice(0, half)
        second = slice(1, R, 2) if c["adjacent"] else slice(half, R)
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn.unsqueeze(1)
        y[..., first], y[..., second] = z.real, z.imag
        return y

    caches = []
    kept = s["slots"] >= 0
    at = s["slots"][kept]
    for cache, x, scale in ((s["k_cache"], rows(s["k"], s["k_weight"]), s["k_scale"]), (s["v_cache"], s["v"].double(), s["v_scale"])):
        pool = cache.double()
        flat = pool.transpose(1, 2).reshape(-1, c["kv_heads"], c["head_size"])
        flat[at] = (x / scale).clamp(-448, 448)[kept] if c["cache"] == "e4m3" else x[kept]
        caches.append(flat.view(pool.shape[0], c["block_size"], c["kv_heads"], c["head_size"]).transpose(1, 2).contiguous())
    return {"query": rows(s["q"], s["q_weight"]), "k_cache": caches[0], "v_cache": caches[1]}


def _exact_bounds(s, c):
    B, out = c["block_size"], s["k_bounds"].double()
    tables, lens = s["block_tables"].tolist(), s["context_lens"].tolist()
    new = [1] * len(lens) if s["new_tokens"] is None else s["new_tokens"].tolist()
    for table, L, m in zip(tables, lens, new):
        ends = list(range((L - m) // B, (L - 1) // B + 1))
        whole = [b for b in ends if (b + 1) * B <= L]
        at = torch.tensor([table[b] for b in whole], device="cuda", dtype=torch.long)
        keys = s["k_cache"][at].double().sort(dim=2).values
        out[at] = torch.stack((keys[:, :, 0], keys[:, :, -1]), 2)
        for b in set(ends) - set(whole):
            keys = s["k_cache"][table[b]][:, :L - b * B].double().sort(dim=1).values
            out[table[b]] = torch.stack((keys[:, 0], keys[:, -1]), 1)
    return {"k_bounds": out}


def _exact_sparse(s, c):
    B, H, D, K = c["block_size"], c["kv_heads"], c["head_size"], c["select"]
    G, lens = c["q_heads"] // H, s["context_lens"].tolist()
    out = torch.zeros(s["query"].shape, dtype=torch.float64, device="cuda")
    selected = torch.full(s["selected"].shape, -1, dtype=torch.int32)
    for r, L in enumerate(lens):
        n = -(-L // B)
        table = s["block_tables"][r, :n].long()
        q = s["query"][r].double().view(H, G, 1, D)
        low, high = s["k_bounds"][table].double().permute(2, 1, 0, 3).unsqueeze(2)      # [H, 1, n, D] each
        score = torch.stack([torch.maximum(q[h] * low[h], q[h] * high[h]).sum(-1).amax(0) for h in range(H)]).cpu()
        for h in range(H):
            always = set(range(min(c["first"], n))) | set(range(max(0, n - c["recent"]), n))
            rest = sorted((-x, b) for b, x in enumerate(score[h].tolist()) if b not in always)
            mine = sorted(always | {b for _, b in rest[:max(0, K - len(always))]}) if n > K else list(range(n))
            selected[r, h, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            at = table[torch.tensor(mine, device="cuda")]
            tokens = len(mine) * B - (n * B - L)                   # the newest block is the last, and may be partial
            k, v = (x[at, h].reshape(-1, D)[:tokens].double() for x in (s["k_cache"], s["v_cache"]))
            p = torch.softmax(q[h, :, 0] @ k.t() * (s["scale"] * s["k_scale"]), -1)
            out[r, h * G:(h + 1) * G] = p @ v * s["v_scale"]
    return {"out": out, "selected": selected.cuda()}
