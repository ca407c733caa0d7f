"""Plain forms, in 64 bits, of the calls of a step that does not wait for the
host: tables from lengths, block-scaled codes and attention over them, draft
verification. Everything on the CPU, one request at a time."""
from __future__ import annotations

import math

import torch

CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
LARGEST = {"e4m3": 448, "int8": 127}
LEAST_SCALE = 2.0 ** -96


def table_of(seqs, most, seed=0):
    """Scattered block ids [seqs, most], none of them 0, and the pool's size."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randperm(seqs * most, generator=g) + 1).view(seqs, most).to(torch.int32), seqs * most + 1


# ------------------------------------------------------------------ tables

def extend(table, lens, new, stack, free, B, room):
    """(table, slots, positions, starts, lens, free, denied requests)"""
    table = table.clone()
    slots, positions, starts, out, denied = [], [], [0], [], []
    asked, needed, F = 0, 0, free
    for s, (L, n) in enumerate(zip(lens, new)):
        fine = L >= 0 and n >= 0 and L + n <= table.shape[1] * B
        want = n if fine else 0
        need = -(-(L + want) // B) - -(-L // B) if want else 0
        needed += need
        asked += want
        got = want if (need == 0 or needed <= F) and asked <= room else 0
        if got != n:
            denied.append(s)
        for at in range(L, L + got):
            if at % B == 0:
                free -= 1
                table[s, at // B] = stack[free]
            slots.append(int(table[s, at // B]) * B + at % B)
            positions.append(at)
        starts.append(len(slots))
        out.append(L + got)
    pad = room - len(slots)
    return table, slots + [-1] * pad, positions + [0] * pad, starts, out, free, denied


# ------------------------------------------------------------------ codes

def fresh_scale(most: float, kind: str) -> float:
    """The scale for a largest magnitude, as a binary32 value."""
    if not math.isfinite(most):
        return math.nan
    if kind == "int8":
        scale = float((torch.tensor(most, dtype=torch.float32) / torch.tensor(127.0)).item())
    else:
        scale = 0.0
        if most > 0:
            scale = 2.0 ** math.floor(math.log2(most / 448.0))
            while most > 448.0 * scale:
                scale *= 2
            while most <= 448.0 * scale / 2:
                scale /= 2
    return max(scale, LEAST_SCALE)


def encode(x: torch.Tensor, scale: float, kind: str) -> torch.Tensor:
    """Codes of binary32 values: the quotient is a binary32 one."""
    y = x.float() / torch.full_like(x, scale, dtype=torch.float32)
    if kind == "int8":
        return torch.nan_to_num(y.round().clamp(-127, 127)).to(torch.int8)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn)


def append(key, value, caches, scales, table, lens, starts, kind):
    """In place on CPU tensors caches = (k, v), scales = (k, v)."""
    B = caches[0].shape[2]
    for x, cache, scale in ((key, caches[0], scales[0]), (value, caches[1], scales[1])):
        for s, L in enumerate(lens):
            n = starts[s + 1] - starts[s]
            for b in range((L - n) // B, (L - 1) // B + 1) if n else ():
                lo, hi = max(L - n - b * B, 0), min(L - b * B, B)
                at = starts[s] + b * B + lo - (L - n)
                rows = x[at:at + hi - lo].float()
                blk = int(table[s, b])
                for h in range(cache.shape[1]):
                    fresh = fresh_scale(float(rows[:, h].abs().max()), kind)
                    old = float(scale[blk, h])
                    now = fresh
                    if lo > 0:
                        now = math.nan if math.isnan(old) or math.isnan(fresh) else max(old, fresh)
                        if now != old:
                            ratio = torch.tensor(old, dtype=torch.float32) / torch.tensor(now, dtype=torch.float32)
                            c = cache[blk, h, :lo].float() * ratio
                            c = torch.nan_to_num(c.round()) if kind == "int8" else c
                            cache[blk, h, :lo] = c.to(cache.dtype)
                    cache[blk, h, lo:hi] = encode(rows[:, h], now, kind)
                    scale[blk, h] = now


def pool(num_blocks, heads, B, D, kind, seed, spread=0.5):
    """A cache of codes and scales whose blocks differ in size."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(num_blocks, heads, B, D, generator=g)
    x *= torch.exp(spread * torch.randn(num_blocks, heads, 1, 1, generator=g))
    most = x.abs().amax((2, 3))
    if kind == "int8":
        scale = most / 127
    else:
        scale = torch.exp2(torch.ceil(torch.log2(most / 448)))
    codes = x / scale.view(num_blocks, heads, 1, 1)
    codes = codes.round().to(torch.int8) if kind == "int8" else codes.to(torch.float8_e4m3fn)
    return codes, scale


# ------------------------------------------------------------------ attention

def attention(query, k_cache, v_cache, k_scales, v_scales, table, lens, starts, scale, out_type):
    """The output in 64 bits and how far a call may be off, row by row of each
    sequence; rows of no sequence stay NaN.

    The bound: half a step of the output's type; a weight rounded to binary16 (2^-11
    relative, or where its bits thin out 2^-28 of the largest value scale, the weights
    lying within [2^3, 2^15] for the largest); logits wrong by d from binary32
    products and sums (2^-20 of the products' magnitudes) move a weight by 2 d and
    its exponential by 2^-21."""
    H, B, D = k_cache.shape[1:]
    T, Hq = query.shape[:2]
    G = Hq // H
    want = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    tol = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    for s, L in enumerate(lens):
        q0, Q = starts[s], starts[s + 1] - starts[s]
        if Q == 0:
            continue
        if L == 0:
            want[q0:q0 + Q] = 0.0
            tol[q0:q0 + Q] = 0.0
            continue
        ids = table[s, :-(-L // B)].long()

        def values(cache, scales):
            x = cache.view(torch.uint8)[ids].view(cache.dtype).to(torch.float32).double() * scales[ids].double().view(-1, H, 1, 1)
            return x.permute(1, 0, 2, 3).reshape(H, -1, D)[:, :L]

        k, v = values(k_cache, k_scales), values(v_cache, v_scales)
        b_most = v_scales[ids].double().amax(0)                                   # [H]
        q = query[q0:q0 + Q].double().view(Q, H, G, D).permute(1, 0, 2, 3).reshape(H, Q * G, D)
        logits = torch.einsum("hrd,hkd->hrk", q, k) * scale
        size = torch.einsum("hrd,hkd->hrk", q.abs(), k.abs()) * scale
        seen = (L - Q + torch.arange(Q)).repeat_interleave(G)
        hidden = torch.arange(L) > seen.view(-1, 1)
        p = torch.softmax(logits.masked_fill(hidden, -math.inf), -1)
        o = torch.einsum("hrk,hkd->hrd", p, v)
        off = size.masked_fill(hidden, 0.0).amax(-1, keepdim=True) * 2.0 ** -20
        a = torch.einsum("hrk,hkd->hrd", p, v.abs())
        largest = 448 if k_cache.dtype == torch.float8_e4m3fn else 127
        bound = (torch.finfo(out_type).eps / 2 * o.abs() + (2.0 ** -11 + 2.0 ** -20 + 2 * off) * a
                 + L * 2.0 ** -28 * largest * b_most.view(H, 1, 1) + torch.finfo(out_type).tiny)
        put = lambda x: x.view(H, Q, G, D).permute(1, 0, 2, 3).reshape(Q, Hq, D)  # noqa: E731
        want[q0:q0 + Q], tol[q0:q0 + Q] = put(o), put(bound)
    return want, tol


def assert_close(got, want, tol, what=""):
    """Within the bound; rows of no sequence (NaN in want) are not looked at."""
    there = ~want.isnan()
    off = (got.double().cpu() - want).abs()
    worst = (off / tol.clamp(min=1e-300))[there & (tol > 0)]
    assert bool((off[there] <= tol[there]).all()), f"{what}: {float(worst.max()) if worst.numel() else 'inf'} of the bound"


# ------------------------------------------------------------------ verification

def verify(target, draft, drafted, uniforms, starts):
    """(tokens [S, K + 1], accepted, borders): `borders` tells for each request how near
    a decision was to its border, relative to what it was made of."""
    S, K = drafted.shape
    tokens = torch.full((S, K + 1), -1, dtype=torch.int64)
    accepted, near = [], []
    for s in range(S):
        row, n = starts[s], starts[s + 1] - starts[s] - 1
        if n < 0:
            accepted.append(0)
            near.append(1.0)
            continue
        a = 0
        while a < n:
            x = int(drafted[s, a])
            q = 1.0 if draft is None else float(draft[s, a, x])
            if not float(uniforms[s, a]) * q < float(target[row + a, x]):
                break
            a += 1
        w = target[row + a].double()
        if a < n:
            other = torch.zeros_like(w)
            if draft is None:
                other[int(drafted[s, a])] = math.inf
            else:
                other = draft[s, a].double()
            beyond = (w - other).clamp(min=0)
            w = beyond if float(beyond.sum()) > 0 else w
        sums = w.cumsum(0)
        goal = float(uniforms[s, K]) * float(sums[-1])
        at = int((sums <= goal).sum())
        tokens[s, :a] = drafted[s, :a]
        tokens[s, a] = at
        accepted.append(a)
        low = float(sums[at - 1]) if at else 0.0
        near.append(min(abs(goal - low) if at else 1.0, abs(float(sums[at]) - goal)) / float(sums[-1]))
    return tokens, torch.tensor(accepted, dtype=torch.int32), near
