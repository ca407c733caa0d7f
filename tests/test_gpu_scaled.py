"""The block-scaled 8-bit cache: the append against its definition, code by code,
and the attention against softmax in 64 bits."""
import math
import random

import pytest
import torch

import step_common as sc

pytestmark = pytest.mark.gpu


def pk():
    from paged_kv_cache_141_gb300 import binding
    return binding


# ------------------------------------------------------------------ append

def run_append(kind, dtype, H, D, B, lens, news, seed=0, prefix=None, strided=False, extra=0):
    """Appends news[s] newest tokens into contexts of lens[s]; `prefix`: what the pool holds first."""
    g = torch.Generator().manual_seed(seed)
    S, T = len(lens), sum(news)
    table, nb = sc.table_of(S, max(1, max(-(-L // B) for L in lens)), seed)
    caches, scales = zip(*(sc.pool(nb, H, B, D, kind, seed + i) for i in range(2)))
    if prefix:
        prefix(caches, scales)
    kv = torch.randn(T + extra, 2 * H, D, generator=g)
    kv *= torch.exp(torch.randn(T + extra, 2 * H, 1, generator=g))            # tokens of different size
    kv = kv.to(sc.TYPES[dtype])
    k, v = kv[:, :H], kv[:, H:]
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    dev = [x.cuda() for x in (*caches, *scales)]
    kd, vd = (kv.cuda()[:, :H], kv.cuda()[:, H:]) if strided else (k.contiguous().cuda(), v.contiguous().cuda())
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = all(n == 1 for n in news) and not extra and seed % 2 == 0
    pk().scaled_append(kd, vd, *dev, table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                       max_new_tokens=max(news) if news else 1,
                       query_start=None if one else torch.tensor(starts, dtype=torch.int32, device="cuda"), dev_status=status)
    sc.append(k, v, caches, scales, table, lens, starts, kind)
    assert int(status) == 0
    for name, got, want in zip(("k codes", "v codes", "k scales", "v scales"), dev, (*caches, *scales)):
        got = got.cpu()
        if got.dtype == torch.float32:
            assert got.equal(want) or bool(((got == want) | (got.isnan() & want.isnan())).all()), name
        else:
            assert got.view(torch.uint8).equal(want.view(torch.uint8)), name
    return dev


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_types(kind, dtype, D):
    run_append(kind, dtype, 2, D, 16, [1, 16, 17, 40, 33, 100], [1, 3, 2, 40, 20, 5], seed=D, strided=D == 128)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("B", [1, 5, 8, 24, 32, 128, 1024])
def test_append_blocks(kind, B):
    lens = [1, B, B + 1, 2 * B + 3, 3 * B]
    run_append(kind, "bf16", 3, 128, B, lens, [min(L, n) for L, n in zip(lens, (1, 1, 1, B + 2, 3 * B))], seed=B)
    run_append(kind, "f16", 1, 64, B, lens, [1] * 5, seed=2 * B)


def test_append_none_and_padding():
    run_append("int8", "bf16", 2, 128, 16, [0, 5, 20], [0, 0, 4], extra=3)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_starts_a_block_anew(kind):
    # what an earlier request left in the block (a huge scale, NaN) does not count when the first row is written
    def stale(caches, scales):
        scales[0].fill_(1e30)
        scales[1].fill_(math.nan)
    run_append(kind, "bf16", 2, 64, 16, [1, 17, 33, 16], [1, 1, 1, 16], prefix=stale)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_append_zeros_and_small_values(kind):
    for fill in (0.0, 2.0 ** -24, 1e-38):
        k = torch.full((4, 1, 64), fill, device="cuda")
        caches, scales = zip(*(sc.pool(3, 1, 16, 64, kind, i) for i in range(2)))
        dev = [x.cuda() for x in (*caches, *scales)]
        table = torch.tensor([[2]], dtype=torch.int32)
        pk().scaled_append(k, k, *dev, table.cuda(), torch.tensor([4], dtype=torch.int32, device="cuda"), 4,
                           torch.tensor([0, 4], dtype=torch.int32, device="cuda"))
        sc.append(k.cpu(), k.cpu(), caches, scales, table, [4], [0, 4], kind)
        assert dev[2].cpu().equal(scales[0]) and dev[0].cpu().view(torch.uint8).equal(caches[0].view(torch.uint8))


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_append_of_what_is_not_finite_shows(kind, bad):
    k = torch.randn(2, 2, 64, device="cuda")
    v = k.clone()
    k[1, 1, 5] = bad
    caches, scales = zip(*(sc.pool(3, 2, 16, 64, kind, i) for i in range(2)))
    dev = [x.cuda() for x in (*caches, *scales)]
    table, lens = torch.tensor([[1, 2]], dtype=torch.int32).cuda(), torch.tensor([5], dtype=torch.int32, device="cuda")
    pk().scaled_append(k, v, *dev, table, lens, 2, torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    assert dev[2][1].isnan().tolist() == [False, True] and not bool(dev[3].isnan().any())
    # it stays, whatever comes after, until the block starts anew
    pk().scaled_append(v[:1].contiguous(), v[:1].contiguous(), *dev, table, lens + 1)
    assert dev[2][1].isnan().tolist() == [False, True]
    out = torch.empty(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    ws = pk().alloc_scaled_workspace(1, 1, 2, 2, 64, 1, 32)
    pk().scaled_attention(out, torch.ones_like(out), *dev, table, lens + 1, 32, 0.125, ws)
    assert bool(out[0, 1].isnan().all()) and not bool(out[0, 0].isnan().any())
    pk().scaled_append(v, v, *dev, table, lens - 3, 2, torch.tensor([0, 2], dtype=torch.int32, device="cuda"))
    assert not bool(dev[2][1].isnan().any())


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_tokens_one_by_one_stay_near(kind):
    """16 tokens of growing size, appended one by one: a code's error is at most half a step of the
    final scale for each growth (integers); E4M3 codes only lose what becomes subnormal."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(16, 1, 128, generator=g) * torch.linspace(0.1, 3, 16).view(16, 1, 1)
    caches, scales = zip(*(sc.pool(2, 1, 16, 128, kind, i) for i in range(2)))
    dev = [t.cuda() for t in (*caches, *scales)]
    table = torch.tensor([[1]], dtype=torch.int32, device="cuda")
    for t in range(16):
        row = x[t:t + 1].cuda()
        pk().scaled_append(row, row, *dev, table, torch.tensor([t + 1], dtype=torch.int32, device="cuda"))
    got = dev[0][1, 0].cpu().float().double() * float(dev[2][1, 0])
    want, step = x[:, 0].double(), float(dev[2][1, 0])
    if kind == "int8":
        assert float((got - want).abs().max()) <= 16 * step / 2
        # sixteen roundings of variance step^2 / 12 at most, a tenth more for the sample
        assert float((got - want).norm()) <= 1.1 * (16 / 12 * want.numel()) ** 0.5 * step
    else:
        # half a step of a normal code is 2^-4 of it, of a subnormal one 2^-10 of the scale, once for each growth
        assert bool(((got - want).abs() <= want.abs() * 2.0 ** -4 + 6 * step * 2.0 ** -10).all())


def test_append_bad_data():
    k = torch.randn(4, 1, 64, device="cuda")
    caches, scales = zip(*(sc.pool(5, 1, 16, 64, "int8", i) for i in range(2)))
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for table, lens, starts, most, flag in (
            ([[1], [5]], [4, 4], [0, 1, 2], 1, pk().DEV_BAD_BLOCK_ID),       # past the pool
            ([[1], [-1]], [4, 4], [0, 1, 2], 1, pk().DEV_BAD_BLOCK_ID),
            ([[1], [2]], [4, 17], [0, 1, 2], 1, pk().DEV_BAD_LEN),           # longer than its table
            ([[1], [2]], [4, -1], [0, 1, 2], 1, pk().DEV_BAD_LEN),
            ([[1], [2]], [4, 1], [0, 1, 3], 4, pk().DEV_BAD_LEN),            # more new tokens than tokens
            ([[1], [2]], [4, 4], [0, 1, 3], 1, pk().DEV_BAD_LEN),            # more than max_new_tokens
            ([[1], [2]], [4, 8], [0, 1, 6], 6, pk().DEV_BAD_LEN),            # past the rows
            ([[1], [2]], [4, 4], [0, 1, 0], 4, pk().DEV_BAD_LEN)):
        dev = [x.cuda() for x in (*caches, *scales)]
        status = t([0])
        pk().scaled_append(k, k, *dev, t(table), t(lens), most, t(starts), dev_status=status)
        assert int(status) == flag
        want_c, want_s = [c.clone() for c in caches], [s.clone() for s in scales]
        sc.append(k.cpu(), k.cpu(), want_c, want_s, torch.tensor(table[:1]), lens[:1], starts[:2], "int8")
        for got, want in zip(dev, (*want_c, *want_s)):
            assert got.cpu().equal(want)                                     # the first sequence alone was written


# ------------------------------------------------------------------ attention

def run_attention(kind, dtype, Hq, H, D, B, lens, queries, seed=0, spread=0.5, prepare=None, max_len=None, tail=0, q_gain=1.0):
    S, T = len(lens), sum(queries)
    g = torch.Generator().manual_seed(seed + 77)
    most = max(1, max(-(-L // B) for L in lens))
    table, nb = sc.table_of(S, most, seed)
    (kc, ks), (vc, vs) = (sc.pool(nb, H, B, D, kind, seed + i, spread) for i in range(2))
    if prepare:
        prepare(kc, vc, ks, vs, table)
    # behind every context's end lie an earlier request's codes: here the largest, or NaN
    for s, L in enumerate(lens):
        if L % B:
            for c in (kc, vc):
                c.view(torch.uint8)[int(table[s, L // B]), :, L % B:] = 0x7F
    query = (q_gain * torch.randn(T + tail, Hq, D, generator=g)).to(sc.TYPES[dtype])
    starts = [0]
    for n in queries:
        starts.append(starts[-1] + n)
    scale = D ** -0.5
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full_like(query, 7.0).cuda()
    status = t([0])
    Q, cap = max(queries), max(lens) if max_len is None else max_len
    one = all(n == 1 for n in queries) and not tail
    ws = pk().alloc_scaled_workspace(S, T + tail, Hq, H, D, Q, cap)
    ws.fill_(0xFF)                                                           # NaN: nothing may be read that was not written
    pk().scaled_attention(out, query.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(), t(lens), cap, scale, ws,
                          query_start=None if one else t(starts), max_queries_per_seq=Q, dev_status=status)
    assert int(status) == 0
    want, tol = sc.attention(query, kc, vc, ks, vs, table, lens, starts, scale, query.dtype)
    sc.assert_close(out, want, tol)
    assert bool((out[T:] == 7.0).all())
    return out


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (16, 2), (12, 4)])
def test_decode(kind, dtype, D, heads):
    run_attention(kind, dtype, *heads, D, 16, [1, 15, 16, 17, 31, 32, 33, 129, 300], [1] * 9, seed=D)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("B", [1, 5, 8, 24, 32, 48, 128, 1024])
def test_decode_blocks(kind, B):
    run_attention(kind, "bf16", 8, 2, 128, B, [1, B, B + 1, 3 * B + 2, 200], [1] * 5, seed=B)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("heads", [(8, 8), (40, 2), (9, 1), (17, 1), (33, 1), (128, 1)])
def test_decode_groups(kind, heads):
    run_attention(kind, "f16", *heads, 128, 16, [70, 3, 257], [1] * 3)


def test_empty_contexts():
    run_attention("int8", "bf16", 8, 2, 128, 16, [0, 5, 0, 300], [1] * 4)
    run_attention("e4m3", "f16", 8, 2, 64, 16, [0, 5, 0, 300], [1] * 4, max_len=5000)      # partitions
    run_attention("e4m3", "f16", 8, 2, 64, 16, [0, 0], [1] * 2)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_empty_contexts_of_many_rows(D):
    run_attention("int8", "bf16", 40, 1, D, 16, [0, 5, 0, 300], [1] * 4)
    run_attention("e4m3", "f16", 600, 2, D, 16, [0, 0, 70], [1] * 3)
    run_attention("e4m3", "f16", 40, 1, D, 16, [0, 5, 0, 300], [1] * 4, max_len=5000)      # partitions


@pytest.mark.parametrize("S", [2, 127, 128, 129, 200])
def test_many_sequences_of_many_rows(S):
    # contexts of one length, of none, and in no order: each sequence is served once
    lens = [(37 * s) % 61 if s % 3 else 40 for s in range(S)]
    run_attention("int8", "bf16", 8, 1, 64, 8, lens, [min(L, (5 * s) % 7) for s, L in enumerate(lens)], seed=S)
    run_attention("e4m3", "f16", 36, 1, 64, 16, lens, [1] * S, seed=S)
    run_attention("e4m3", "bf16", 36, 1, 256, 16, lens, [1] * S, seed=S)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("lens", [[5000], [4096, 255, 256, 257, 1, 2048], [1, 20001]])
def test_decode_partitions(kind, lens):
    out = run_attention(kind, "bf16", 8, 2, 128, 16, lens, [1] * len(lens))
    # a larger bound cuts the context elsewhere: the same result to rounding
    other = run_attention(kind, "bf16", 8, 2, 128, 16, lens, [1] * len(lens), max_len=3 * max(lens) + 11)
    assert float((out.float() - other.float()).abs().max()) <= 2.0 ** -7 * float(out.float().abs().max())


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("bf16", 256)])
@pytest.mark.parametrize("queries", [[2, 2, 2, 2], [5, 1, 3, 4], [0, 8, 1, 0], [1, 40, 17, 64]])
def test_drafts(kind, dtype, D, queries):
    lens = [max(n, L) for n, L in zip(queries, (2, 64, 333, 700))]
    run_attention(kind, dtype, 8, 2, D, 16, lens, queries, seed=len(queries) + D, tail=3)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("heads", [(4, 4), (8, 1), (12, 2)])
def test_chunks(kind, heads):
    run_attention(kind, "bf16", *heads, 128, 16, [300, 130, 1], [300, 77, 1])
    run_attention(kind, "f16", *heads, 64, 24, [129, 400], [129, 130])


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("B", [1, 4, 8, 16, 24, 40, 48, 128, 1024])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64), ("f16", 128), ("bf16", 256), ("f16", 256)])
def test_many_rows_over_blocks(kind, B, dtype, D):
    lens = [500, 45, 1300, 129, 9]
    run_attention(kind, dtype, 8, 1, D, B, lens, [6, 45, 30, 1, 9], seed=B + D, tail=2)
    run_attention(kind, dtype, 4, 2, D, B, lens, [200, 45, 150, 129, 0], seed=B + D)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows_in_partitions(kind, D):
    # few sequences, long contexts: the tcgen05 kernel's partitions, some of which a row does not see
    for _ in range(5):                                                       # (warps run ahead of each other by turns)
        run_attention(kind, "bf16", 8, 1, D, 16, [9000, 1025, 4096], [7, 6, 5], seed=D)
    run_attention(kind, "f16", 8, 1, D, 8, [3000, 2048], [300, 1], seed=D)
    run_attention(kind, "bf16", 8, 1, D, 32, [5000], [1100], seed=D)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_blocks_of_very_different_size(kind):
    # value scales over twenty octaves, an all-zero block, one with scale 0; keys alike, within the range of exp
    def prepare(kc, vc, ks, vs, table):
        ids = table[0].long()
        vs[ids] *= torch.exp2(torch.linspace(-14, 6, len(ids))).view(-1, 1)
        vc.view(torch.uint8)[ids[3]] = 0
        vs[ids[4]] = 0.0
        ks[ids[5]] = 0.0
        ks[ids[6:8]] *= 8
    for L in (500, 3000):
        run_attention(kind, "bf16", 8, 2, 128, 16, [L], [1], prepare=prepare)
        run_attention(kind, "bf16", 8, 2, 128, 16, [L], [50], prepare=prepare)
        run_attention(kind, "f16", 8, 2, 64, 8, [L], [90], prepare=prepare)
        run_attention(kind, "bf16", 8, 2, 128, 16, [L], [6], prepare=prepare)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
def test_sharp_and_flat_rows(kind):
    run_attention(kind, "f16", 8, 2, 128, 16, [700, 90], [1, 1], q_gain=30.0)
    run_attention(kind, "bf16", 8, 2, 128, 16, [700, 90], [3, 3], q_gain=30.0)
    run_attention(kind, "bf16", 8, 2, 128, 16, [700, 90], [1, 1], q_gain=1e-6)
    run_attention(kind, "bf16", 8, 2, 128, 16, [700, 90], [1, 1], q_gain=0.0)


@pytest.mark.parametrize("gain", [1e30, 1e-30])
def test_query_beyond_binary16(gain):
    # the query's size goes into the row's power of two; the keys' scales take it back
    def prepare(kc, vc, ks, vs, table):
        ks /= gain
    run_attention("int8", "bf16", 8, 2, 128, 16, [300, 5], [1, 1], prepare=prepare, q_gain=gain)


def test_bad_data():
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    H, D, B = 2, 64, 16
    (kc, ks), (vc, vs) = (sc.pool(9, H, B, D, "int8", i) for i in range(2))
    pool = [x.cuda() for x in (kc, vc, ks, vs)]
    q = torch.randn(8, 4, D, dtype=torch.bfloat16, device="cuda")
    good = torch.tensor([[1, 2, 3], [4, 5, 6]], dtype=torch.int32)
    for table, lens, starts, cap, flag in (
            (good, [40, 49], [0, 3, 8], 100, pk().DEV_BAD_LEN),              # longer than its table
            (good, [40, 33], [0, 3, 8], 32, pk().DEV_BAD_LEN),               # longer than the bound (both)
            (good, [40, 4], [0, 3, 8], 48, pk().DEV_BAD_LEN),                # more queries than tokens
            (good, [40, -3], [0, 3, 8], 48, pk().DEV_BAD_LEN),
            (good, [40, 40], [0, 3, 9], 48, pk().DEV_BAD_LEN),               # past the rows
            (good, [40, 40], [0, 3, 2], 48, pk().DEV_BAD_LEN),
            (torch.tensor([[1, 2, 3], [4, 9, 6]], dtype=torch.int32), [40, 40], [0, 3, 8], 48, pk().DEV_BAD_BLOCK_ID),
            (torch.tensor([[1, 2, 3], [-1, 5, 6]], dtype=torch.int32), [40, 40], [0, 3, 8], 48, pk().DEV_BAD_BLOCK_ID)):
        out = torch.full_like(q, 7.0)
        status = t([0])
        ws = pk().alloc_scaled_workspace(2, 8, 4, H, D, 5, cap)
        pk().scaled_attention(out, q, *pool, table.cuda(), t(lens), cap, 0.125, ws, query_start=t(starts), max_queries_per_seq=5,
                              dev_status=status)
        assert int(status) == flag
        if cap == 48:                                                        # the first sequence is fine
            want, tol = sc.attention(q.cpu()[:3], kc, vc, ks, vs, table[:1], lens[:1], [0, 3], 0.125, torch.bfloat16)
            sc.assert_close(out[:3], want, tol)


def test_far_blocks():
    """Rows whose byte offsets pass 32 bits."""
    H, D, B, nb = 1, 256, 1024, 16400                                       # 4.3e9 bytes a cache
    kc, vc = (torch.zeros(nb, H, B, D, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(nb, H, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(1030, H, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.tensor([[nb - 1, nb - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1030], dtype=torch.int32, device="cuda")
    pk().scaled_append(k, v, kc, vc, ks, vs, table, lens, 1030, torch.tensor([0, 1030], dtype=torch.int32, device="cuda"))
    q = torch.randn(1, 4, D, generator=g, device="cuda").bfloat16()
    out = torch.empty_like(q)
    ws = pk().alloc_scaled_workspace(1, 1, 4, H, D, 1, 2048)
    pk().scaled_attention(out, q, kc, vc, ks, vs, table, lens, 2048, D ** -0.5, ws)
    ids = table[0].long()
    near = [x[ids].cpu() for x in (kc, vc, ks, vs)]
    want, tol = sc.attention(q.cpu(), *near, torch.tensor([[0, 1]]), [1030], [0, 1], D ** -0.5, torch.bfloat16)
    sc.assert_close(out, want, tol)
    assert int(kc[:-2].count_nonzero()) == 0
