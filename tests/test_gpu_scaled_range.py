"""Attention over block-scaled codes where scales lie far apart or are not finite: a
row's result depends on what the row sees, and its precision on its own weights."""
import math

import pytest
import torch

import step_common as sc

pytestmark = pytest.mark.gpu


def pk():
    from paged_kv_cache_141_gb300 import binding
    return binding


def reference(query, kc, vc, ks, vs, table, lens, starts, scale, out_type):
    """The output in 64 bits, hidden tokens left out altogether, and how far a call may be off.

    The bound: half a step of the output's type; each weight p b (softmax times value
    scale) rounded to binary16 once, 2^-11 of itself (2^-22 in two terms, for a binary16
    output), or where its bits thin out half of binary16's least step, 2^-25, of weights
    whose largest stands at 2^5 or more: 2^-30 of the row's largest; logits wrong by d
    from binary32 products and sums (2^-20 of the products' magnitudes) move a weight
    by 2 d, and its exponential and the sums by 2^-20."""
    H, B, D = kc.shape[1:]
    T, Hq = query.shape[:2]
    G = Hq // H
    want, tol = (torch.full((T, Hq, D), math.nan, dtype=torch.float64) for _ in range(2))
    term = 2.0 ** -22 if out_type == torch.float16 else 2.0 ** -11
    largest = 448 if kc.dtype == torch.float8_e4m3fn else 127
    for s, L in enumerate(lens):
        q0, Q = starts[s], starts[s + 1] - starts[s]
        ids = table[s, :-(-L // B)].long()
        codes = lambda c: c.view(torch.uint8)[ids].view(c.dtype).float().double().permute(1, 0, 2, 3).reshape(H, -1, D)[:, :L]  # noqa: E731
        wide = lambda x: x[ids].double().t().repeat_interleave(B, 1)[:, None, :L]  # noqa: E731
        q = query[q0:q0 + Q].double().view(Q, H, G, D).permute(1, 0, 2, 3).reshape(H, Q * G, D)
        hidden = torch.arange(L) > (L - Q + torch.arange(Q)).repeat_interleave(G).view(-1, 1)
        logits = torch.einsum("hrd,hkd->hrk", q, codes(kc)) * wide(ks) * scale
        size = (torch.einsum("hrd,hkd->hrk", q.abs(), codes(kc).abs()) * wide(ks) * scale).masked_fill(hidden, 0.0)
        p = torch.softmax(logits.masked_fill(hidden, -math.inf), -1)
        w = (p * wide(vs)).masked_fill(hidden, 0.0)
        o = torch.einsum("hrk,hkd->hrd", w, codes(vc))
        a = torch.einsum("hrk,hkd->hrd", w, codes(vc).abs())
        off = size.amax(-1, keepdim=True) * 2.0 ** -20
        bound = (torch.finfo(out_type).eps / 2 * o.abs() + (term + 2.0 ** -20 + 2 * off) * a
                 + L * 2.0 ** -30 * largest * w.amax(-1, keepdim=True) + torch.finfo(out_type).tiny)
        put = lambda x: x.view(H, Q, G, D).permute(1, 0, 2, 3).reshape(Q, Hq, D)  # noqa: E731
        want[q0:q0 + Q], tol[q0:q0 + Q] = put(o), put(bound)
    return want, tol


def call(query, pool, table, lens, starts, cap=None):
    kc = pool[0]
    T, Hq, D = query.shape
    S, H = len(lens), kc.shape[1]
    Q = max(b - a for a, b in zip(starts, starts[1:]))
    cap = max(lens) if cap is None else cap
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, status = torch.full_like(query, 7.0).cuda(), t([0])
    ws = pk().alloc_scaled_workspace(S, T, Hq, H, D, Q, cap)
    ws.fill_(0xFF)
    pk().scaled_attention(out, query.cuda(), *(x.cuda() for x in pool), table.cuda(), t(lens), cap, D ** -0.5, ws, query_start=t(starts),
                          max_queries_per_seq=Q, dev_status=status)
    assert int(status) == 0
    return out


# rows of a KV head: tiles of 8, 16 and 32 rows, the tcgen05 kernel with one and with two tiles
SHAPES = [(128, 8, 2, 1), (64, 8, 2, 3), (128, 8, 2, 7), (256, 8, 2, 1), (256, 8, 2, 4),
          (128, 8, 1, 6), (64, 8, 1, 14), (128, 8, 2, 40), (256, 8, 1, 6), (256, 8, 2, 50)]


class Case:
    def __init__(self, kind, dtype, shape, lens, B=16, seed=0):
        self.D, self.Hq, self.H, Q = shape
        g = torch.Generator().manual_seed(seed + self.D + Q)
        self.table, nb = sc.table_of(len(lens), max(-(-L // B) for L in lens), seed)
        (self.kc, self.ks), (self.vc, self.vs) = (sc.pool(nb, self.H, B, self.D, kind, seed + i, 0.3) for i in range(2))
        self.lens, self.B, self.Q, self.kind = lens, B, Q, kind
        self.starts = [Q * s for s in range(len(lens) + 1)]
        self.query = torch.randn(Q * len(lens), self.Hq, self.D, generator=g)
        self.query[..., 0] = 4.0
        self.query = self.query.to(sc.TYPES[dtype])

    def logit_of(self, block, nats):
        """Every row's logit with every token of the block, for every sequence."""
        ids = self.table[:, block].long()
        codes = self.kc.float()
        codes[ids] = 0.0
        codes[ids, :, :, 0] = math.copysign(96.0, nats)
        self.kc = codes.to(self.kc.dtype)
        self.ks[ids] = abs(nats) / (4.0 * 96.0 * self.D ** -0.5)

    def check(self, cap=None):
        pool = (self.kc, self.vc, self.ks, self.vs)
        got = call(self.query, pool, self.table, self.lens, self.starts, cap).double().cpu()
        want, tol = reference(self.query, *pool, self.table, self.lens, self.starts, self.D ** -0.5, self.query.dtype)
        assert bool((got.isnan() == want.isnan()).all()), f"rows of NaN: {int(got.isnan().any(-1).sum())}, {int(want.isnan().any(-1).sum())} expected"
        there = ~want.isnan()
        ratio = ((got - want).abs() / tol)[there]
        assert float(ratio.max()) <= 1.0, f"{float(ratio.max())} of the bound"
        return want


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("octaves", [20, 45, 80])
def test_large_values_that_hardly_count(kind, dtype, shape, octaves):
    # a block of huge values whose softmax weights are e^-60: first, in the middle, last but one
    for block in (0, 5, 11):
        c = Case(kind, dtype, shape, [200, 193])
        c.logit_of(block, -60.0)
        c.vs[c.table[:, block].long()] *= 2.0 ** octaves
        c.check()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] > 1])
@pytest.mark.parametrize("octaves", [12, 20, 45, 80])
def test_large_values_that_a_row_does_not_see(kind, dtype, shape, octaves):
    # the newest block's values are huge; the rows before it do not see them
    c = Case(kind, dtype, shape, [shape[3] // 2 + 192, shape[3] // 2 + 128])
    for s, L in enumerate(c.lens):
        ids = c.table[s, (L - c.Q // 2) // c.B:].long()
        c.vs[ids] *= 2.0 ** octaves
        if dtype == "f16":                                   # (the outputs of those who do stay within binary16)
            c.vc.view(torch.uint8)[ids] = 0
    c.check()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("nats", [20.0, 50.0])
def test_the_heaviest_tokens_have_no_value(kind, shape, nats):
    # a block that takes nearly all of the softmax, with values of zero: the others' weights are e^-20, e^-50
    for block in (0, 7, 11):
        c = Case(kind, "bf16", shape, [200, 195])
        c.logit_of(block, nats)
        c.vs[c.table[:, block].long()] = 0.0
        c.check()


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("shape", SHAPES[:1] + SHAPES[4:6] + SHAPES[7:])
def test_value_scales_that_grow_and_shrink(kind, shape):
    # 40 octaves up, or down, over 60 blocks, with partitions of the context beside one
    for step in (2.0 ** 0.7, 2.0 ** -0.7):
        for B, cap in ((16, None), (8, 9000)):
            c = Case(kind, "bf16", shape, [950, 700], B=B)
            for s in range(2):
                ids = c.table[s].long()
                c.vs[ids] *= (step ** (torch.arange(len(ids)) * B / 16)).view(-1, 1)
            c.check(cap)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("of", ["keys", "values", "both"])
def test_what_is_not_a_number_stays_where_it_is_seen(kind, dtype, shape, of):
    # scales of NaN in the newest block, where tokens before it are queries too, and in one of two sequences' last
    c = Case(kind, dtype, shape, [shape[3] // 2 + 192, shape[3] + 120])
    bad = c.table[0, (c.lens[0] - c.Q // 2) // c.B:-(-c.lens[0] // c.B)].long()
    for x in {"keys": [c.ks], "values": [c.vs], "both": [c.ks, c.vs]}[of]:
        x[bad, -1] = math.nan
    want = c.check()
    rows = want[:c.Q].isnan().any(-1)
    assert bool(rows.any()) == (len(bad) > 0) and not bool(rows[0].any() and c.Q > 1) and not bool(want[c.Q:].isnan().any())


@pytest.mark.parametrize("heads", [(8, 2), (8, 1)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_bad_draft_leaves_the_tokens_before_it(heads, bad):
    """Through the append: the last of six new tokens is not finite, and begins a block."""
    Hq, H = heads
    D, B, L = 128, 16, 161
    g = torch.Generator().manual_seed(3)
    table, nb = sc.table_of(1, 11, 1)
    k, v = (torch.randn(L, H, D, generator=g).bfloat16() for _ in range(2))
    query = torch.randn(6, Hq, D, generator=g).bfloat16().cuda()
    outs = []
    for x in (None, k, v):
        put = [t.clone().cuda() for t in (k, v)]
        if x is not None:
            put[0 if x is k else 1][-1, :, 3] = bad
        kc, vc = (torch.zeros(nb, H, B, D, dtype=torch.int8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros(nb, H, device="cuda") for _ in range(2))
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        pk().scaled_append(*put, kc, vc, ks, vs, table.cuda(), t([L]), L, t([0, L]))
        out = torch.empty_like(query)
        ws = pk().alloc_scaled_workspace(1, 6, Hq, H, D, 6, L)
        pk().scaled_attention(out, query, kc, vc, ks, vs, table.cuda(), t([L]), L, D ** -0.5, ws, query_start=t([0, 6]), max_queries_per_seq=6)
        outs.append(out)
    for out in outs[1:]:
        assert out[:5].equal(outs[0][:5]) and bool(out[5].isnan().all())


@pytest.mark.parametrize("shape", SHAPES)
def test_calls_repeat_bit_for_bit(shape):
    c = Case("int8", "bf16", shape, [2100, 350, 64])
    pool = (c.kc, c.vc, c.ks, c.vs)
    first = call(c.query, pool, c.table, c.lens, c.starts)
    for _ in range(3):
        assert call(c.query, pool, c.table, c.lens, c.starts).equal(first)
