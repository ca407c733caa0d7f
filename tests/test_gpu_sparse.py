"""key_bounds and sparse_decode on the GPU against plain forms in 64 bits.

Bounds and selections are compared for equality. The output's tolerance,
derived: the decode rounds it once (half a step of its type, relative); its
softmax weights carry ex2.approx's 2^-22, the binary32 sums and scores (about
2^-17 relative here: |scale q k| stays below 2^5 and is accumulated over at
most 256 products) and their cut to 16-bit terms (2^-16 for two terms of a
16-bit cache, 2^-11 for the one binary16 term of an E4M3 cache), each against
sum_i p_i |v_i|, twice (numerator and sum): 2^-13 and 2^-9 of that sum, and
2^-15 for binary32, cover them.
"""
import pytest
import torch

from paged_kv_cache_141_gb300 import binding as pk

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
WEIGHTS = {"f32": 2.0 ** -15, "f16": 2.0 ** -13, "bf16": 2.0 ** -13, "e4m3": 2.0 ** -9}


class Pool:
    def __init__(self, lens, Hq=8, Hkv=2, D=128, B=16, dtype="bf16", e4m3=False, seed=0, max_blocks=None):
        g = torch.Generator().manual_seed(seed)
        self.S, self.Hq, self.Hkv, self.D, self.B, self.e4m3, self.dtype = len(lens), Hq, Hkv, D, B, e4m3, dtype
        self.dt = TYPES[dtype]
        n = [-(-L // B) for L in lens]
        self.max_blocks = max_blocks or max(1, max(n))
        self.num_blocks = sum(n) + 3
        perm = torch.randperm(self.num_blocks - 1, generator=g) + 1          # block 0: NaN, in the padding
        self.tables = torch.zeros((self.S, self.max_blocks), dtype=torch.int32)
        at = 0
        for s, k in enumerate(n):
            self.tables[s, :k] = perm[at:at + k].int()
            at += k
        self.lens, self.max_len = lens, max(lens)
        shape = (self.num_blocks, Hkv, B, D)
        caches = []
        for _ in range(2):
            x = torch.randn(shape, generator=g) * (1 + (torch.rand(D, generator=g) < 0.1).float())
            x = (x * 40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else x.to(self.dt)
            nan = 0x7F if e4m3 else float("nan")
            x[0] = nan
            for s, L in enumerate(lens):
                if L % B:
                    x[self.tables[s, L // B], :, L % B:] = nan
            caches.append(x.cuda())
        self.kc, self.vc = caches
        self.ks, self.vs = (0.021, 0.027) if e4m3 else (1.0, 1.0)
        self.query = torch.randn((self.S, Hq, D), generator=g).to(self.dt).cuda()
        self.tables = self.tables.cuda()
        self.context = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.bounds = torch.full((self.num_blocks, Hkv, 2, D), float("nan"), dtype=self.dt, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.scale = D ** -0.5

    def keys(self, cache):
        return (cache.view(torch.float8_e4m3fn) if self.e4m3 else cache).double()

    def want_bounds(self, s, j):
        """Bounds of logical block j of sequence s: [Hkv, 2, D]."""
        k = self.keys(self.kc[self.tables[s, j]])[:, :min(self.B, self.lens[s] - j * self.B)]
        return torch.stack((k.amin(1), k.amax(1)), 1)

    def fill_bounds(self):
        pk.key_bounds(self.bounds, self.kc, self.tables, self.context, self.max_len, new_tokens=self.context,
                      max_new_tokens=self.max_len, dev_status=self.status)

    def decode(self, K, first=1, recent=1, ws=None, **kw):
        out = torch.full_like(self.query, 7.5)
        sel = torch.full((self.S, self.Hkv, K), 99, dtype=torch.int32, device="cuda")
        ws = ws if ws is not None else pk.alloc_sparse_workspace(self.S, self.Hq, self.Hkv, self.D, self.B,
                                                                 self.max_len, K)
        pk.sparse_decode(out, self.query, self.kc, self.vc, self.bounds, self.tables, self.context, self.max_len,
                         self.scale, K, ws, first, recent, selected=sel, k_scale=self.ks, v_scale=self.vs,
                         dev_status=self.status, **kw)
        torch.cuda.synchronize()
        return out, sel

    def want_selected(self, s, h, K, first, recent):
        L, B, G = self.lens[s], self.B, self.Hq // self.Hkv
        n = -(-L // B)
        if n <= K:
            return list(range(n))
        q = self.query[s, h * G:(h + 1) * G].double()
        bnd = self.bounds[self.tables[s, :n].long(), h].double()             # [n, 2, D]
        t = torch.where(q[:, None] < 0, q[:, None] * bnd[None, :, 0], q[:, None] * bnd[None, :, 1])
        score = t.sum(-1)
        score = torch.where(score.isnan(), float("inf"), score).amax(0).tolist()
        rest = sorted(range(first, n - recent), key=lambda b: (-score[b], b))
        return sorted(list(range(first)) + rest[:K - first - recent] + list(range(n - recent, n)))

    def check(self, out, sel, K, first=1, recent=1):
        G = self.Hq // self.Hkv
        sel, got = sel.cpu().tolist(), out.double()
        for s, L in enumerate(self.lens):
            for h in range(self.Hkv):
                want = self.want_selected(s, h, K, first, recent)
                assert sel[s][h] == want + [-1] * (K - len(want)), (s, h)
                rows = got[s, h * G:(h + 1) * G]
                if L == 0:
                    assert bool((rows == 0).all())
                    continue
                tok = torch.tensor([b * self.B + i for b in want for i in range(self.B) if b * self.B + i < L])
                blk = self.tables[s].long()[(tok // self.B).cuda()]
                k, v = (self.keys(c)[blk, h, (tok % self.B).cuda()] for c in (self.kc, self.vc))
                p = torch.softmax(self.query[s, h * G:(h + 1) * G].double() @ k.t() * (self.scale * self.ks), -1)
                ref, mass = p @ v * self.vs, p @ v.abs() * self.vs
                tol = torch.finfo(self.dt).eps / 2 * ref.abs() + WEIGHTS["e4m3" if self.e4m3 else self.dtype] * mass
                err = (rows - ref).abs()
                assert bool((err <= tol).all()), (s, h, float((err - tol).max()))


# ------------------------------------------------------------------ bounds

@pytest.mark.parametrize("dtype,e4m3", [("f32", False), ("f16", False), ("bf16", False), ("f16", True), ("bf16", True)])
@pytest.mark.parametrize("D,B", [(64, 16), (128, 16), (256, 16), (128, 1), (64, 7), (128, 48), (256, 1024)])
def test_bounds_of_new_tokens(dtype, e4m3, D, B):
    lens = [1, B, B + 1, 3 * B - 1, 0, 5 * B + B // 2, 4 * B]
    new = [1, B, 1, 2 * B, 0, B + B // 2 + 1, 0]
    p = Pool(lens, D=D, B=B, dtype=dtype, e4m3=e4m3, seed=B)
    before = torch.full_like(p.bounds, 3.5)
    p.bounds.copy_(before)
    pk.key_bounds(p.bounds, p.kc, p.tables, p.context, p.max_len, torch.tensor(new, dtype=torch.int32, device="cuda"),
                  max(new), dev_status=p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    want = before.double()
    for s, (L, m) in enumerate(zip(lens, new)):
        for j in range((L - m) // B, -(-L // B)) if m else ():
            want[p.tables[s, j].long()] = p.want_bounds(s, j)
    assert torch.equal(p.bounds.double(), want)


def test_bounds_default_is_the_newest_block():
    p = Pool([16, 17, 1, 40, 0])
    before = p.bounds.clone()
    pk.key_bounds(p.bounds, p.kc, p.tables, p.context, p.max_len, dev_status=p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    touched = torch.zeros(p.num_blocks, dtype=torch.bool)
    for s, j in ((0, 0), (1, 1), (2, 0), (3, 2)):
        blk = int(p.tables[s, j])
        touched[blk] = True
        assert torch.equal(p.bounds[blk].double(), p.want_bounds(s, j))
    assert bool(p.bounds[~touched].isnan().all()) and bool(before.isnan().all())


def test_bounds_nan_and_infinite_keys():
    p = Pool([48], dtype="f16")
    b = p.tables[0].tolist()
    p.kc[b[0], 0, 3, 5] = float("nan")
    p.kc[b[1], 1, 2, 7] = float("inf")
    p.kc[b[2], 1, 2, 9] = float("-inf")
    p.fill_bounds()
    torch.cuda.synchronize()
    got = p.bounds.double()
    nan = torch.zeros_like(got[b[0], 0], dtype=torch.bool)
    nan[:, 5] = True
    assert torch.equal(got[b[0], 0].isnan(), nan)
    assert got[b[1], 1, 1, 7] == float("inf") and got[b[2], 1, 0, 9] == float("-inf")
    for j in range(3):
        want = p.want_bounds(0, j)
        assert torch.equal(torch.nan_to_num(got[b[j]], 1e9), torch.nan_to_num(want, 1e9))


def test_bounds_bad_data_is_flagged_and_skipped():
    p = Pool([32, 32, 32, 32])
    p.tables[0, 1] = p.num_blocks
    p.tables[1, 1] = -7
    new = torch.tensor([1, 1, 33, -1], dtype=torch.int32, device="cuda")
    pk.key_bounds(p.bounds, p.kc, p.tables, p.context, 32, new, 40, dev_status=p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == pk.DEV_BAD_BLOCK_ID | pk.DEV_BAD_LEN
    assert bool(p.bounds.isnan().all())
    p.status.zero_()
    p.context[2], p.context[3] = -5, 1000
    pk.key_bounds(p.bounds, p.kc, p.tables[2:].contiguous(), p.context[2:].contiguous(), 32, dev_status=p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == pk.DEV_BAD_LEN and bool(p.bounds.isnan().all())


# ------------------------------------------------------------------ sparse decode

@pytest.mark.parametrize("dtype,e4m3", [("f32", False), ("f16", False), ("bf16", False), ("f16", True), ("bf16", True)])
@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 128, 16), (4, 4, 64, 16), (6, 2, 256, 16), (16, 1, 128, 32),
                                        (8, 2, 64, 5), (5, 1, 128, 8), (64, 2, 128, 16)])
def test_types_and_heads(dtype, e4m3, Hq, Hkv, D, B):
    lens = [B * 40 + 3, 1, B * 12, 0, B * 25 + 1, B * 11 - 1, B * 13]
    p = Pool(lens, Hq, Hkv, D, B, dtype, e4m3, seed=D + B)
    p.fill_bounds()
    out, sel = p.decode(12, 1, 2)
    assert int(p.status.item()) == 0
    p.check(out, sel, 12, 1, 2)


@pytest.mark.parametrize("K,first,recent", [(1, 0, 1), (2, 1, 1), (3, 0, 3), (5, 0, 1), (40, 2, 3), (200, 1, 1),
                                            (1000, 7, 9)])
def test_selection_sizes(K, first, recent):
    p = Pool([16 * 300 + 5, 16 * 41, 16 * 200 - 3, 700], seed=K)
    p.fill_bounds()
    out, sel = p.decode(K, first, recent)
    assert int(p.status.item()) == 0
    p.check(out, sel, K, first, recent)


@pytest.mark.parametrize("lens,K", [([30000], 64), ([40001, 3, 9000], 100), ([131072], 33)])
def test_long_contexts(lens, K):
    p = Pool(lens, 8, 2, seed=1)
    p.fill_bounds()
    out, sel = p.decode(K, 1, 2)
    assert int(p.status.item()) == 0
    p.check(out, sel, K, 1, 2)


@pytest.mark.parametrize("dtype,e4m3", [("f16", False), ("bf16", True), ("f32", False)])
def test_long_contexts_of_other_types(dtype, e4m3):
    p = Pool([33333, 20001], 8, 2, dtype=dtype, e4m3=e4m3, seed=2)
    p.fill_bounds()
    out, sel = p.decode(70, 2, 1)
    assert int(p.status.item()) == 0
    p.check(out, sel, 70, 2, 1)


@pytest.mark.parametrize("L,B,K,first", [(400003, 16, 40, 1), (30001, 1, 50, 0), (12000, 1, 9000, 3), (150000, 8, 33, 2)])
def test_more_blocks_than_shared_memory_keeps(L, B, K, first):
    p = Pool([L, 17 * B], 4, 1, 64, B, seed=4)
    p.fill_bounds()
    out, sel = p.decode(K, first, 2)
    assert int(p.status.item()) == 0
    p.check(out, sel, K, first, 2)


@pytest.mark.parametrize("group", [1, 3, 8, 9, 64, 128])
def test_every_group_size(group):
    p = Pool([16 * 60 + 1, 16 * 300], group * 2, 2, 64, seed=group)
    p.fill_bounds()
    out, sel = p.decode(20)
    assert int(p.status.item()) == 0
    p.check(out, sel, 20)


@pytest.mark.parametrize("lens,K", [([1500, 30, 900, 0], 70), ([64 * 16 + 3], 60), ([49 * 16, 1, 48 * 16], 100),
                                    ([300] * 20 + [2000], 90), ([900] * 37, 50)])
@pytest.mark.parametrize("D,e4m3", [(128, False), (64, True), (256, False)])
def test_short_contexts_shared_by_a_cluster(lens, K, D, e4m3):
    # few blocks to score, many to attend to: some CTAs of a cluster have neither
    p = Pool(lens, 8, 2, D, e4m3=e4m3, seed=K)
    p.fill_bounds()
    out, sel = p.decode(K, 1, 2)
    assert int(p.status.item()) == 0
    p.check(out, sel, K, 1, 2)


def test_close_scores_in_a_crowd():
    # many blocks whose scores differ by less than the approximate scores' error, ties among them
    p = Pool([16 * 700], Hq=4, Hkv=1, D=128, seed=5)
    p.fill_bounds()
    blk = p.tables[0].long()
    base = p.bounds[blk[0]].clone()
    g = torch.Generator().manual_seed(7)
    step = torch.randint(0, 40, (700,), generator=g).cuda()
    p.bounds[blk] = base
    p.bounds[blk, 0, 1, 17] = (2.0 ** -6 * (1 + step * 2.0 ** -7)).to(p.dt)          # the only difference
    p.query[..., 17] = 2.0 ** -8
    for K in (30, 200, 500):
        out, sel = p.decode(K, 1, 1)
        p.check(out, sel, K, 1, 1)


def test_many_sequences():
    lens = [(37 * i) % 900 for i in range(300)]
    p = Pool(lens, 8, 2, 64, seed=3)
    p.fill_bounds()
    out, sel = p.decode(10, 1, 1)
    assert int(p.status.item()) == 0
    p.check(out, sel, 10)


def test_all_blocks_equals_the_dense_decode_of_a_head():
    # every block selected: the plain decode's result, up to rounding order
    p = Pool([1000, 513, 16], seed=6)
    p.fill_bounds()
    out, sel = p.decode(63)
    dense = torch.empty_like(out)
    pk.decode(dense, p.query, p.kc, p.vc, p.tables, p.context, p.max_len, p.scale)
    torch.cuda.synchronize()
    assert bool(((out.float() - dense.float()).abs() <= 2.0 ** -7 * dense.float().abs() + 2.0 ** -11).all())
    p.check(out, sel, 63)


def test_ties_go_to_the_lowest_block():
    for e4m3 in (False, True):
        p = Pool([16 * 100, 16 * 77 + 1], seed=8, e4m3=e4m3)
        for s in range(2):                                   # keys alike in all blocks, then a few better ones
            blk = p.tables[s, :p.lens[s] // 16].long()
            p.kc[blk] = p.kc[blk[0]].clone()
        p.fill_bounds()
        out, sel = p.decode(9, 0, 1)
        assert sel[0, 0].tolist() == list(range(8)) + [99] and sel[1, 1].tolist() == list(range(8)) + [77]
        p.check(out, sel, 9, 0, 1)
    p = Pool([16 * 300], seed=8)
    p.query.zero_()                                          # all scores zero
    p.fill_bounds()
    out, sel = p.decode(50, 2, 3)
    p.check(out, sel, 50, 2, 3)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_scores_that_binary32_cannot_tell_apart(dtype):
    # a large common part and differences far below its binary32 step decide the order
    p = Pool([16 * 64], Hq=2, Hkv=2, D=64, dtype=dtype, seed=9)
    p.fill_bounds()
    p.query.fill_(0)
    p.query[..., 0], p.query[..., 1] = 256.0, 2.0 ** -9
    blk = p.tables[0].long()
    p.bounds.zero_()
    p.bounds[blk, :, 1, 0] = 1.0
    p.bounds[blk, :, 1, 0] += torch.where(torch.arange(64, device="cuda") % 7 == 3, 2.0 ** -7, 0.0).to(p.dt)[:, None]
    order = torch.randperm(64, generator=torch.Generator().manual_seed(1)).cuda()
    p.bounds[blk, :, 1, 1] = (order[:, None] * 2.0 ** -8).to(p.dt)            # exact in every type
    out, sel = p.decode(20, 0, 1)
    p.check(out, sel, 20, 0, 1)


@pytest.mark.parametrize("dtype,size", [("bf16", 2.0 ** -66), ("bf16", 2.0 ** -80), ("bf16", 2.0 ** 63), ("bf16", 2.0 ** 90),
                                        ("f32", 2.0 ** -60), ("f32", 2.0 ** -70), ("f16", 2.0 ** -12)])
def test_very_small_and_large_magnitudes(dtype, size):
    # the squares of these pass binary32's range at either end
    p = Pool([16 * 120], dtype=dtype, seed=11)
    p.fill_bounds()
    p.bounds.copy_((p.bounds.double().nan_to_num(0) * size).to(p.dt))
    p.query.copy_((p.query.double() * size).to(p.dt))
    sel = p.decode(15, 1, 1)[1]
    for h in range(2):
        assert sel[0, h].tolist() == p.want_selected(0, h, 15, 1, 1)


def test_infinite_and_nan_bounds_come_first():
    p = Pool([16 * 60], dtype="f16", seed=10)
    p.fill_bounds()
    blk = p.tables[0].long()
    p.bounds[blk[40], 0, 1] = float("inf")
    p.bounds[blk[41], 0] = float("nan")
    p.bounds[blk[42], 1] = float("-inf")
    p.query[0, 0, 3] = 0.0
    out, sel = p.decode(5, 1, 1)
    assert sel[0, 0].tolist() == p.want_selected(0, 0, 5, 1, 1) and {40, 41} <= set(sel[0, 0].tolist())
    assert sel[0, 1].tolist() == p.want_selected(0, 1, 5, 1, 1)
    p.query[0, 5] = float("nan")                             # every score of head 1 is NaN: the lowest blocks
    out, sel = p.decode(5, 1, 1)
    assert sel[0, 1].tolist() == [0, 1, 2, 3, 59]


def test_bad_table_entries_and_lengths_are_flagged():
    p = Pool([16 * 50, 16 * 50, 100])
    p.fill_bounds()
    p.tables[0, 0] = p.num_blocks + 3                        # always selected: the decode meets it
    p.tables[1, 20] = -1                                     # scored: skipped unless nothing else is left
    out, sel = p.decode(8, 1, 1)
    assert int(p.status.item()) == pk.DEV_BAD_BLOCK_ID
    assert 20 not in sel[1, 0].tolist()
    p.status.zero_()
    p.context[2] = -3
    p.decode(8, 1, 1)
    assert int(p.status.item()) & pk.DEV_BAD_LEN


def test_padded_batch_workspace_reuse_and_graph():
    p = Pool([16 * 90 + 1, 0, 16 * 33, 0], seed=12)
    p.fill_bounds()
    ws = pk.alloc_sparse_workspace(p.S, p.Hq, p.Hkv, p.D, p.B, p.max_len, 16)
    ws.fill_(0xFF)
    out, sel = p.decode(16, 1, 2, ws)
    p.check(out, sel, 16, 1, 2)
    again, sel2 = p.decode(16, 1, 2, ws)
    assert torch.equal(out, again) and torch.equal(sel, sel2)
    # captured, with the lengths changed before the replay
    side, o2, s2 = torch.cuda.Stream(), torch.empty_like(out), torch.empty_like(sel)
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pk.sparse_decode(o2, p.query, p.kc, p.vc, p.bounds, p.tables, p.context, p.max_len, p.scale, 16, ws, 1, 2,
                             selected=s2, dev_status=p.status)
        graph.replay()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, o2) and torch.equal(sel, s2)
    p.lens = [16 * 70, 0, 16 * 20 + 0, 0]
    p.context.copy_(torch.tensor(p.lens, dtype=torch.int32))
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.synchronize()
    p.check(o2, s2, 16, 1, 2)


def test_two_calls_at_once_on_two_streams():
    a, b = Pool([16 * 200, 777], seed=13), Pool([16 * 150 + 9, 3001], seed=14)
    a.fill_bounds()
    b.fill_bounds()
    torch.cuda.synchronize()
    want = [x.decode(11)[0].clone() for x in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [torch.empty_like(w) for w in want]
    ws = [pk.alloc_sparse_workspace(x.S, x.Hq, x.Hkv, x.D, x.B, x.max_len, 11) for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, o, w, st in zip((a, b), got, ws, streams):
            pk.sparse_decode(o, x.query, x.kc, x.vc, x.bounds, x.tables, x.context, x.max_len, x.scale, 11, w,
                             stream=st)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_draft_tokens_as_rows():
    # four query tokens of one sequence: the table repeated, each with the length it sees
    p = Pool([16 * 80 + 2], seed=15)
    p.fill_bounds()
    rows = Pool([16 * 80 + 2 - 3 + i for i in range(4)], seed=15, max_blocks=81)
    rows.kc, rows.vc, rows.bounds, rows.num_blocks = p.kc, p.vc, p.bounds, p.num_blocks
    rows.tables = p.tables.expand(4, -1).contiguous()
    out, sel = rows.decode(10, 1, 2)
    assert int(rows.status.item()) == 0
    rows.check(out, sel, 10, 1, 2)


def test_wrong_arguments():
    p = Pool([100])
    ws = pk.alloc_sparse_workspace(1, 8, 2, 128, 16, 100, 4)
    call = lambda **kw: pk.sparse_decode(**{**dict(                                       # noqa: E731
        out=p.query.clone(), query=p.query, k_cache=p.kc, v_cache=p.vc, k_bounds=p.bounds, block_tables=p.tables,
        context_lens=p.context, max_context_len=100, scale=0.1, num_select=4, workspace=ws), **kw})
    for kw in (dict(num_select=0), dict(first_blocks=-1), dict(recent_blocks=0), dict(first_blocks=3, recent_blocks=2),
               dict(scale=0.0), dict(scale=-1.0), dict(workspace=ws[:128]), dict(workspace=ws[1:])):
        with pytest.raises(pk.PagedKVError):
            call(**kw)
    for kw in (dict(k_bounds=p.bounds.float()), dict(k_bounds=p.bounds[:1]), dict(out=p.query.float()),
               dict(selected=torch.zeros(1, 2, 5, dtype=torch.int32, device="cuda")),
               dict(selected=torch.zeros(1, 2, 4, device="cuda")), dict(workspace=ws.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(ValueError):
        pk.key_bounds(p.bounds[:, :1], p.kc, p.tables, p.context, 100)
    with pytest.raises(pk.PagedKVError):                     # max_new_tokens without new_tokens
        pk.key_bounds(p.bounds, p.kc, p.tables, p.context, 100, max_new_tokens=2)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 128, 16), (32, 2, 128, 16), (8, 2, 128, 8), (4, 4, 256, 16), (16, 1, 256, 16),
                                        (6, 2, 64, 16), (32, 2, 64, 16), (6, 2, 128, 7)])
@pytest.mark.parametrize("K,first", [(70, 1), (7, 0)])
def test_nan_codes_of_an_e4m3_pool_show(dtype, Hq, Hkv, D, B, K, first):
    """A NaN code in a selected token: a key's makes its head's rows NaN, a value's its component; all else keeps
    the tolerances. (The codes behind a context's end are NaN throughout.)"""
    lens = [1, B, 20 * B + 3, 60 * B, 33 * B + 1]
    G = Hq // Hkv
    for code in (0x7F, 0xFF):
        for cache in ("key", "value"):
            p = Pool(lens, Hq, Hkv, D, B, dtype, True, seed=B + D)
            bad = [(0, 0, 0, 3), (2, 20 * B + 2, 0, D - 1), (3, 0, Hkv - 1, 17), (4, 33 * B, Hkv - 1, D // 2)]
            for s, t, h, d in bad:                       # the first and the newest block: selected (a NaN key always is)
                if first or cache == "key" or t >= p.B * (-(-lens[s] // p.B) - 1):
                    (p.kc if cache == "key" else p.vc)[p.tables[s, t // B].long(), h, t % B, d] = code
            p.fill_bounds()
            out, sel = p.decode(K, first)
            want = torch.zeros(out.shape, dtype=torch.bool)
            for s, t, h, d in bad:
                if (p.kc if cache == "key" else p.vc)[p.tables[s, t // B].long(), h, t % B, d].item() == code:
                    want[s, h * G:(h + 1) * G, slice(None) if cache == "key" else d] = True
            assert torch.equal(out.isnan().cpu(), want), (code, cache)
            for s, L in enumerate(lens):
                for h in range(Hkv):
                    blocks = [b for b in sel[s, h].tolist() if b >= 0]
                    assert blocks == p.want_selected(s, h, K, first, 1)
                    tok = torch.tensor([b * B + i for b in blocks for i in range(B) if b * B + i < L])
                    blk = p.tables[s].long()[(tok // B).cuda()]
                    k, v = (p.keys(c)[blk, h, (tok % B).cuda()] for c in (p.kc, p.vc))
                    w = torch.softmax(p.query[s, h * G:(h + 1) * G].double() @ k.t() * (p.scale * p.ks), -1)
                    ref, mass = w @ v * p.vs, w @ v.abs() * p.vs
                    tol = torch.finfo(p.dt).eps / 2 * ref.abs() + WEIGHTS["e4m3"] * mass
                    got = out[s, h * G:(h + 1) * G].double()
                    assert bool((((got - ref).abs() <= tol) | (got.isnan() & ref.isnan())).all())


@pytest.mark.parametrize("dtype,e4m3,Hq", [("bf16", False, 8), ("f16", False, 8), ("bf16", True, 8), ("f16", True, 8),
                                           ("f16", False, 32), ("bf16", True, 32), ("f16", True, 32)])
def test_weights_keep_their_bits(dtype, e4m3, Hq):
    """Values that cancel against the exact weights (64 contexts of one block; each head in a share of the
    components), so that the output's rounding is negligible and what is left is the weights' error. Tolerance,
    against sum_i p_i |v_i|: one component of the query is not zero and |scale q k log2 e| <= 2, so a weight errs by
    ex2.approx's 2^-22 and by the rounding of its argument, below 8 with the reference's shift: 2^-22 ln 2; the
    products' sum loses up to 17 2^-23 of its largest term, about a sixth of the whole: 2^-21.5. Together 2^-20.2."""
    S, Hkv, D, B = 64, 2, 128, 16
    G = Hq // Hkv
    p = Pool([B] * S, Hq, Hkv, D, B, dtype, e4m3, seed=5)
    g = torch.Generator().manual_seed(6)
    cast = (lambda x: (x.clamp(-448, 448)).to(torch.float8_e4m3fn)) if e4m3 else (lambda x: x.to(p.dt))
    back = lambda x: x.view(torch.uint8) if e4m3 else x
    p.ks, p.vs, p.scale = (2.0 ** -6, 0.027, 1.0) if e4m3 else (1.0, 1.0, 1.0)
    k = cast(torch.rand((S, Hkv, B), generator=g) * (1.38 / p.ks))
    q = (0.7 + 0.3 * torch.rand((S, Hkv, G), generator=g)).to(p.dt)
    w = torch.softmax((q.double().unsqueeze(-1) * k.double().unsqueeze(2)) * p.ks, -1)          # [S, Hkv, G, B]
    head = torch.arange(D) * G // D
    w = w[:, :, head].transpose(2, 3)                                                         # [S, Hkv, B, D]
    v = torch.zeros((S, Hkv, B, D), dtype=torch.float64)
    left = torch.zeros((S, Hkv, D), dtype=torch.float64)
    top = 200.0 if e4m3 else 1.0
    for t in range(B):
        new = top * torch.randn((S, Hkv, D), generator=g).double() if t < 4 else -left / w[:, :, t]
        v[:, :, t] = cast(new.float()).double()
        left += w[:, :, t] * v[:, :, t]
    blocks = p.tables[:, 0].long()
    p.kc.zero_(), p.query.zero_()
    p.kc[blocks, :, :, 0] = back(k).cuda()
    p.vc[blocks] = back(cast(v.float())).cuda()
    p.query.view(S, Hkv, G, D)[..., 0] = q.cuda()
    p.fill_bounds()
    out, _ = p.decode(4)
    got = out.view(S, Hkv, G, D).gather(2, head.view(1, 1, 1, D).expand(S, Hkv, 1, D).cuda()).squeeze(2).double().cpu()
    mass = (w * v.abs()).sum(2) * p.vs
    ref = left * p.vs
    tol = torch.finfo(p.dt).eps / 2 * ref.abs() + 2.0 ** -20 * mass + (2.0 ** -25 if dtype == "f16" else 0.0)
    assert float((ref.abs() / mass).max()) < 2.0 ** -9
    assert bool(((got - ref).abs() <= tol).all()), float(((got - ref).abs() / mass).max())


@pytest.mark.parametrize("dtype,Hq,B,size", [("bf16", 8, 16, 2.0 ** -96), ("bf16", 8, 16, 2.0 ** -120), ("bf16", 32, 16, 2.0 ** -110),
                                             ("bf16", 8, 5, 2.0 ** -110), ("f32", 8, 16, 2.0 ** -80), ("f32", 8, 16, 2.0 ** -140),
                                             ("f32", 32, 16, 2.0 ** -100)])
def test_products_that_all_underflow(dtype, Hq, B, size):
    """Query and bounds whose products pass below binary32's range (bfloat16's range too, with 2^40 to spare): the
    order is that of the exact scores all the same. One sequence each with a zero query, and with zero keys (but for
    one that is not, in the last)."""
    p = Pool([B * 120, B * 97 + 1, B * 50, B * 600], Hq, 2, 128, B, dtype, seed=13)
    p.fill_bounds()
    p.bounds.copy_((p.bounds.double().nan_to_num(0) * size).to(p.dt))
    p.query.copy_((p.query.double() * size).to(p.dt))
    assert bool((p.query != 0).any()) and bool((p.bounds != 0).any())
    p.query[1] = 0
    p.bounds[p.tables[2, :50].long()] = 0
    p.bounds[p.tables[3].long()] = 0
    p.bounds[p.tables[3, 571].long(), :, 1, 77] = size
    sel = p.decode(15, 1, 1)[1]
    for s in range(4):
        for h in range(2):
            assert sel[s, h].tolist() == p.want_selected(s, h, 15, 1, 1), (s, h)


def spread(shape, g, bits):
    """Signed magnitudes log-uniform over 2^-bits .. 2^bits."""
    x = torch.exp2((2 * torch.rand(shape, generator=g, device="cuda") - 1) * bits)
    return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.5, -x, x)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D,G", [(64, 1), (64, 12), (128, 8), (128, 16), (256, 4), (256, 9)])
@pytest.mark.parametrize("values", ["normal", "spread", "one sign", "cancelling"])
def test_approximate_scores_err_less_than_the_selection_takes_them_to(dtype, D, G, values):
    """A context of more blocks than shared memory keeps scores for leaves its approximate scores at the start of the
    workspace (bfloat16's times 2^40): each within 2^-16 of the sum of its terms' magnitudes, as the selection
    assumes (a quarter of it here: the margin)."""
    n, B, dt = 25000, 1, TYPES[dtype]
    g = torch.Generator(device="cuda").manual_seed(D + G)
    query = torch.randn((1, G, D), generator=g, device="cuda")
    bounds = torch.randn((n, 1, 2, D), generator=g, device="cuda")
    if values == "spread":
        query, bounds = spread(query.shape, g, 4), spread(bounds.shape, g, 8)
    elif values == "one sign":
        query, bounds = 1 + torch.rand(query.shape, generator=g, device="cuda"), 1 + torch.rand(bounds.shape, generator=g, device="cuda")
    elif values == "cancelling":                       # the second half of the components takes the first half's sum back
        query[..., D // 2:] = -query[..., :D // 2]
        half = torch.randn((n, 1, 1, D // 2), generator=g, device="cuda").to(dt).float()
        bounds = torch.cat((half, half), -1).expand(n, 1, 2, D).contiguous()
        bounds[:, :, :, -1] += torch.rand((n, 1, 1), generator=g, device="cuda") * 4    # (so that the best ones are clear)
    query, bounds = query.to(dt), bounds.to(dt)
    lo, hi = torch.minimum(bounds[:, :, 0], bounds[:, :, 1]), torch.maximum(bounds[:, :, 0], bounds[:, :, 1])
    bounds = torch.stack((lo, hi), 2)
    cache = torch.zeros((n, 1, B, D), device="cuda", dtype=dt)
    table = torch.arange(n, device="cuda", dtype=torch.int32).view(1, n)
    context = torch.full((1,), n * B, device="cuda", dtype=torch.int32)
    ws = pk.alloc_sparse_workspace(1, G, 1, D, B, n * B, 50)
    out = torch.empty_like(query)
    pk.sparse_decode(out, query, cache, cache, bounds, table, context, n * B, 1.0, 50, ws, 0, 1)
    got = ws[:4 * (n - 1)].view(torch.float32).double() * (2.0 ** -40 if dtype == "bf16" else 1.0)
    q, b = query[0].double(), bounds[:n - 1, 0].double()                       # [G, D], [n, 2, D]
    neg, pos = q.clamp(max=0), q.clamp(min=0)
    want = (neg @ b[:, 0].t() + pos @ b[:, 1].t()).amax(0)
    mag = (neg.abs() @ b[:, 0].abs().t() + pos @ b[:, 1].abs().t()).amax(0)
    taken = torch.isinf(got) | torch.isnan(got)                                # marked by the search, where that was needed
    assert int(taken.sum()) < n // 2
    worst = float(((got - want).abs() / mag)[~taken].max())
    assert worst <= 2.0 ** -18, worst


def test_subnormal_bounds_and_query_elements_count():
    """bfloat16 bounds, and query elements, below its normal range decide where others are level."""
    for swap in (False, True):
        p = Pool([16 * 200], 8, 2, 128, 16, seed=17)
        p.bounds.zero_()
        p.query.zero_()
        tiny = (torch.arange(p.num_blocks, device="cuda") * 37 % 113 + 1).double() * 2.0 ** -133
        p.query[..., 0], p.query[..., 1] = 2.0 ** 100, 2.0 ** -20
        p.bounds[:, :, :, 0] = tiny.to(p.dt).view(-1, 1, 1)
        p.bounds[:, :, :, 1] = 2.0 ** -30
        if swap:
            p.query[..., 0] = 2.0 ** -132
            p.bounds[:, :, :, 0] = (tiny * 2.0 ** 233).to(p.dt).view(-1, 1, 1)
        sel = p.decode(15, 1, 1)[1]
        for h in range(2):
            assert sel[0, h].tolist() == p.want_selected(0, h, 15, 1, 1)


@pytest.mark.parametrize("dtype,e4m3", [("bf16", False), ("f32", False), ("f16", True)])
def test_bounds_of_a_block_that_several_sequences_name(dtype, e4m3):
    """Sequences that see the same tokens of a block give its bounds; of those that see different ones, every
    element is that of one of them. The longest alone (rows of one sequence's query tokens) gives the longest's."""
    p = Pool([16 * 40 + 9], dtype=dtype, e4m3=e4m3, seed=21)
    L = p.lens[0]
    newest = p.tables[0, L // 16].long()
    full = torch.stack([p.want_bounds(0, j) for j in range(L // 16)])
    ends = []
    for m in (3, 6, 9):
        k = p.keys(p.kc[newest])[:, :m]
        ends.append(torch.stack((k.amin(1), k.amax(1)), 1))
    lens = [L - 6, L, L - 3, L] * 16
    rows = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pk.key_bounds(p.bounds, p.kc, p.tables.expand(64, -1).contiguous(), rows, L, rows, L, dev_status=p.status)
    torch.cuda.synchronize()
    assert int(p.status.item()) == 0
    assert torch.equal(p.bounds[p.tables[0, :L // 16].long()].double(), full)
    got = p.bounds[newest].double()
    assert bool(torch.stack([got == e for e in ends]).any(0).all())
    pk.key_bounds(p.bounds, p.kc, p.tables, p.context, L, dev_status=p.status)
    assert torch.equal(p.bounds[newest].double(), ends[2])


@pytest.mark.parametrize("Hq,Hkv,D,B", [(8, 2, 128, 16), (32, 2, 128, 16), (16, 1, 256, 16), (8, 2, 128, 8), (32, 2, 64, 16)])
@pytest.mark.parametrize("sizes", [(2.0 ** 20, 2.0 ** 30), (2.0 ** -30, 2.0 ** -18), (2.0 ** 40, 2.0 ** -40)])
def test_e4m3_pools_with_queries_beyond_binary16(Hq, Hkv, D, B, sizes):
    """bfloat16 queries far above and below binary16's range, heads of one group of different size: the scores have
    the precision of ordinary ones (each head's scale brings them to the same logits as size 1 would)."""
    lens = [1, 300, 40 * B]
    for size in sizes:
        p = Pool(lens, Hq, Hkv, D, B, "bf16", True, seed=41)
        p.query.copy_((p.query.double() * size).to(p.dt))
        p.query[:, ::2] /= 4.0
        p.scale /= size
        p.fill_bounds()
        out, sel = p.decode(20)
        p.check(out, sel, 20)
