"""The append with norms and rotation, the key bounds and the block-sparse
decode run together, as a serving loop would: a prompt in chunks, then decode
steps, with the library's block allocator. Every step's cache, bounds,
selection and output are held to 64-bit forms computed from the unrotated
projections."""
import numpy as np
import pytest
import torch

from paged_kv_cache_141_gb300 import binding as pk
from test_gpu_rope import Step, table
from test_gpu_sparse import Pool

pytestmark = pytest.mark.gpu


class Loop:
    """Sequences that grow together over one pool. The parent classes' checks
    are reused: Pool for bounds, selection and attention, Step for the append."""

    def __init__(self, prompts, steps, dtype, e4m3, B=16, Hq=8, Hkv=2, D=128, seed=0):
        self.B, self.Hq, self.Hkv, self.D, self.steps = B, Hq, Hkv, D, steps
        S = self.S = len(prompts)
        total = [p + steps for p in prompts]
        pages = sum(-(-t // B) for t in total) + 1
        self.alloc = pk.BlockAllocator(pages, B)
        self.width = max(-(-t // B) for t in total)
        self.pool = Pool([0] * S, Hq, Hkv, D, B, dtype, e4m3, seed, max_blocks=self.width)
        p = self.pool
        nan = 0x7F if e4m3 else float("nan")
        shape = (pages, Hkv, B, D)
        p.kc, p.vc = (torch.full(shape, nan, dtype=p.kc.dtype, device="cuda") for _ in range(2))
        p.bounds = torch.full((pages, Hkv, 2, D), float("nan"), dtype=p.dt, device="cuda")
        p.num_blocks, p.max_len = pages, max(total)
        self.host_tables = [[np.zeros(self.width, np.int32), 0] for _ in prompts]
        self.lens = [0] * S
        g = torch.Generator().manual_seed(seed + 1)
        self.g, self.dt, self.e4m3 = g, p.dt, e4m3
        self.cos_sin = table(p.max_len, D)
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2))
        self.ks, self.vs = (0.02, 0.025) if e4m3 else (1.0, 1.0)
        p.ks, p.vs = self.ks, self.vs
        self.K = 12
        self.ws = pk.alloc_sparse_workspace(S, Hq, Hkv, D, B, p.max_len, self.K)

    def append(self, new):
        """new[s] more tokens for every sequence, one call."""
        slots, positions = [], []
        for s, m in enumerate(new):
            for i in range(m):
                at = self.lens[s] + i
                arr, n = self.host_tables[s]
                slot, n, copy = self.alloc.append_slot((arr, n), at)
                assert copy is None
                self.host_tables[s][1] = n
                slots.append(slot)
                positions.append(at)
            self.lens[s] += m
        T = len(slots)
        st = Step.__new__(Step)
        st.dims = (T, self.Hq, self.Hkv, self.D, self.D, self.B)
        qkv = torch.randn((T, self.Hq + 2 * self.Hkv, self.D), generator=self.g).to(self.dt).cuda()
        st.q, st.k, st.v = qkv.split((self.Hq, self.Hkv, self.Hkv), 1)
        st.num_blocks, st.axes, st.freq_axes, st.adjacent = self.pool.num_blocks, 1, None, False
        st.slots = torch.tensor(slots, dtype=torch.int64, device="cuda")
        st.positions = torch.tensor([positions], dtype=torch.int64, device="cuda")
        st.cos_sin, st.kc, st.vc = self.cos_sin, self.pool.kc, self.pool.vc
        st.e4m3, st.dt, st.qw, st.kw, st.eps = self.e4m3, self.dt, self.qw, self.kw, 1e-6
        st.ks, st.vs = self.ks, self.vs
        st.out = torch.empty((T, self.Hq, self.D), dtype=self.dt, device="cuda")
        st.status = self.pool.status
        before = st.kc.clone(), st.vc.clone()
        assert st.run() == 0
        # the new tokens by their formula; every other slot as it was
        y, err = st.rotated(st.q, st.qw)
        assert bool(((st.out.double() - y).abs() <= torch.finfo(self.dt).eps / 2 * y.abs() + err + 2.0 ** -25).all())
        flat = [c.transpose(1, 2).reshape(-1, self.Hkv, self.D) for c in (st.kc, st.vc, *before)]
        rest = torch.ones(flat[0].shape[0], dtype=torch.bool, device="cuda")
        rest[st.slots] = False
        for now, was in ((flat[0], flat[2]), (flat[1], flat[3])):
            bits = torch.uint8 if self.e4m3 else torch.int16
            assert torch.equal(now[rest].view(bits), was[rest].view(bits))
        y, err = st.rotated(st.k, st.kw)
        if self.e4m3:
            got = flat[0].view(torch.float8_e4m3fn).double()[st.slots]
            y = (y / self.ks).clamp(-448, 448)
            tol = 2.0 ** -4 * y.abs() + 2.0 ** -10 + 2 * err / self.ks
        else:
            got = flat[0].double()[st.slots]
            tol = torch.finfo(self.dt).eps / 2 * y.abs() + err + 2.0 ** -25
        assert bool(((got - y).abs() <= tol).all())
        p = self.pool
        p.lens = list(self.lens)
        p.context.copy_(torch.tensor(self.lens, dtype=torch.int32))
        p.tables.copy_(torch.from_numpy(np.stack([t for t, _ in self.host_tables])))
        return st.out

    def bounds(self, new):
        p = self.pool
        pk.key_bounds(p.bounds, p.kc, p.tables, p.context, p.max_len, torch.tensor(new, dtype=torch.int32).cuda(),
                      max(new), dev_status=p.status)
        torch.cuda.synchronize()
        for s, L in enumerate(self.lens):
            for j in range(-(-L // self.B)):
                assert torch.equal(p.bounds[p.tables[s, j].long()].double(), p.want_bounds(s, j)), (s, j)


@pytest.mark.parametrize("dtype,e4m3", [("bf16", False), ("f16", False), ("bf16", True)])
def test_serving_loop(dtype, e4m3):
    prompts, steps = [300, 37, 511], 12
    loop = Loop(prompts, steps, dtype, e4m3, seed=21)
    for chunk in (100, 211, 200):                            # the prompts in chunks, ragged at the end
        new = [max(0, min(chunk, n - L)) for n, L in zip(prompts, loop.lens)]
        loop.append(new)
        loop.bounds(new)
    p = loop.pool
    for step in range(steps):
        p.query = loop.append([1] * loop.S)
        loop.bounds([1] * loop.S)
        out, sel = p.decode(loop.K, 1, 2, loop.ws)
        assert int(p.status.item()) == 0
        p.check(out, sel, loop.K, 1, 2)
    # a selection of every block is the decode over the same pool
    out, _ = p.decode(loop.width)
    dense = torch.empty_like(out)
    pk.decode_auto(dense, p.query, p.kc, p.vc, p.tables, p.context, p.max_len, p.scale, None, 512, p.ks, p.vs)
    torch.cuda.synchronize()
    # (both round their output, and each one's weights are off by at most 2^-9 of sum p |v| < 1)
    eps = torch.finfo(p.dt).eps
    assert bool(((out.float() - dense.float()).abs() <= 2 * eps * dense.float().abs() + 2.0 ** -8).all())


def test_caches_past_32_bit_offsets():
    """Blocks whose element offsets pass 2^32: append, bounds and sparse decode there."""
    Hq, Hkv, D, B = 8, 8, 128, 16
    nb = 2 ** 32 // (Hkv * B * D) + 40
    kc, vc = (torch.empty((nb, Hkv, B, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    bounds = torch.empty((nb, Hkv, 2, D), dtype=torch.bfloat16, device="cuda")
    blocks = torch.arange(nb - 24, nb, dtype=torch.int32)
    T = 24 * B - 5
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g).to(torch.bfloat16).cuda()
    q, k, v = qkv.split((Hq, Hkv, Hkv), 1)
    out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    at = torch.arange(T)
    slots = (blocks.long()[at // B] * B + at % B).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk.rope_and_cache(out, q, k, v, kc, vc, table(T, D), at.cuda(), slots, dev_status=status)
    small = Pool([T], Hq, Hkv, D, B)
    small.kc, small.vc = kc[nb - 24:].clone(), vc[nb - 24:].clone()       # the same blocks at small offsets
    ctx = torch.tensor([T], dtype=torch.int32, device="cuda")
    pk.key_bounds(bounds, kc, blocks[None].cuda(), ctx, T, ctx, T, dev_status=status)
    small.tables, small.context, small.max_blocks = torch.arange(24, dtype=torch.int32, device="cuda")[None], ctx, 24
    small.bounds = bounds[nb - 24:].clone()
    small.query = out[-1:].clone()
    for s in range(24):
        assert torch.equal(small.bounds[s].double(), small.want_bounds(0, s))
    ws = pk.alloc_sparse_workspace(1, Hq, Hkv, D, B, T, 8)
    o = torch.empty_like(small.query)
    sel = torch.empty((1, Hkv, 8), dtype=torch.int32, device="cuda")
    pk.sparse_decode(o, small.query, kc, vc, bounds, blocks[None].cuda(), ctx, T, small.scale, 8, ws, selected=sel,
                     dev_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    small.check(o, sel, 8)
    assert torch.equal(small.vc.transpose(1, 2).reshape(-1, Hkv, D)[:T], v)


@pytest.mark.parametrize("dtype,e4m3", [("bf16", False), ("bf16", True)])
def test_copied_blocks(dtype, e4m3):
    """Blocks moved to other ids, then bounds from the first of them on: the context decodes as it did. A fork whose
    newest block is copied and appended to needs that block's bounds alone."""
    p = Pool([16 * 60 + 5], dtype=dtype, e4m3=e4m3, seed=23)
    L = p.lens[0]
    kc, vc = (torch.cat((c, torch.full_like(c[:10], 0x7F if e4m3 else float("nan")))) for c in (p.kc, p.vc))
    p.bounds = torch.cat((p.bounds, torch.full_like(p.bounds[:10], 100.0)))       # (of a block's earlier owner)
    p.kc, p.vc, p.num_blocks = kc, vc, p.num_blocks + 10
    p.fill_bounds()
    out, sel = p.decode(20)
    table = p.tables.clone()
    moved = list(range(30, 38))
    fresh = torch.arange(p.num_blocks - 10, p.num_blocks - 2)
    pairs = torch.stack((table[0, moved].cpu().long(), fresh), 1).cuda()
    pk.copy_blocks(p.kc, p.vc, pairs, dev_status=p.status)
    p.tables[0, moved] = fresh.int().cuda()
    back = torch.tensor([L - 30 * 16], dtype=torch.int32, device="cuda")
    pk.key_bounds(p.bounds, p.kc, p.tables, p.context, L, back, L, dev_status=p.status)
    again, same = p.decode(20)
    assert torch.equal(out, again) and torch.equal(sel, same) and int(p.status.item()) == 0
    # the fork: a copy of the newest block, one more token (in both caches the first token's rows)
    last = L // 16
    fork = p.num_blocks - 1
    pk.copy_blocks(p.kc, p.vc, torch.tensor([[int(p.tables[0, last]), fork]], device="cuda"), dev_status=p.status)
    p.tables[0, last] = fork
    for c in (p.kc, p.vc):
        c[fork, :, L % 16] = c[p.tables[0, 0].long(), :, 0]
    p.lens, p.max_len, p.context = [L + 1], L + 1, p.context + 1
    pk.key_bounds(p.bounds, p.kc, p.tables, p.context, L + 1, dev_status=p.status)
    out, sel = p.decode(20)
    assert int(p.status.item()) == 0
    p.check(out, sel, 20)


def test_steps_without_a_wait_equal_steps_with_one():
    """Append, bounds and sparse decode back to back on one stream: each kernel starts while the one before it runs,
    and reads what that one writes (query, caches, bounds). Bit for bit the results of the same calls one at a time."""
    S, Hq, Hkv, D, B, steps = 24, 32, 8, 128, 16, 40
    g = torch.Generator().manual_seed(31)
    lens = torch.randint(200, 900, (S,), generator=g)
    width = (900 + steps) // B + 1
    tables = (torch.randperm(S * width, generator=g) + 1).view(S, width).int().cuda()
    shape = (S * width + 1, Hkv, B, D)
    kc0, vc0 = (torch.randn(shape, generator=g).bfloat16().cuda() for _ in range(2))
    qkv = torch.randn((steps, S, Hq + 2 * Hkv, D), generator=g).bfloat16().cuda()
    angle = torch.rand((1024, D // 2), generator=g) * 6.28
    cos_sin = torch.cat((angle.cos(), angle.sin()), 1).cuda()
    at = [(lens + i) for i in range(steps)]
    slots = [(tables.cpu().gather(1, (a // B).view(-1, 1)).view(-1).long() * B + a % B).cuda() for a in at]
    positions, context = [a.cuda() for a in at], [(a + 1).int().cuda() for a in at]
    max_len = int(lens.max()) + steps
    results = []
    for wait in (True, False):
        kc, vc = kc0.clone(), vc0.clone()
        bounds = torch.full((shape[0], Hkv, 2, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        pk.key_bounds(bounds, kc, tables, lens.int().cuda(), max_len, lens.int().cuda(), max_len)
        q, outs = torch.empty((S, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.empty((steps, S, Hq, D), dtype=torch.bfloat16, device="cuda")
        ws = pk.alloc_sparse_workspace(S, Hq, Hkv, D, B, max_len, 12)
        torch.cuda.synchronize()
        for i in range(steps):
            x = qkv[i]
            pk.rope_and_cache(q, x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], kc, vc, cos_sin, positions[i], slots[i])
            if wait:
                torch.cuda.synchronize()
            pk.key_bounds(bounds, kc, tables, context[i], max_len)
            if wait:
                torch.cuda.synchronize()
            pk.sparse_decode(outs[i], q, kc, vc, bounds, tables, context[i], max_len, D ** -0.5, 12, ws)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        results.append((outs, kc, vc, bounds[tables.flatten().long()]))
    for a, b in zip(*results):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
