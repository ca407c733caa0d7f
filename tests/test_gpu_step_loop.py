"""Speculative steps over a block-scaled cache that never wait for the host, eager
and as a CUDA graph, against the same steps on the host: room for every request's
tokens, their append, the attention to them, the verification of the drafts, and
the rejected ones given back."""
import random

import pytest
import torch

import step_common as sc

pytestmark = pytest.mark.gpu

S, K, H, HQ, D, B, V, MOST, POOL = 6, 3, 2, 8, 64, 16, 257, 12, 60


def pk():
    from paged_kv_cache_141_gb300 import binding
    return binding


class Device:
    """The state that a serving program keeps, and one step on it."""

    def __init__(self, kind, seed):
        g = torch.Generator().manual_seed(seed)
        z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d, device="cuda")  # noqa: E731
        self.stack = (torch.randperm(POOL, generator=g) + 1).to(torch.int32).cuda()
        self.free = torch.tensor([POOL], dtype=torch.int32, device="cuda")
        self.table, self.lens = z(S, MOST) - 1, z(S)
        self.kc, self.vc = (torch.full((POOL + 1, H, B, D), 77, dtype=torch.uint8, device="cuda").view(sc.CODES[kind]) for _ in range(2))
        self.ks, self.vs = (torch.full((POOL + 1, H), 1e4, device="cuda") for _ in range(2))
        T = S * (K + 1)
        self.new, self.drop = z(S), z(S)
        self.slots, self.pos, self.start = z(T, d=torch.int64), z(T, d=torch.int64), z(S + 1)
        self.k, self.v = (z(T, H, D, d=torch.bfloat16) for _ in range(2))
        self.q, self.out = (z(T, HQ, D, d=torch.bfloat16) for _ in range(2))
        self.target, self.draft = z(T, V, d=torch.float32), z(S, K, V, d=torch.float32)
        self.drafted, self.u = z(S, K, d=torch.int64), z(S, K + 1, d=torch.float32)
        self.tokens, self.accepted, self.rejected = z(S, K + 1, d=torch.int64), z(S), z(S)
        self.status = z(1)
        self.ws = pk().alloc_scaled_workspace(S, T, HQ, H, D, K + 1, MOST * B)

    def step(self):
        p = pk()
        p.extend_tables(self.table, self.lens, self.new, self.stack, self.free, self.slots, self.start, B, positions=self.pos,
                        dev_status=self.status)
        p.scaled_append(self.k, self.v, self.kc, self.vc, self.ks, self.vs, self.table, self.lens, K + 1, self.start,
                        dev_status=self.status)
        p.scaled_attention(self.out, self.q, self.kc, self.vc, self.ks, self.vs, self.table, self.lens, MOST * B, D ** -0.5, self.ws,
                           query_start=self.start, max_queries_per_seq=K + 1, dev_status=self.status)
        p.verify_drafts(self.tokens, self.accepted, self.target, self.drafted, self.u, self.start, draft_probs=self.draft,
                        rejected=self.rejected, dev_status=self.status)
        p.trim_tables(self.table, self.lens, self.rejected, self.stack, self.free, B, dev_status=self.status)

    def end(self, which):
        """Requests that are done give back everything."""
        drop = torch.zeros_like(self.drop)
        drop[which] = self.lens[which]
        pk().trim_tables(self.table, self.lens, drop, self.stack, self.free, B, dev_status=self.status)


class Host:
    def __init__(self, dev):
        self.stack, self.free = dev.stack.tolist(), POOL
        self.table, self.lens = dev.table.cpu(), [0] * S
        self.caches = [x.cpu() for x in (dev.kc, dev.vc)]
        self.scales = [x.cpu() for x in (dev.ks, dev.vs)]

    def drop(self, counts):
        back = []
        for s, d in enumerate(counts):
            L = self.lens[s]
            back += self.table[s, -(-(L - d) // B):-(-L // B)].tolist()
            self.lens[s] = L - d
        self.stack[self.free:self.free + len(back)] = back[::-1]
        self.free += len(back)

    def step(self, dev, x, kind):
        T = S * (K + 1)
        self.table, slots, pos, start, self.lens, self.free, denied = sc.extend(self.table, self.lens, x["new"].tolist(), self.stack, self.free, B, T)
        assert not denied
        assert dev.slots.tolist() == slots and dev.pos.tolist() == pos and dev.start.tolist() == start
        sc.append(x["k"], x["v"], self.caches, self.scales, self.table, self.lens, start, kind)
        n = start[-1]
        want, tol = sc.attention(x["q"], *self.caches, *self.scales, self.table, self.lens, start, D ** -0.5, torch.bfloat16)
        sc.assert_close(dev.out, want, tol)
        tokens, accepted, near = sc.verify(x["target"], x["draft"], x["drafted"], x["u"], start)
        assert min(near) > 2.0 ** -43
        assert dev.tokens.cpu().equal(tokens) and dev.accepted.cpu().equal(accepted)
        counts = [max(start[s + 1] - start[s] - 1, 0) - int(accepted[s]) for s in range(S)]
        assert dev.rejected.tolist() == counts
        self.drop(counts)
        return n

    def check(self, dev):
        assert dev.lens.tolist() == self.lens and int(dev.free) == self.free and dev.stack.tolist()[:self.free] == self.stack[:self.free]
        for s, L in enumerate(self.lens):
            n = -(-L // B)
            assert dev.table[s, :n].tolist() == self.table[s, :n].tolist()
            for b in self.table[s, :n].tolist():
                for got, want in zip((dev.ks, dev.vs), self.scales):
                    assert got[b].cpu().equal(want[b])
                for got, want in zip((dev.kc, dev.vc), self.caches):
                    assert got.view(torch.uint8)[b].cpu().equal(want.view(torch.uint8)[b])
        assert int(dev.status) == 0


def inputs(seed, active):
    """A step's inputs: every active request has one to K drafts; a request that starts brings K + 1 tokens."""
    g, r = torch.Generator().manual_seed(seed), random.Random(seed)
    T = S * (K + 1)
    new = torch.tensor([r.randint(1, K + 1) if a else 0 for a in active], dtype=torch.int32)
    size = torch.exp(0.7 * torch.randn(T, 1, 1, generator=g))
    x = {"new": new, "q": torch.randn(T, HQ, D, generator=g).bfloat16()}
    x["k"], x["v"] = ((torch.randn(T, H, D, generator=g) * size).bfloat16() for _ in range(2))
    logits = 2 * torch.randn(T, V, generator=g)
    x["target"] = torch.softmax(logits, -1)
    x["draft"] = torch.softmax(2 * torch.randn(S, K, V, generator=g), -1)
    at = 0
    for s in range(S):                                       # the drafter is near the target
        for i in range(int(new[s]) - 1):
            x["draft"][s, i] = torch.softmax(logits[at + i] + 0.6 * torch.randn(V, generator=g), -1)
        at += int(new[s])
    x["drafted"] = torch.multinomial(x["draft"].view(S * K, V), 1, generator=g).view(S, K)
    x["u"] = torch.rand(S, K + 1, generator=g)
    return x


def load(dev, x):
    for name, value in x.items():
        getattr(dev, name).copy_(value)


@pytest.mark.parametrize("kind", ["int8", "e4m3"])
@pytest.mark.parametrize("graph", [False, True])
def test_steps(kind, graph):
    dev = Device(kind, 5)
    host = Host(dev)
    r = random.Random(11)
    active = [True] * S
    stream = torch.cuda.Stream()                              # not the default one
    with torch.cuda.stream(stream):
        run = dev.step
        if graph:
            load(dev, inputs(999, [False] * S))               # a step of no request changes nothing
            dev.step()
            stream.synchronize()
            assert int(dev.free) == POOL and dev.lens.tolist() == [0] * S
            cap = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cap, stream=stream):
                dev.step()
            run = cap.replay
        for t in range(30):
            x = inputs(100 + t, active)
            load(dev, x)
            run()
            stream.synchronize()
            host.step(dev, x, kind)
            host.check(dev)
            # now and then a request ends, and another takes its row a step later
            done = [s for s in range(S) if active[s] and (host.lens[s] > 80 or r.random() < 0.05)]
            if done:
                dev.end(done)
                host.drop([host.lens[s] if s in done else 0 for s in range(S)])
                stream.synchronize()
                host.check(dev)
            active = [s not in done for s in range(S)]
    assert max(host.lens) > 40


def test_two_streams_of_steps():
    """Two servers at once, each with a pool and a workspace of its own, give what each gives alone."""
    servers = [(Device("int8", 3 + i), torch.cuda.Stream()) for i in range(2)]
    alone = [Device("int8", 3 + i) for i in range(2)]
    steps = [[inputs(50 * i + t, [True] * S) for t in range(6)] for i in range(2)]
    torch.cuda.synchronize()
    for i, dev in enumerate(alone):
        for x in steps[i]:
            load(dev, x)
            dev.step()
            torch.cuda.synchronize()
    for t in range(6):
        for i, (dev, stream) in enumerate(servers):
            with torch.cuda.stream(stream):
                load(dev, steps[i][t])
                dev.step()
    torch.cuda.synchronize()
    for (dev, _), other in zip(servers, alone):
        for name in ("table", "lens", "free", "kc", "ks", "vs", "tokens", "accepted", "status"):
            a, b = getattr(dev, name), getattr(other, name)
            assert (a.view(torch.uint8) if a.element_size() == 1 else a).equal(b.view(torch.uint8) if b.element_size() == 1 else b), name
        n = int(dev.start[-1])
        assert dev.out[:n].equal(other.out[:n])


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("queries", [1, 5, 40])
def test_repeated_and_replayed_calls_are_bit_identical(queries, D):
    lens = [700, 64, 2500]
    table, nb = sc.table_of(3, 160, 1)
    (kc, ks), (vc, vs) = (sc.pool(nb, 2, 16, D, "e4m3", i) for i in range(2))
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = [x.cuda() for x in (kc, vc, ks, vs)] + [table.cuda(), t(lens)]
    q = torch.randn(3 * queries, 8, D, device="cuda").bfloat16()
    qs = t([0, queries, 2 * queries, 3 * queries])
    ws = pk().alloc_scaled_workspace(3, 3 * queries, 8, 2, D, queries, 2560)
    outs = [torch.empty_like(q) for _ in range(2)]
    call = lambda out: pk().scaled_attention(out, q, *args, 2560, 0.09, ws, query_start=qs, max_queries_per_seq=queries)  # noqa: E731
    call(outs[0])
    call(outs[1])
    g = torch.cuda.CUDAGraph()
    stream = torch.cuda.Stream()
    replayed = torch.empty_like(q)
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        call(replayed)
    ws.fill_(0xFF)
    g.replay()
    torch.cuda.synchronize()
    assert outs[0].equal(outs[1]) and outs[0].equal(replayed)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_replays_follow_lengths_that_change(D):
    # many rows: which context is the longest, who has how many tokens and who none, change between replays
    table, nb = sc.table_of(4, 100, 3)
    (kc, ks), (vc, vs) = (sc.pool(nb, 1, 16, D, "int8", i) for i in range(2))
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    lens, starts, status = t([50] * 4), t([0, 9, 18, 27, 36]), t([0])
    query = torch.randn(36, 8, D).half()
    out = torch.empty_like(query).cuda()
    ws = pk().alloc_scaled_workspace(4, 36, 8, 1, D, 20, 1600)
    args = [query.cuda(), *(x.cuda() for x in (kc, vc, ks, vs, table)), lens, 1600, D ** -0.5, ws]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        pk().scaled_attention(out, *args, query_start=starts, max_queries_per_seq=20, dev_status=status)
    for L, n in (([1600, 9, 300, 77], [9, 9, 9, 9]), ([20, 1600, 0, 1100], [16, 20, 0, 0]), ([5, 6, 1599, 1], [5, 6, 20, 1])):
        at = [0]
        for k in n:
            at.append(at[-1] + k)
        lens.copy_(t(L))
        starts.copy_(t(at))
        out.fill_(7.0)
        g.replay()
        want, tol = sc.attention(query, kc, vc, ks, vs, table, L, at, D ** -0.5, query.dtype)
        sc.assert_close(out, want, tol)
        assert int(status) == 0 and bool((out[at[-1]:] == 7.0).all())


def test_copied_blocks_keep_their_codes():
    """Copy-on-write of a scaled cache: copy_blocks moves the codes, indexing the scales."""
    (kc, ks), (vc, vs) = (sc.pool(6, 2, 16, 64, "int8", i) for i in range(2))
    dev = [x.cuda() for x in (kc, vc, ks, vs)]
    pk().copy_blocks(dev[0], dev[1], torch.tensor([[1, 4], [2, 5]], device="cuda"))
    for scales in dev[2:]:
        scales[[4, 5]] = scales[[1, 2]]
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    out = torch.empty_like(q)
    table = torch.tensor([[1, 2], [4, 5]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([20, 20], dtype=torch.int32, device="cuda")
    q[1] = q[0]
    ws = pk().alloc_scaled_workspace(2, 2, 4, 2, 64, 1, 32)
    pk().scaled_attention(out, q, *dev, table, lens, 32, 0.125, ws)
    assert out[0].equal(out[1])
