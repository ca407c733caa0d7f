"""rope_and_cache on the GPU against its formula in 64 bits.

Tolerances, derived: with u = 2^-24, the rotation of (a, b) by (c, s) in
binary32 rounds two products and a sum, at most 3 u (|a c| + |b s|); the norm
factor carries the sum of squares' rounding (at most 16 fused steps in a lane
and 4 exchanges of positive terms: 20 u on the sum, 10 u on its root), the
mean's (1 u), rsqrtf's 2 ulp (4 u) and the two products by it (2 u). 24 u
(|a c| + |b s|) covers both. The store rounds once: half a step of the output
type, relative, or half its smallest subnormal.
"""
import numpy as np
import pytest
import torch

from paged_kv_cache_141_gb300 import binding as pk

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_SUBNORMAL = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
SENTINEL = 7.5


def table(max_position, rotary, dev="cuda"):
    inv = 10000.0 ** (-torch.arange(0, rotary, 2, dtype=torch.float64) / rotary)
    angle = torch.arange(max_position, dtype=torch.float64)[:, None] * inv
    return torch.cat((angle.cos(), angle.sin()), 1).float().to(dev)


class Step:
    def __init__(self, T, Hq, Hkv, D, R=None, B=16, dtype="bf16", e4m3=False, axes=1, adjacent=False, norm=False,
                 seed=0, max_position=2048, fused=True):
        g = torch.Generator().manual_seed(seed)
        self.dims = (T, Hq, Hkv, D, R or D, B)
        R = R or D
        dt = TYPES[dtype]
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g).to(dt).cuda()
        parts = qkv.split((Hq, Hkv, Hkv), 1)
        self.q, self.k, self.v = parts if fused else [x.contiguous() for x in parts]
        self.num_blocks = T // B + 5
        slots = torch.randperm(self.num_blocks * B, generator=g)[:T]
        if T > 2:
            slots[T // 2] = -1
        self.slots = slots.cuda()
        self.positions = torch.randint(0, max_position, (axes, T), generator=g).cuda()
        self.axes = axes
        self.freq_axes = None
        if axes > 1:
            self.freq_axes = [int(x) for x in torch.randint(0, axes, (R // 2,), generator=g)]
        self.cos_sin = table(max_position, R)
        cdt = torch.uint8 if e4m3 else dt
        fill = 0x42 if e4m3 else SENTINEL
        shape = (self.num_blocks, Hkv, B, D)
        self.kc, self.vc = (torch.full(shape, fill, dtype=cdt, device="cuda") for _ in range(2))
        self.e4m3, self.adjacent, self.dt = e4m3, adjacent, dt
        self.qw = (1 + 0.3 * torch.randn(D, generator=g)).cuda() if norm else None
        self.kw = (1 + 0.3 * torch.randn(D, generator=g)).cuda() if norm else None
        self.eps, self.ks, self.vs = 1e-5, 0.017, 0.023
        self.out = torch.full((T, Hq, D), SENTINEL, dtype=dt, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        pos = self.positions[0].contiguous() if self.axes == 1 else self.positions
        args = dict(q_weight=self.qw, k_weight=self.kw, eps=self.eps, freq_axes=self.freq_axes,
                    adjacent_pairs=self.adjacent, k_scale=self.ks, v_scale=self.vs, dev_status=self.status)
        args.update(kw)
        pk.rope_and_cache(self.out, self.q, self.k, self.v, self.kc, self.vc, self.cos_sin, pos, self.slots, **args)
        torch.cuda.synchronize()
        return int(self.status.item())

    def rotated(self, x, w):
        """(y, bound on the binary32 error), in 64 bits, component by component."""
        T, _, _, D, R, _ = self.dims
        x = x.double()
        if w is not None:
            x = x / (x.square().sum(-1, keepdim=True) / D + self.eps).sqrt() * w.double()
        axis = torch.tensor(self.freq_axes or [0] * (R // 2), device="cuda")
        y, err = x.clone(), x.abs().clone()
        for i in range(R // 2):
            row = self.cos_sin[self.positions[axis[i]]].double()
            c, s = row[:, i, None], row[:, R // 2 + i, None]
            ia, ib = (2 * i, 2 * i + 1) if self.adjacent else (i, i + R // 2)
            a, b = x[..., ia], x[..., ib]
            y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
            err[..., ia], err[..., ib] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
        return y, 24 * 2.0 ** -24 * err

    def check(self, tokens=None):
        T, Hq, Hkv, D, R, B = self.dims
        live = torch.ones(T, dtype=torch.bool, device="cuda") if tokens is None else tokens
        y, err = self.rotated(self.q, self.qw)
        tol = torch.finfo(self.dt).eps / 2 * y.abs() + err + HALF_SUBNORMAL[self.dt]
        assert bool(((self.out.double() - y).abs() <= tol)[live].all()), "query"
        assert bool((self.out[~live] == SENTINEL).all()), "skipped tokens' queries keep their contents"
        kept = live & (self.slots >= 0) & (self.slots < self.num_blocks * B)
        at = self.slots[kept]
        y, err = self.rotated(self.k, self.kw)
        y, err = y[kept], err[kept]
        flat = [c.transpose(1, 2).reshape(-1, Hkv, D) for c in (self.kc, self.vc)]
        if self.e4m3:
            got = flat[0].view(torch.float8_e4m3fn).double()[at]
            want = (y / self.ks).clamp(-448, 448)
            # half a step of E4M3 (2^-4 relative, 2^-10 below the normal range)
            tol = 2.0 ** -4 * want.abs() + 2.0 ** -10 + 2 * err / self.ks
            assert bool(((got - want).abs() <= tol).all()), "E4M3 key"
            codes = (self.v.float()[kept] / self.vs).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            assert torch.equal(flat[1][at], codes), "E4M3 value"
        else:
            tol = torch.finfo(self.dt).eps / 2 * y.abs() + err + HALF_SUBNORMAL[self.dt]
            assert bool(((flat[0].double()[at] - y).abs() <= tol).all()), "key"
            assert torch.equal(flat[1][at], self.v[kept]), "value bits"
        rest = torch.ones(flat[0].shape[0], dtype=torch.bool, device="cuda")
        rest[at] = False
        fill = 0x42 if self.e4m3 else SENTINEL
        for f in flat:
            assert bool((f[rest] == fill).all()), "slots of no token keep their contents"


@pytest.mark.parametrize("T", [1, 2, 31, 257, 2000])
@pytest.mark.parametrize("Hq,Hkv", [(32, 8), (8, 8), (7, 1), (12, 2)])
def test_heads_and_tokens(T, Hq, Hkv):
    s = Step(T, Hq, Hkv, 128, seed=T)
    assert s.run() == 0
    s.check()


@pytest.mark.parametrize("T,Hq,Hkv", [(130, 64, 64), (305, 32, 8), (601, 32, 8), (1401, 32, 8), (3001, 16, 4),
                                      (9001, 7, 1)])
@pytest.mark.parametrize("D,dtype,e4m3", [(64, "bf16", False), (128, "f16", True), (256, "f32", False)])
def test_tokens_of_one_to_many_row_groups(T, Hq, Hkv, D, dtype, e4m3):
    s = Step(T, Hq, Hkv, D, dtype=dtype, e4m3=e4m3, norm=True, seed=T + D)
    assert s.run() == 0
    s.check()


@pytest.mark.parametrize("dtype,e4m3", [("f32", False), ("f16", False), ("bf16", False), ("f32", True), ("f16", True),
                                        ("bf16", True)])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 16), (128, 128), (128, 96), (256, 256), (256, 64)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_types_and_rotated_widths(dtype, e4m3, D, R, adjacent, norm):
    s = Step(37, 6, 2, D, R, dtype=dtype, e4m3=e4m3, adjacent=adjacent, norm=norm, seed=D + R)
    assert s.run() == 0
    s.check()


@pytest.mark.parametrize("axes", [1, 2, 3, 4])
@pytest.mark.parametrize("D,R,adjacent,dtype", [(128, 128, False, "bf16"), (128, 64, True, "f16"),
                                                (256, 224, False, "f32")])
def test_several_axes(axes, D, R, adjacent, dtype):
    s = Step(45, 8, 4, D, R, dtype=dtype, axes=axes, adjacent=adjacent, norm=True, seed=axes)
    assert s.run() == 0
    s.check()
    # consecutive sections, as rope_sections makes them
    if axes == 3:
        s = Step(45, 8, 4, D, R, dtype=dtype, axes=3, adjacent=adjacent, seed=9)
        s.freq_axes = list(pk.rope_sections((R // 8, 3 * R // 16, R // 2 - R // 8 - 3 * R // 16)))
        assert s.run() == 0
        s.check()


@pytest.mark.parametrize("B", [1, 5, 8, 32, 1024])
def test_block_sizes(B):
    s = Step(70, 4, 2, 64, B=B, norm=True)
    assert s.run() == 0
    s.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", [0.011, 1.0, 1 / 3, 3e-5, 1e-39, 2e38, 448.0])
def test_e4m3_values_are_the_quotients_codes(dtype, scale):
    """Every stored value has the code of the IEEE quotient: random ones, midpoints of two codes and
    their neighbours, quotients below the normal range, beyond the largest, and special values."""
    T, Hkv, D = 1500, 2, 64
    s = Step(T, 2, Hkv, D, dtype=dtype, e4m3=True, fused=False)
    g = torch.Generator().manual_seed(1)
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (codes[:-1] + codes[1:]) / 2
    v = torch.randn((T, Hkv, D), generator=g).double() * 40
    pick = torch.randint(0, 126, (T, Hkv, D), generator=g)
    near = mid[pick] * (1 + torch.randint(-3, 4, (T, Hkv, D), generator=g) * 2.0 ** -23)
    v = torch.where(torch.rand((T, Hkv, D), generator=g) < 0.5, near, v)
    v[:, 0, 0] = torch.where(torch.arange(T) % 2 == 0, 0.0, -0.0)
    v[:, 0, 1:6] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1e4, 2.0 ** -11])
    s.v = (v * scale).to(s.dt).cuda()
    s.slots = torch.arange(T, device="cuda")
    s.ks = s.vs = scale
    assert s.run() == 0
    want = (s.v.float() / torch.tensor(scale, dtype=torch.float32, device="cuda"))
    nan = want.isnan()
    want = want.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    got = s.vc.transpose(1, 2).reshape(-1, Hkv, D)[:T]
    assert torch.equal(got[~nan], want[~nan])
    assert bool(((got[nan] & 0x7F) == 0x7F).all())


def test_only_one_norm_and_large_prompt():
    s = Step(5000, 16, 4, 128, norm=True, dtype="f16")
    s.kw = None
    assert s.run() == 0
    s.check()
    s = Step(300, 16, 4, 128, norm=True)
    s.qw = None
    assert s.run() == 0
    s.check()


def test_in_place_query_and_equal_results_over_forms():
    a, b = (Step(333, 8, 2, 128, norm=True, seed=4, fused=f) for f in (True, False))
    assert a.run() == 0
    before = b.q
    b.out = b.q = before.clone()
    assert b.run() == 0
    assert torch.equal(a.out, b.out) and torch.equal(a.kc, b.kc) and torch.equal(a.vc, b.vc)


def test_one_axis_equals_equal_axes():
    a = Step(100, 8, 2, 128, axes=3, norm=True, seed=5)
    a.positions[1:] = a.positions[0]
    b = Step(100, 8, 2, 128, axes=3, norm=True, seed=5)
    b.positions, b.axes, b.freq_axes = a.positions[:1], 1, None
    assert a.run() == 0 and b.run() == 0
    assert torch.equal(a.out, b.out) and torch.equal(a.kc, b.kc)


def test_bad_positions_and_slots_set_bits_and_are_skipped():
    s = Step(64, 8, 2, 128, norm=True, axes=2)
    live = torch.ones(64, dtype=torch.bool, device="cuda")
    for t, axis, pos in ((3, 0, -1), (9, 1, 2048), (40, 0, 2 ** 40)):
        s.positions[axis, t] = pos
        live[t] = False
    assert s.run() == pk.DEV_BAD_POSITION
    clean = s.positions.clone()
    s.positions = torch.where(live, clean, 0)            # the check only looks at live tokens
    s.check(live)
    s = Step(64, 8, 2, 128)
    s.slots[5] = s.num_blocks * 16
    s.slots[6] = 2 ** 50
    assert s.run() == pk.DEV_BAD_SLOT
    s.check()


def test_zero_rows_infinities_and_nan_stay_in_their_rows():
    s = Step(8, 4, 2, 128, norm=True, dtype="f32")
    q = s.q.clone()
    q[1, 2] = 0
    q[2, 1, 5] = float("nan")
    q[3, 0, 7] = float("inf")
    s.q = q
    assert s.run() == 0
    assert bool((s.out[1, 2] == 0).all())
    bad = torch.zeros(8, 4, dtype=torch.bool, device="cuda")
    bad[2, 1] = bad[3, 0] = True
    assert bool(torch.isfinite(s.out[~bad]).all()) and bool(torch.isnan(s.out[2, 1]).all())


def test_graph_replay_on_another_stream():
    s = Step(50, 8, 2, 128, norm=True, seed=2)
    side = torch.cuda.Stream()
    assert s.run() == 0
    want = s.out.clone(), s.kc.clone()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pk.rope_and_cache(s.out, s.q, s.k, s.v, s.kc, s.vc, s.cos_sin, s.positions[0].contiguous(), s.slots,
                              s.qw, s.kw, s.eps, dev_status=s.status)
    s.out.zero_()
    s.kc.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.out, want[0])
    at = s.slots[s.slots >= 0]
    flat = lambda c: c.transpose(1, 2).reshape(-1, 2, 128)[at]      # noqa: E731
    assert torch.equal(flat(s.kc), flat(want[1]))


def test_empty_call_and_wrong_arguments():
    s = Step(4, 4, 2, 64)
    none = s.q[:0]
    pk.rope_and_cache(s.out[:0], none, s.k[:0], s.v[:0], s.kc, s.vc, s.cos_sin, s.positions[0, :0], s.slots[:0])
    with pytest.raises(ValueError):
        s.run(q_weight=torch.ones(64, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        pk.rope_and_cache(s.out, s.q.transpose(0, 1), s.k, s.v, s.kc, s.vc, s.cos_sin, s.positions[0], s.slots)
    with pytest.raises(ValueError):                                  # several axes without freq_axes
        pk.rope_and_cache(s.out, s.q, s.k, s.v, s.kc, s.vc, s.cos_sin, s.positions.expand(2, 4).contiguous(), s.slots)
    with pytest.raises(pk.PagedKVError):                             # rotary_dim 40: not a multiple of 16
        pk.rope_and_cache(s.out, s.q, s.k, s.v, s.kc, s.vc, table(8, 40), s.positions[0].contiguous(), s.slots)
    torch.cuda.synchronize()
