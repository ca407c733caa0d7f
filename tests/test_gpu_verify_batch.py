"""Draft verification: batches whose requests take a cluster of small CTAs, goals on and
next to a border between two tokens, sums over many tiles, steps without drafts."""
from fractions import Fraction

import pytest
import torch

import step_common as sc
from test_gpu_verify import check, inputs, pk

pytestmark = pytest.mark.gpu


# More than 76 requests: CTAs of 128 threads; by tiles of 512 tokens clusters of 2, 4 and 8 of them, one of
# which holds no tile at 9 tiles, and single CTAs.
@pytest.mark.parametrize("S,K,V", [(80, 2, 9000), (100, 3, 5001), (77, 1, 4500), (90, 1, 2600), (310, 1, 9000), (620, 1, 3000), (81, 0, 32000)])
@pytest.mark.parametrize("sampled", [True, False])
def test_batches(S, K, V, sampled):
    check(*inputs(S, K, V, S + K + V, sampled), spread=(S + K) % 3)


@pytest.mark.parametrize("sampled", [True, False])
def test_ragged_batches(sampled):
    check(*inputs(96, 3, 5001, 7, sampled, rows=[(0, 4, 1, 3, 2, 4)[s % 6] for s in range(96)]))


@pytest.mark.parametrize("V", [5001, 9000])
def test_nothing_beyond_the_drafter_in_a_batch(V):
    target, draft, drafted, uniforms, starts = inputs(90, 1, V, 2)
    for s in range(0, 90, 2):                                # every other request: from the target itself
        draft[s, 0] = target[starts[s]] * 4 + 1e-3
        uniforms[s, 0] = 0.9
    assert check(target, draft, drafted, uniforms, starts)[::2].tolist() == [0] * 45


def test_a_token_outside_the_vocabulary_in_a_batch():
    target, draft, drafted, uniforms, starts = inputs(90, 1, 5001, 4, False)
    drafted[7], drafted[50] = 5001, -1
    out = torch.empty(90, 2, dtype=torch.int64, device="cuda")
    acc, status = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (90, 1))
    pk().verify_drafts(out, acc, target.cuda(), drafted.cuda(), uniforms.cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"),
                       dev_status=status)
    assert int(status) == pk().DEV_BAD_TOKEN
    for s in (7, 50):                                        # rejected; nothing taken from the draw
        sums = target[starts[s]].double().cumsum(0)
        want = int((sums <= float(uniforms[s, 1]) * float(sums[-1])).sum())
        assert acc[s] == 0 and out[s].tolist() == [want, -1]


def whole_rows(S, V, seed):
    """Rows of whole numbers below 2^24 whose sum is 2^24 exactly, some of them 0."""
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(0, 2 * (2 ** 24 // V), (S, V), generator=g)
    w[torch.rand(S, V, generator=g) < 0.3] = 0
    w[:, V // 2] = 0
    w[:, V // 3] = 0
    w[:, V // 3] = 2 ** 24 - w.sum(1)
    assert bool((w >= 0).all()) and bool((w < 2 ** 24).all())
    return w


@pytest.mark.parametrize("S,V", [(3, 600), (2, 9000), (100, 9000), (80, 3000), (620, 700)])
@pytest.mark.parametrize("drafts", [False, True])
def test_goals_on_a_border(S, V, drafts):
    # every sum is exact, and so is u W: on a border the token behind it, 2^-24 below one the token before it
    g = torch.Generator().manual_seed(V)
    w = whole_rows(S, V, S + V)
    sums = w.cumsum(1)
    at = torch.randint(0, V - 1, (S,), generator=g)
    for below in (0, 1):
        goal = (sums.gather(1, at.view(-1, 1)).view(-1) - below).clamp(min=0)
        goal = torch.where(goal == 2 ** 24, goal - 1, goal)
        want = (sums <= goal.view(-1, 1)).sum(1)
        u = (goal.double() * 2.0 ** -24).float()
        assert bool((u.double() * 2.0 ** 24 == goal).all())
        t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        K = int(drafts)
        out = torch.empty(S, K + 1, dtype=torch.int64, device="cuda")
        acc = torch.empty(S, dtype=torch.int32, device="cuda")
        if drafts:
            # the weights are what lies beyond the drafter; u q(x) = p(x) for its token, which is not below
            q = torch.randint(0, 4, (S, V), generator=g)
            p = w + q
            p[:, V // 2], q[:, V // 2] = 2 ** 20, 2 ** 21
            rows = (p.float() * 2.0 ** -25).repeat_interleave(2, 0)
            assert bool((rows[::2].double() * 2.0 ** 25 == p).all())
            call = lambda first: pk().verify_drafts(  # noqa: E731
                out, acc, rows.cuda(), torch.full((S, 1), V // 2).cuda(), torch.stack([torch.full((S,), first), u], 1).cuda(),
                t(list(range(0, 2 * S + 1, 2))), draft_probs=(q.float() * 2.0 ** -25).view(S, 1, V).cuda())
            call(0.5 - 2.0 ** -25)
            assert acc.tolist() == [1] * S and out[:, 0].tolist() == [V // 2] * S
            call(0.5)
            assert acc.tolist() == [0] * S and out[:, 1].tolist() == [-1] * S
        else:
            pk().verify_drafts(out, acc, w.float().cuda(), torch.empty(S, 0, dtype=torch.int64).cuda(), u.view(S, 1).cuda(), t(list(range(S + 1))))
        assert out[:, 0].tolist() == want.tolist()


# Sixteen values of a lane whose sums, added tile after tile, lose what lies below the smaller half of a pair.
VALUES = ["0x1.2bb564p-44", "0x1.6be390p-28", "0x1.2a0f90p-34", "0x1.6fd12cp-29", "0x1.46e854p-24", "0x1.bafc86p-29", "0x1.437942p-31",
          "0x1.a3c100p-35", "0x1.e40da8p-33", "0x1.ff7f82p-43", "0x1.c368a2p-36", "0x1.420610p-33", "0x1.171858p-46", "0x1.812970p-35",
          "0x1.e9b1c0p-36", "0x1.85fcc4p-33"]


@pytest.mark.parametrize("S,V", [(1, 2 ** 22), (609, 2 ** 18)])
def test_sums_over_many_tiles(S, V):
    """Every tile the same, 128 of them a warp, four a lane; u = 1/16, and so much more in the last value that
    the goal lies 2^-39.9 of itself above the border behind a sixteenth of the tiles. The goal is kept to
    (99 + 3 4 + 3 8) 2^-48 of itself (a tile's tree; four tiles; the trees over lanes and warps), the border
    to 99 2^-48: 2^-40.1 in all."""
    values = [float.fromhex(x) for x in VALUES]
    tile, tiles = sum(Fraction(x) for x in values) * 32, V // 512
    last = torch.tensor(values[-1] + 1.0e-12 * float(tile * tiles), dtype=torch.float32).item()
    total = tile * tiles + Fraction(last) - Fraction(values[-1])
    above = total / 16 - tile * tiles / 16
    assert 2.0 ** -40 < above / (total / 16) < 2.0 ** -39.8 and above < Fraction(values[0])
    row = torch.tensor(values, dtype=torch.float32).repeat_interleave(32).repeat(tiles)
    row[-1] = last
    out = torch.empty(S, 1, dtype=torch.int64, device="cuda")
    acc = torch.empty(S, dtype=torch.int32, device="cuda")
    pk().verify_drafts(out, acc, row.cuda().repeat(S, 1), torch.empty(S, 0, dtype=torch.int64, device="cuda"),
                       torch.full((S, 1), 1 / 16, device="cuda"), torch.arange(S + 1, dtype=torch.int32, device="cuda"))
    assert out.view(-1).tolist() == [V // 16] * S


@pytest.mark.parametrize("S", [620, 609])
def test_larger_vocabularies_one_after_another(S):
    # a CTA a request: 8 bytes of shared memory for each 512 tokens, first some 49 KB, then 64 KB
    for V in (3200000, 2 ** 22):
        target = torch.zeros(1, V, device="cuda")
        target[0, V - 3] = 0.25
        out = torch.empty(S, 1, dtype=torch.int64, device="cuda")
        acc = torch.empty(S, dtype=torch.int32, device="cuda")
        starts = torch.ones(S + 1, dtype=torch.int32, device="cuda")           # the first request alone has a row
        starts[0] = 0
        pk().verify_drafts(out, acc, target, torch.empty(S, 0, dtype=torch.int64, device="cuda"), torch.full((S, 1), 0.5, device="cuda"), starts)
        assert out.view(-1).tolist() == [V - 3] + [-1] * (S - 1)


@pytest.mark.parametrize("S", [1, 5, 90])
def test_steps_without_drafts(S):
    # draft_probs as a program keeps them, of no drafts: [S, 0, V]
    target, _, drafted, uniforms, starts = inputs(S, 0, 700, S)
    out = torch.empty(S, 1, dtype=torch.int64, device="cuda")
    acc = torch.empty(S, dtype=torch.int32, device="cuda")
    pk().verify_drafts(out, acc, target.cuda(), drafted.cuda(), uniforms.cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"),
                       draft_probs=torch.empty(S, 0, 700, device="cuda"))
    want, accepted, _ = sc.verify(target, None, drafted, uniforms, starts)
    assert out.tolist() == want.tolist() and acc.tolist() == accepted.tolist()
    # and views that are not evenly spaced are still refused
    with pytest.raises(ValueError):
        pk().verify_drafts(torch.empty(2, 3, dtype=torch.int64, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda"),
                           torch.ones(6, 8, device="cuda"), torch.zeros(2, 2, dtype=torch.int64, device="cuda"),
                           torch.zeros(2, 3, device="cuda"), torch.tensor([0, 3, 6], dtype=torch.int32, device="cuda"),
                           draft_probs=torch.ones(2, 3, 8, device="cuda")[:, :2])
