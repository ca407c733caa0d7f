"""Draft verification against its definition in 64 bits."""
import pytest
import torch

import step_common as sc

pytestmark = pytest.mark.gpu


def pk():
    from paged_kv_cache_141_gb300 import binding
    return binding


def inputs(S, K, V, seed, sampled=True, sharp=2.0, noise=0.7, rows=None):
    g = torch.Generator().manual_seed(seed)
    rows = [K + 1] * S if rows is None else rows
    starts = [0]
    for n in rows:
        starts.append(starts[-1] + n)
    T = starts[-1]
    logits = torch.randn(max(T, 1), V, generator=g) * sharp
    target = torch.softmax(logits, -1)
    draft = torch.zeros(S, K, V)
    for s in range(S):
        for i in range(min(K, max(rows[s] - 1, 0))):
            draft[s, i] = torch.softmax(logits[starts[s] + i] + noise * torch.randn(V, generator=g), -1)
    drafted = torch.full((S, K), -5, dtype=torch.int64)
    for s in range(S):
        for i in range(min(K, max(rows[s] - 1, 0))):
            drafted[s, i] = int(torch.multinomial(draft[s, i], 1, generator=g))
    uniforms = torch.rand(S, K + 1, generator=g)
    return target[:T], draft if sampled else None, drafted, uniforms, starts


def check(target, draft, drafted, uniforms, starts, spread=0):
    S, K = drafted.shape
    V = target.shape[1]
    wide = lambda x: torch.nn.functional.pad(x, (0, spread)).cuda()[..., :V]  # noqa: E731
    out = torch.full((S, K + 1), 77, dtype=torch.int64, device="cuda")
    acc, rej = (torch.full((S,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pk().verify_drafts(out, acc, wide(target), drafted.cuda(), uniforms.cuda(), torch.tensor(starts, dtype=torch.int32, device="cuda"),
                       draft_probs=None if draft is None else wide(draft), rejected=rej, dev_status=status)
    want, accepted, near = sc.verify(target, draft, drafted, uniforms, starts)
    # sums kept to 2^-44 put a border, and the goal, at most 2^-43 of the whole away
    assert min(near, default=1.0) > 2.0 ** -43, "inputs next to a border"
    assert acc.tolist() == accepted.tolist()
    assert out.tolist() == want.tolist()
    drafts = [max(b - a - 1, 0) for a, b in zip(starts, starts[1:])]
    assert rej.tolist() == [n - a for n, a in zip(drafts, accepted.tolist())]
    assert int(status) == 0
    return accepted


@pytest.mark.parametrize("S,K,V", [(1, 0, 1), (1, 1, 2), (3, 4, 31), (2, 5, 512), (5, 3, 513), (1, 4, 8191), (2, 4, 32000), (1, 2, 128256),
                                   (40, 3, 3001), (320, 2, 700), (2, 40, 300)])
@pytest.mark.parametrize("sampled", [True, False])
def test_verify(S, K, V, sampled):
    check(*inputs(S, K, V, S * 1000 + K * 10 + V, sampled), spread=(S + K) % 3)


def test_every_outcome_occurs():
    accepted = check(*inputs(64, 4, 600, 5))
    assert set(accepted.tolist()) == {0, 1, 2, 3, 4}


def test_ragged_requests():
    check(*inputs(6, 4, 1000, 3, rows=[5, 1, 0, 3, 0, 2]))
    check(*inputs(3, 4, 1000, 3, False, rows=[0, 5, 4]))


def test_identical_distributions_accept_all():
    target, draft, drafted, uniforms, starts = inputs(8, 4, 500, 9, noise=0.0)
    for s in range(8):
        draft[s] = target[starts[s]:starts[s] + 4]
    assert check(target, draft, drafted, uniforms, starts).tolist() == [4] * 8


@pytest.mark.parametrize("V", [5, 700, 20000])
def test_nothing_beyond_the_drafter(V):
    # a drafter above the target everywhere: rejected, and drawn from the target itself
    target, draft, drafted, uniforms, starts = inputs(4, 1, V, 2)
    for s in range(4):
        draft[s, 0] = target[starts[s]] * 4 + 1e-3
    uniforms[:, 0] = 0.9
    assert check(target, draft, drafted, uniforms, starts).tolist() == [0] * 4


@pytest.mark.parametrize("V", [3, 600, 40000])
def test_draw_at_the_ends(V):
    target, draft, drafted, uniforms, starts = inputs(2, 0, V, 4)
    target[0, :V // 2] = 0.0
    target[1, V // 2 + 1:] = 0.0
    out = torch.empty(2, 1, dtype=torch.int64, device="cuda")
    acc = torch.empty(2, dtype=torch.int32, device="cuda")
    for u, want in ((0.0, [V // 2, 0]), (1 - 2.0 ** -24, [None, V // 2])):
        pk().verify_drafts(out, acc, target.cuda(), drafted.cuda(), torch.full((2, 1), u).cuda(),
                           torch.tensor(starts, dtype=torch.int32, device="cuda"))
        got = out.view(-1).tolist()
        assert all(w is None or g == w for g, w in zip(got, want)), (u, got)
        assert all(float(target[s, t]) > 0 for s, t in enumerate(got))


def test_frequencies():
    """The drawn tokens follow the target: 4096 requests with one draft each, 12 tokens."""
    g = torch.Generator().manual_seed(8)
    p = torch.softmax(torch.randn(12, generator=g), 0)
    q = torch.softmax(torch.randn(12, generator=g), 0)
    S = 4096
    drafted = torch.multinomial(q, S, replacement=True, generator=g).view(S, 1)
    out = torch.empty(S, 2, dtype=torch.int64, device="cuda")
    acc = torch.empty(S, dtype=torch.int32, device="cuda")
    pk().verify_drafts(out, acc, p.repeat(2 * S, 1).cuda(), drafted.cuda(), torch.rand(S, 2, generator=g).cuda(),
                       torch.arange(0, 2 * S + 1, 2, dtype=torch.int32, device="cuda"), draft_probs=q.repeat(S, 1, 1).cuda())
    first = torch.bincount(out[:, 0].cpu(), minlength=12).double() / S
    # five standard deviations of a frequency
    assert bool(((first - p.double()).abs() <= 5 * (p.double() * (1 - p.double()) / S).sqrt()).all())


def test_bad_data():
    target, draft, drafted, uniforms, starts = inputs(4, 2, 100, 6)
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(target=target, drafted=drafted, starts=starts):
        out = torch.full((4, 3), 77, dtype=torch.int64, device="cuda")
        acc, status = t([77] * 4), t([0])
        pk().verify_drafts(out, acc, target.cuda(), drafted.cuda(), uniforms.cuda(), t(starts), draft_probs=draft.cuda(), dev_status=status)
        return out.tolist(), acc.tolist(), int(status)

    fine = call()
    assert fine[2] == 0
    far = drafted.clone()
    far[1, 0], far[2, 1] = 100, -1
    out, acc, status = call(drafted=far)
    assert status == pk().DEV_BAD_TOKEN and acc[1] == 0 and acc[2] <= 1 and out[0] == fine[0][0] and out[3] == fine[0][3]
    assert 0 <= out[1][0] < 100
    out, acc, status = call(starts=[0, 3, 6, 9, 13])                         # more rows than drafts and one
    assert status == pk().DEV_BAD_LEN and out[3] == [-1] * 3 and acc[3] == 0 and out[:3] == fine[0][:3]
    out, acc, status = call(starts=[0, 3, 2, 9, 12])
    assert status == pk().DEV_BAD_LEN and out[1] == [-1] * 3 and out[0] == fine[0][0] and out[3] == fine[0][3]
    odd = target.clone()
    odd[0:3, 50] = float("nan")
    odd[3:6] = 0.0
    out, acc, status = call(target=odd)
    assert status == pk().DEV_BAD_PROB and out[1] == [-1] * 3 and out[0][acc[0]] == -1 and out[2:] == fine[0][2:]


@pytest.mark.parametrize("token", [2 ** 32 + 5, 2 ** 63 - 1, 100, -1, -2 ** 63])
def test_a_token_outside_the_vocabulary_takes_nothing_away(token):
    target = torch.zeros(2, 100, device="cuda")
    target[:, 5:7] = 0.5
    out = torch.empty(1, 2, dtype=torch.int64, device="cuda")
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    acc, status = t([77]), t([0])
    pk().verify_drafts(out, acc, target, torch.tensor([[token]], device="cuda"), torch.tensor([[0.5, 0.25]], device="cuda"), t([0, 2]),
                       dev_status=status)
    assert out.tolist() == [[5, -1]] and acc.tolist() == [0] and int(status) == pk().DEV_BAD_TOKEN
