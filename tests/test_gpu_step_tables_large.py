"""Block tables and slot maps on the device: as many requests as a call takes, and slots
that a kernel of their own fills."""
import random

import pytest
import torch

from test_gpu_step_tables import State, pk, run_extend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S", [8191, 16383, 16384])
def test_extend_of_many_requests(S):
    r = random.Random(S)
    lens = [r.choice((0, 1, 7, 8, r.randint(0, 30))) for _ in range(S)]
    new = [r.choice((0, 1, 1, 5, r.randint(0, 9))) for _ in range(S)]
    assert run_extend(State(lens, 5, 8, sum(new) + 3, S), new, in_place=S % 2 == 0) == ([], 0)
    # all blocks of one request, and none of the others
    some = [0] * S
    some[S // 2] = 30
    assert run_extend(State(lens, 8, 8, 9, S), some) == ([], 0)


@pytest.mark.parametrize("spare", [0, 700, 3001])
def test_many_slots_and_too_few_blocks(spare):
    # more than 16,384 places: those who need a block that is not there get none, the others their slots (of 3001 all)
    r = random.Random(spare)
    lens = [r.randint(0, 300) for _ in range(200)]
    new = [r.choice((0, 1, 3, r.randint(0, 400))) for _ in range(200)]
    denied, status = run_extend(State(lens, 90, 8, spare, 3), new, room=30000)
    assert bool(denied) == (spare < 3001) and status == (pk().DEV_NO_BLOCKS if denied else 0)


def test_many_slots_and_too_few_places():
    denied, status = run_extend(State([3] * 300, 16, 16, 5000), [100] * 300, room=20050)
    assert denied == list(range(200, 300)) and status == pk().DEV_BAD_LEN


@pytest.mark.parametrize("S", [0, 3])
def test_many_slots_of_no_request(S):
    st = State([5] * S, 4, 16, 20)
    assert run_extend(st, [0] * S, room=20000) == ([], 0)


@pytest.mark.parametrize("S", [2500, 16384])
@pytest.mark.parametrize("shared", [False, True])
def test_trim_of_many_requests(S, shared):
    r = random.Random(S)
    lens = [r.randint(0, 40) for _ in range(S)]
    drop = [r.choice((0, L, min(L, 3), r.randint(0, L))) for L in lens]
    out = [r.choice((0, 1, 3)) for _ in range(S)] if shared else [0] * S
    st = State(lens, 5, 8, 5, S).device()
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pk().trim_tables(st.d_table, st.d_lens, t(drop), st.d_stack, st.d_free, 8, shared_blocks=t(out) if shared else None, dev_status=st.status)
    back, table = [], st.table.tolist()
    for s, (L, d) in enumerate(zip(lens, drop)):
        first = max(-(-(L - d) // 8), out[s])
        if d:
            back += table[s][first:max(first, -(-L // 8))]
    stack = st.stack.tolist()
    stack[5:5 + len(back)] = back[::-1]
    assert st.d_stack.tolist() == stack and int(st.d_free) == 5 + len(back)
    assert st.d_lens.tolist() == [L - d for L, d in zip(lens, drop)] and int(st.status) == 0


def test_as_many_blocks_as_a_stack_holds():
    """2^31 - 1 blocks of one token, taken by one call and given back by another."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("takes 34 GB")
    S, most, N, part = 16384, 131072, 2 ** 31 - 1, 2 ** 27
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.full((S, most), -1, dtype=torch.int32, device="cuda")
    stack = torch.arange(N, dtype=torch.int32, device="cuda")
    slots = torch.full((N,), -2, dtype=torch.int64, device="cuda")
    lens, new, free, status, starts = t([0] * S), t([most] * (S - 1) + [most - 1]), t([N]), t([0]), t([0] * (S + 1))
    pk().extend_tables(table, lens, new, stack, free, slots, starts, 1, dev_status=status)
    assert int(status) == 0 and int(free) == 0 and lens.equal(new) and int(starts[S]) == N
    flat = table.view(-1)
    for a in range(0, N, part):
        b = min(N, a + part)
        want = torch.arange(N - 1 - a, N - 1 - b, -1, dtype=torch.int32, device="cuda")
        assert flat[a:b].equal(want) and slots[a:b].equal(want.long())
    assert int(flat[N]) == -1
    del slots
    stack.fill_(-3)
    pk().trim_tables(table, lens, new, stack, free, 1, dev_status=status)
    assert int(status) == 0 and int(free) == N and int(lens.count_nonzero()) == 0
    for a in range(0, N, part):
        b = min(N, a + part)
        assert stack[a:b].equal(torch.arange(a, b, dtype=torch.int32, device="cuda"))
