"""Block tables and slot maps built on the device, against the host's."""
import random

import pytest
import torch

import step_common as sc

pytestmark = pytest.mark.gpu


def pk():
    from paged_kv_cache_141_gb300 import binding
    return binding


class State:
    def __init__(self, lens, most, B, spare, seed=0):
        self.B, S = B, len(lens)
        r = random.Random(seed)
        held = [-(-L // B) for L in lens]
        ids = r.sample(range(1, 10 * (sum(held) + spare) + 1), sum(held) + spare)
        self.table = torch.full((S, most), -7, dtype=torch.int32)
        at = 0
        for s, n in enumerate(held):
            self.table[s, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
            at += n
        self.stack = torch.tensor(ids[at:] + ids[:at], dtype=torch.int32)
        self.free, self.lens = spare, list(lens)

    def device(self):
        t = lambda x, d=torch.int32: torch.tensor(x, dtype=d, device="cuda")  # noqa: E731
        self.d_table, self.d_stack = self.table.cuda(), self.stack.cuda()
        self.d_lens, self.d_free, self.status = t(self.lens), t([self.free]), t([0])
        return self


def run_extend(st, new, room=None, in_place=True, positions=True):
    room = sum(max(n, 0) for n in new) if room is None else room
    S = len(new)
    st.device()
    slots = torch.full((room,), 99, dtype=torch.int64, device="cuda")
    pos = torch.full((room,), 99, dtype=torch.int64, device="cuda") if positions else None
    qs = torch.full((S + 1,), 99, dtype=torch.int32, device="cuda")
    lens_out = None if in_place else torch.full((S,), 99, dtype=torch.int32, device="cuda")
    free_out = None if in_place else torch.full((1,), 99, dtype=torch.int32, device="cuda")
    before = (st.d_lens.clone(), st.d_free.clone())
    pk().extend_tables(st.d_table, st.d_lens, torch.tensor(new, dtype=torch.int32, device="cuda"), st.d_stack, st.d_free,
                       slots, qs, st.B, positions=pos, new_lens=lens_out, new_num_free=free_out, dev_status=st.status)
    torch.cuda.synchronize()
    table, w_slots, w_pos, w_qs, w_lens, w_free, denied = sc.extend(st.table, st.lens, new, st.stack.tolist(), st.free, st.B, room)
    assert st.d_table.cpu().equal(table)
    assert slots.tolist() == w_slots
    assert pos is None or pos.tolist() == w_pos
    assert qs.tolist() == w_qs
    if not in_place:
        assert st.d_lens.equal(before[0]) and st.d_free.equal(before[1])
    assert (st.d_lens if in_place else lens_out).tolist() == w_lens
    assert (st.d_free if in_place else free_out).tolist() == [w_free]
    assert st.d_stack.cpu().equal(st.stack)
    return denied, int(st.status.item())


@pytest.mark.parametrize("S", [0, 1, 2, 31, 33, 128, 129, 1000, 1025, 2500])
@pytest.mark.parametrize("B", [1, 16, 24])
def test_extend(S, B):
    r = random.Random(S * 100 + B)
    lens = [r.choice((0, 1, B, B - 1, r.randint(0, 5 * B))) for _ in range(S)]
    new = [r.choice((0, 1, 1, 5, B, r.randint(0, 3 * B))) for _ in range(S)]
    st = State(lens, 10, B, sum(new) + 3, S)
    assert run_extend(st, new, in_place=S % 2 == 0, positions=B != 24) == ([], 0)


@pytest.mark.parametrize("n,B", [(1, 16), (15, 16), (16, 16), (17, 16), (4097, 16), (131072, 16), (70001, 7)])
def test_one_long_request(n, B):
    st = State([3], -(-(n + 3) // B), B, -(-(n + 3) // B), n)
    assert run_extend(st, [n])[0] == []


def test_padded_slot_map():
    st = State([5, 0, 31], 8, 16, 20)
    assert run_extend(st, [3, 2, 4], room=100) == ([], 0)


@pytest.mark.parametrize("spare", [0, 1, 5, 17])
def test_too_few_blocks(spare):
    # those that still fit are served, in order; who needs no block is served all the same
    r = random.Random(spare)
    lens = [r.randint(0, 60) for _ in range(300)]
    new = [r.randint(0, 20) for _ in range(300)]
    st = State(lens, 8, 16, spare, 3)
    denied, status = run_extend(st, new)
    assert denied and status == pk().DEV_NO_BLOCKS


def test_too_few_places():
    st = State([0] * 40, 4, 16, 200)
    denied, status = run_extend(st, [7] * 40, room=100)
    assert denied == list(range(14, 40)) and status == pk().DEV_BAD_LEN


def test_bad_counts():
    st = State([10, 20, 30, 0], 3, 16, 30)
    denied, status = run_extend(st, [-1, 29, 5, 49], room=60)      # below zero; past the table; fine; past the table
    assert denied == [0, 1, 3] and status == pk().DEV_BAD_LEN


@pytest.mark.parametrize("free,taken_as", [(-3, 0), (50, 30)])
def test_bad_free_count(free, taken_as):
    st = State([0, 0], 4, 16, 30)
    st.free = taken_as
    st.device()
    st.d_free.fill_(free)
    slots = torch.empty(2, dtype=torch.int64, device="cuda")
    qs = torch.empty(3, dtype=torch.int32, device="cuda")
    pk().extend_tables(st.d_table, st.d_lens, torch.ones(2, dtype=torch.int32, device="cuda"), st.d_stack, st.d_free, slots, qs, 16,
                       dev_status=st.status)
    want = sc.extend(st.table, [0, 0], [1, 1], st.stack.tolist(), taken_as, 16, 2)
    assert slots.tolist() == want[1] and int(st.d_free) == want[5]
    assert int(st.status) & pk().DEV_BAD_BLOCK_ID


# ------------------------------------------------------------------ trim

@pytest.mark.parametrize("S", [0, 1, 33, 700, 1100])
@pytest.mark.parametrize("shared", [False, True])
def test_trim(S, shared):
    r = random.Random(S)
    B = r.choice((8, 16, 24))
    lens = [r.randint(0, 9 * B) for _ in range(S)]
    drop = [r.choice((0, L, min(L, 3), r.randint(0, L))) for L in lens]
    keep_out = [r.choice((0, 1, 4)) for _ in range(S)] if shared else None
    st = State(lens, 9, B, 5, S).device()
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    pk().trim_tables(st.d_table, st.d_lens, t(drop), st.d_stack, st.d_free, B, shared_blocks=t(keep_out) if shared else None,
                     dev_status=st.status)
    back = []
    for s, (L, d) in enumerate(zip(lens, drop)):
        first = max(-(-(L - d) // B), keep_out[s] if shared else 0)
        if d:
            back += st.table[s, first:max(first, -(-L // B))].tolist()
    stack = st.stack.tolist()
    stack[5:5 + len(back)] = back[::-1]
    assert st.d_stack.tolist() == stack and int(st.d_free) == 5 + len(back)
    assert st.d_lens.tolist() == [L - d for L, d in zip(lens, drop)]
    assert st.d_table.cpu().equal(st.table) and int(st.status) == 0


def test_trim_gives_back_what_extend_took():
    r = random.Random(1)
    lens = [r.randint(0, 100) for _ in range(200)]
    new = [r.randint(0, 40) for _ in range(200)]
    st = State(lens, 16, 16, 1000).device()
    n = torch.tensor(new, dtype=torch.int32, device="cuda")
    slots, qs = torch.empty(sum(new), dtype=torch.int64, device="cuda"), torch.empty(201, dtype=torch.int32, device="cuda")
    pk().extend_tables(st.d_table, st.d_lens, n, st.d_stack, st.d_free, slots, qs, 16)
    first = slots.clone()
    pk().trim_tables(st.d_table, st.d_lens, n, st.d_stack, st.d_free, 16)
    assert st.d_lens.tolist() == lens and int(st.d_free) == 1000 and st.d_stack.cpu().equal(st.stack)
    pk().extend_tables(st.d_table, st.d_lens, n, st.d_stack, st.d_free, slots, qs, 16)
    assert slots.equal(first)


def test_trim_refuses_what_is_not_there():
    t = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    st = State([20, 20, 20], 4, 16, 4).device()
    pk().trim_tables(st.d_table, st.d_lens, t([-1, 21, 5]), st.d_stack, st.d_free, 16, dev_status=st.status)
    assert st.d_lens.tolist() == [20, 20, 15] and int(st.d_free) == 5 and int(st.status) == pk().DEV_BAD_LEN
    # a stack without room: nothing moves
    st = State([64, 64], 4, 16, 4).device()
    small = st.d_stack[:8].contiguous()
    before = small.clone()
    pk().trim_tables(st.d_table, st.d_lens, t([64, 64]), small, st.d_free, 16, dev_status=st.status)
    assert st.d_lens.tolist() == [64, 64] and int(st.d_free) == 4 and small.equal(before)
    assert int(st.status) == pk().DEV_BAD_BLOCK_ID
