"""Pages reserved and given back, and the slots of new tokens, against plain lists."""
import random

import numpy as np
import pytest
import torch

import draft_token_verification_11_amd as sv
from tests import step_plain as plain

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


class State:
    """A pool's state on the GPU and as lists."""

    def __init__(self, B, cols, n, spare=0, seed=0):
        order = list(range(n))
        random.Random(seed).shuffle(order)
        self.rows, self.held_, self.stack, self.n = [[-1] * cols for _ in range(B)], [0] * B, order + [-9] * spare, n
        # rows further apart than their entries
        self.wide = torch.full((B, cols + 3), 55, dtype=torch.int32, device=DEV)
        self.table = self.wide[:, :cols]
        self.table.fill_(-1)
        self.held, self.free, self.count = _i32(self.held_), _i32(self.stack), _i32([n])

    def step(self, need):
        sv.cache4_reserve(self.table, self.held, _i32(need), self.free, self.count)
        self.n = plain.reserve(self.rows, self.held_, need, self.stack, self.n)

    def check(self):
        assert int(self.count) == self.n
        assert self.held.tolist() == self.held_
        assert self.table.tolist() == self.rows
        assert self.free.tolist() == self.stack
        assert (self.wide[:, self.table.shape[1]:] == 55).all()


@pytest.mark.parametrize("B,cols,n", [(1, 1, 1), (1, 40, 64), (3, 5, 9), (64, 30, 700), (65, 9, 300), (128, 12, 900),
                                      (129, 12, 900), (1024, 4, 2500),
                                      (1025, 3, 3500), (3000, 3, 5000), (17, 400, 3000)])
def test_random_steps(B, cols, n):
    """Growing, shrinking and ending, with enough pages and with too few."""
    r = random.Random(B)
    s = State(B, cols, n, seed=B)
    for step in range(12):
        top = 64 * cols if step % 3 else max(64, 64 * n // (2 * B))
        s.step([r.choice([0, r.randint(0, min(top, 64 * cols)), 64 * s.held_[b], max(0, 64 * s.held_[b] - 63)]) for b in range(B)])
        s.check()


def test_back_again():
    """A call with the former lengths restores every entry."""
    r = random.Random(5)
    s = State(200, 12, 4000)
    need = [r.randint(0, 64 * 12) for _ in range(200)]
    s.step(need)
    before = [x.clone() for x in (s.table, s.held, s.free, s.count)]
    for _ in range(3):
        s.step([r.choice([0, x, min(768, x + 70), max(0, x - 200)]) for x in need])
        s.check()
        s.step(need)
        s.check()
        assert int(s.count) == int(before[3])
        assert all(torch.equal(x, y) for x, y in zip(before[:2], (s.table, s.held)))
        n = s.n
        assert torch.equal(before[2][:n], s.free[:n])


def test_served_in_turn():
    """The first sequence that finds too few pages and all after it wait, also those that a page
    would do; pages that go back in the same call are there for them."""
    s = State(5, 8, 6)
    s.step([128, 64, 0, 0, 0])
    s.step([64, 256, 512, 64, 64])   # 3 free and one back: two more for 1, then 2 finds too few
    s.check()
    assert s.held_ == [1, 4, 0, 0, 0]
    s.step([64, 256, 0, 64, 64])
    s.check()
    assert s.held_ == [1, 4, 0, 1, 0]
    s.step([64, 0, 0, 64, 64 * 5])
    s.check()
    assert s.held_ == [1, 0, 0, 1, 0]
    s.step([0, 0, 0, 0, 64 * 5 + 1])
    s.check()
    assert s.held_ == [0, 0, 0, 0, 6]


def test_data_faults_change_nothing():
    s = State(6, 4, 20)
    s.step([64, 128, 200, 10, 0, 256])
    s.check()
    s.step([-1, -2147483648, 257, 2147483647, 64, 0])   # lengths that no table holds: the others go on
    s.check()
    assert s.held_ == [1, 2, 4, 1, 1, 0]
    for bad in (-1, 5, 2147483647, -2147483648):
        s.held_[1] = bad
        s.held[1] = bad
        s.step([0, 64, 64, 0, 64, 0])
        s.check()
        s.held_[1] = 2
        s.held[1] = 2
    for bad in (-1, -2147483648, 21, 2147483647):     # a count that the list does not hold
        keep, s.n = s.n, bad
        s.count.fill_(bad)
        s.step([64] * 6)
        s.check()
        s.n = keep
        s.count.fill_(keep)
    s.n = 20                                            # more pages than the list has room for
    s.count.fill_(20)
    s.step([0] * 6)
    s.check()
    s.n = 19
    s.count.fill_(19)
    s.step([0, 128, 256, 64, 64, 0])
    s.check()


def test_most_sequences():
    B, cols = 1 << 16, 2
    s = State(B, cols, B + 500)
    for need in ([64 * (b % 3) for b in range(B)], [128 * (b % 2) for b in range(B)], [0] * B):
        s.step(need)
        s.check()


def test_rows_past_4_gib_apart_and_another_stream():
    wide = torch.full((3, (1 << 30) + 8), 55, dtype=torch.int32, device=DEV)
    table = wide[:, :8]
    table.fill_(-1)
    held, free, count = _i32([0, 0, 0]), _i32(range(20)), _i32([20])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sv.cache4_reserve(table, held, _i32([64, 65, 500]), free, count, stream=s)
    slots = sv.cache4_slots(table, _i32([0, 64, 499]), 1, 20, stream=s)
    s.synchronize()
    assert table.tolist() == [[19] + [-1] * 7, [18, 17] + [-1] * 6, list(range(16, 8, -1))]
    assert held.tolist() == [1, 2, 8] and int(count) == 9
    assert slots.tolist() == [[19 * 64], [17 * 64], [9 * 64 + 51]]
    assert (wide[:, 8:16] == 55).all()


def test_one_sequence_of_many_pages():
    n = 200_000
    held, need, free, count = _i32([0]), _i32([64 * n]), torch.arange(n, dtype=torch.int32, device=DEV), _i32([n])
    table = torch.full((1, n), -1, dtype=torch.int32, device=DEV)
    sv.cache4_reserve(table, held, need, free, count)
    assert torch.equal(table[0], torch.arange(n - 1, -1, -1, dtype=torch.int32, device=DEV)) and int(count) == 0
    sv.cache4_reserve(table, held, _i32([1]), free, count)
    assert table[0, 0] == n - 1 and (table[0, 1:] == -1).all() and int(count) == n - 1 and int(held) == 1
    assert torch.equal(free, torch.arange(n, dtype=torch.int32, device=DEV))


def test_captured_reserve_of_many_sequences():
    """Both kernels in a graph, replayed with other lengths in place."""
    r = random.Random(3)
    s = State(2000, 6, 9000)
    need = _i32([0] * 2000)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        sv.cache4_reserve(s.table, s.held, need, s.free, s.count)
    for _ in range(6):
        lengths = [r.randint(0, 384) for _ in range(2000)]
        need.copy_(_i32(lengths))
        g.replay()
        torch.cuda.synchronize()
        s.n = plain.reserve(s.rows, s.held_, lengths, s.stack, s.n)
        s.check()


def test_slots_of_more_than_32_bits_of_tokens():
    B, T = 1 << 16, (1 << 15) + 1
    table = torch.arange(B, dtype=torch.int32, device=DEV)[:, None].expand(B, 1).contiguous()
    start = torch.arange(B, dtype=torch.int32, device=DEV) % 64
    got = sv.cache4_slots(table, start, T, B, count=torch.ones(B, dtype=torch.int32, device=DEV))
    b = torch.arange(B, device=DEV)
    assert torch.equal(got[:, 0], b * 64 + b % 64)
    assert bool((got[:, 1] == -1).all()) and bool((got[:, T - 1] == -1).all()) and bool((got[-1, 1:] == -1).all())


@pytest.mark.parametrize("T", [1, 7, 300])
def test_slots(T):
    start, count = [0, 63, 60, -1, 10, 200, 250, 5, 2147483647], [T, T, T - 1, T, 0, T, T, T + 1, T]
    cols, n_pages = 12, 40
    table = np.random.default_rng(T).permutation(9 * cols).reshape(9, cols).astype(np.int32) % 45
    table[5, 3] = -1
    for cnt in (count, None):
        got = sv.cache4_slots(_i32(table), _i32(start), T, n_pages, count=None if cnt is None else _i32(cnt)).tolist()
        for b in range(9):
            n = T if cnt is None else cnt[b]
            ok = start[b] >= 0 and 0 <= n <= T and start[b] + n <= 64 * cols
            for i in range(T):
                page = int(table[b, (start[b] + i) // 64]) if ok and i < n else -1
                want = 64 * page + (start[b] + i) % 64 if 0 <= page < n_pages else -1
                assert got[b][i] == want, (b, i)


def test_slots_past_32_bits():
    table = _i32([[2147483646, 0]])
    got = sv.cache4_slots(table, _i32([62]), 3, 2147483647)
    assert got.tolist() == [[64 * 2147483646 + 62, 64 * 2147483646 + 63, 0]]
