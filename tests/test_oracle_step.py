"""The step oracle against hand-worked steps and against what a plan has to keep."""
import numpy as np
import pytest

from oracle import spear_step as ref


def plan(lens, new, held, table, free, rows, page=16, count=None):
    f = np.asarray(free, np.int32)
    return ref.kv_plan(np.asarray(lens), np.asarray(new), np.asarray(held), np.asarray(table, np.int32), f,
                       len(f) if count is None else count, rows, page)


def test_a_step_by_hand():
    """Sequence 0 goes on within its page, 1 has ended and gives back pages 5 and 6, 2
    begins with 20 tokens: its pages are the last one laid on the stack, then the
    one before."""
    cu, kv, slots, pos, seq, held, count, table, free = plan(
        [3, 0, 0], [1, 0, 20], [1, 2, 0], [[4, -1], [5, 6], [-1, -1]], [7, 8, -1, -1], 22, count=2)
    assert cu.tolist() == [0, 1, 1, 21] and kv.tolist() == [4, 0, 20]
    assert table.tolist() == [[4, -1], [5, 6], [6, 5]]
    assert slots.tolist() == [4 * 16 + 3] + [6 * 16 + i for i in range(16)] + [5 * 16 + i for i in range(4)] + [-1]
    assert pos.tolist() == [3] + list(range(20)) + [-1] and seq.tolist() == [0] + [2] * 20 + [-1]
    assert held.tolist() == [1, 0, 2] and count.tolist() == [2] and free.tolist() == [7, 8, -1, -1]


def test_what_stays_on_the_stack_is_written_there():
    cu, _, _, _, _, held, count, _, free = plan([0, 16], [0, 1], [3, 1], [[1, 2, 3], [4, -1, -1]], [9, 0, 0, 0, 0], 4, count=1)
    assert held.tolist() == [0, 2] and count.tolist() == [3]        # 9, 1, 2 stay, 3 is taken
    assert free.tolist() == [9, 1, 2, 0, 0] and cu.tolist() == [0, 0, 1]


def test_from_the_first_that_does_not_fit_none_is_served():
    """One page for two that need one: the second gets nothing, nor does the third,
    though it needs none; an impossible sequence in front is passed over."""
    cu, kv, slots, _, _, held, count, _, _ = plan([5, 16, 16, 3], [99, 1, 1, 1], [1, 1, 1, 1],
                                                  [[0, -1], [1, -1], [2, -1], [3, -1]], [7], 10)
    assert cu.tolist() == [0, 0, 1, 1, 1] and kv.tolist() == [5, 17, 16, 3] and held.tolist() == [1, 2, 1, 1]
    assert count.tolist() == [0] and slots[0] == 7 * 16


@pytest.mark.parametrize("seed", range(20))
def test_pages_are_neither_lost_nor_shared(seed):
    rng = np.random.default_rng(seed)
    B, page, most, cap = 30, 16, 9, 200
    order = rng.permutation(cap).astype(np.int32)
    lens = rng.integers(0, 100, B)
    held = -(-lens // page) + rng.integers(0, 2, B)
    table, at = np.full((B, most), -1, np.int32), 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    count = int(rng.integers(0, cap - at + 1))
    free = np.full(cap, -1, np.int32)
    free[:count] = order[at:at + count]
    ended = rng.random(B) < 0.2
    new = np.where(ended, 0, rng.integers(0, 40, B))
    lens = np.where(ended, 0, lens)
    rows = int(rng.integers(0, new.sum() + 5))
    cu, kv, slots, pos, seq, now, left, table, free = ref.kv_plan(lens, new, held, table, free, count, rows, page)
    used = [int(x) for b in range(B) for x in table[b, :now[b]]] + free[:left[0]].tolist()
    assert sorted(used) == sorted(order[:at + count].tolist())
    assert cu[-1] <= rows and np.all(now * page >= kv)
    got = slots[slots >= 0]
    assert len(got) == cu[-1] and len(set(got.tolist())) == len(got)
