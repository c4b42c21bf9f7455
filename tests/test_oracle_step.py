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


def test_adapters_by_hand():
    """One row with each adapter and one without: rank 1 products in whole numbers."""
    X = np.array([[1, 2], [3, 4], [5, 6]], np.float16)
    A = np.array([[[1, 0]], [[1, 1]]], np.float16)              # picks x0; x0 + x1
    B = np.array([[[1], [10]], [[2], [0]]], np.float16)
    Y = np.ones((3, 2), np.float16)
    out, slack = ref.adapter_add(Y, X, A, B, [0, 1, 2, 3], [1, -1, 0], [0.5, 3.0])
    assert out.tolist() == [[1 + 3 * 3 * 2, 1], [1, 1], [1 + 0.5 * 5, 1 + 0.5 * 50]]
    assert (slack[1] == 0).all() and (slack[[0, 2], [0, 1]] > 0).all()


def test_adapters_merge_into_the_weight():
    """A batch of one adapter is the product with W + s B A."""
    rng = np.random.default_rng(0)
    X, A, B = (rng.normal(size=s).astype(np.float16) for s in ((6, 40), (2, 8, 40), (2, 24, 8)))
    W = rng.normal(size=(24, 40))
    Y = X.astype(np.float64) @ W.T
    out, _ = ref.adapter_add(Y, X, A, B, [0, 2, 6], [1, 1], [0.0, 0.25])
    merged = W + 0.25 * B[1].astype(np.float64) @ A[1].astype(np.float64)
    assert np.allclose(out, X.astype(np.float64) @ merged.T, rtol=1e-12, atol=1e-12)


def test_rules_by_hand():
    """Weights 8, 4, 2, 1, 1 at temperature 1, among a masked token and a NaN."""
    l = np.log(np.array([2.0, 8, 1, 4, 1])).tolist() + [-np.inf, np.nan]
    keep = lambda *r: ref.kept_tokens(l, *r)[0].tolist()  # noqa: E731
    assert keep() == [1, 3, 0, 2, 4]
    assert keep(1.0, 4) == [1, 3, 0, 2] and keep(1.0, 1) == [1] and keep(1.0, 99) == [1, 3, 0, 2, 4]
    assert keep(1.0, 0, 0.4) == [1] and keep(1.0, 0, 0.51) == [1, 3] and keep(1.0, 0, 0.76) == [1, 3, 0]
    assert keep(1.0, 2, 0.66) == [1] and keep(1.0, 2, 0.67) == [1, 3]       # of 12
    assert keep(1.0, 0, 1.0, 0.24) == [1, 3, 0] and keep(1.0, 0, 1.0, 2.0) == [1]
    assert keep(0.0) == keep(-1.0) == keep(float("nan")) == keep(1.0, 0, 0.0) == [1]
    assert np.allclose(ref.sample(l, None, 0.5, 2)[2], [0, 0.8, 0, 0.2, 0, 0, 0])        # 64 to 16
    assert ref.sample([-np.inf, np.nan], None)[0] == -1
    assert ref.kept_tokens([1.0, np.inf, 2.0, np.inf])[0].tolist() == [1, 3]


def test_the_race_draws_from_the_distribution():
    """Frequencies of 20000 draws within five standard deviations."""
    rng = np.random.default_rng(1)
    l = np.array([0.3, -1.0, 1.2, 0.0, 2.0])
    want = ref.sample(l, None, 0.8, 4)[2]
    n = 20000
    got = np.bincount([ref.sample(l, rng.exponential(size=5).astype(np.float32), 0.8, 4)[0] for _ in range(n)], minlength=5)
    assert (np.abs(got / n - want) <= 5 * np.sqrt(want * (1 - want) / n)).all() and got[1] == 0
