"""A step's plan on the GPU against the oracle: whole numbers, every one equal."""
import numpy as np
import pytest
import torch

from oracle import spear_step as ref
import w4_gemm_gated_amd as sp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DEV = "cuda:0"
NAMES = ("cu_q", "kv_lens", "slots", "positions", "sequence", "held", "free_count", "block_table", "free_pages")


def note(msg):
    print(f"[gpu-kv-plan] {msg}", flush=True)


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def state(rng, B, page, max_len, most_new, spare=0.5, ended=0.1, odd=0.0):
    """Sequences with pages in random places; `odd`: the share of rows that no
    plan can serve."""
    lens = rng.integers(0, max_len + 1, B)
    new = rng.integers(0, most_new + 1, B)
    held = -(-lens // page) + (rng.random(B) < 0.3) * rng.integers(0, 4, B)
    end = rng.random(B) < ended
    lens, new = np.where(end, 0, lens), np.where(end, 0, new)
    most = int(max(held.max(initial=0), (-(-(lens + new) // page)).max(initial=0), 1)) + 1
    pages = int(held.sum())
    need = int(np.maximum(0, -(-(lens + new) // page) - held).sum())
    free = int(need * spare) + 1
    order = rng.permutation(pages + free + 5).astype(np.int32)
    table, at = np.full((B, most), -7, np.int32), 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    stack = np.full(pages + free + 5, -3, np.int32)
    stack[:free] = order[at:at + free]
    bad = rng.random(B) < odd
    kind = rng.integers(0, 5, B)
    lens = np.where(bad & (kind == 0), -5, np.where(bad & (kind == 1), lens + held * page + 1, lens))
    new = np.where(bad & (kind == 2), -1, np.where(bad & (kind == 3), most * page * 2, new))
    held = np.where(bad & (kind == 4), most + 3, held)
    return lens, new, held, table, stack, free


def run(s, rows, page, in_place=False, **more):
    lens, new, held, table, stack, free = s
    t = [dev(lens), dev(new), dev(held), dev(table), dev(stack), dev(np.asarray([free]))]
    if in_place:
        more.update(kv_lens=t[0], held_out=t[2], free_out=t[5])
    out = sp.spear_kv_plan(*t, rows, page_size=page, **more)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (*out, t[3], t[4])]


def check(s, rows, page, **more):
    want = ref.kv_plan(*s[:5], s[5], rows, page)
    for in_place in (False, True):
        for name, x, y in zip(NAMES, run(s, rows, page, in_place, **more), want):
            assert np.array_equal(x, y), (name, in_place)


@pytest.mark.parametrize("B,page,max_len,most_new", [
    (1, 16, 0, 1), (1, 16, 40, 700), (1, 1024, 5000, 3000), (2, 16, 17, 1), (64, 16, 500, 1), (255, 32, 100, 40),
    (256, 16, 64, 3), (257, 16, 64, 3), (1024, 64, 900, 5), (1025, 16, 50, 9), (5000, 16, 80, 2), (40, 16, 300, 2000)])
@pytest.mark.parametrize("spare", [0.0, 0.6, 1.0])
def test_against_the_oracle(B, page, max_len, most_new, spare):
    rng = np.random.default_rng(B + page)
    s = state(rng, B, page, max_len, most_new, spare)
    total = int(s[1].sum())
    for rows in (total, total + 7, total * 2 // 3):
        note(f"B {B} page {page} new {total} rows {rows} free {s[5]}")
        check(s, rows, page)


@pytest.mark.parametrize("B", [1023, 1026, 2047, 2048, 2049, 4100])
def test_a_few_sequences_more_or_less_than_threads_hold(B):
    rng = np.random.default_rng(B)
    s = state(rng, B, 16, 90, 6, 0.7)
    total = int(s[1].sum())
    for rows in (total + 3, total * 3 // 4):
        note(f"B {B} new {total} rows {rows}")
        check(s, rows, 16)


@pytest.mark.parametrize("seed", range(4))
def test_sequences_that_cannot_be_served(seed):
    rng = np.random.default_rng(seed)
    s = state(rng, 700, 16, 100, 20, 0.8, odd=0.2)
    total = int(np.maximum(s[1], 0).sum())
    note(f"impossible sequences, seed {seed}")
    check(s, min(total, 20000), 16)
    lens = np.array([2**31 - 1, 2**31 - 1, 5, -2**31])          # sums past 32 bits
    new = np.array([2**31 - 1, 1, 3, -2**31])
    held = np.array([2**31 - 1, 2, 1, -2**31])
    check((lens, new, held, s[3][:4].copy(), s[4], 9), 10, 16)


def test_nothing_to_do():
    note("no sequences, no rows, an empty stack")
    empty = np.zeros(0, np.int64)
    check((empty, empty, empty, np.zeros((0, 3), np.int32), np.arange(4, dtype=np.int32), 3), 5, 16)
    check((empty, empty, empty, np.zeros((0, 3), np.int32), np.zeros(0, np.int32), 0), 0, 16)
    one = np.array([5])
    check((one, one * 0, one * 0 + 1, np.array([[2, 3]], np.int32), np.zeros(0, np.int32), 0), 0, 16)
    check((one, one, one * 0 + 1, np.array([[2, 3]], np.int32), np.zeros(0, np.int32), 0), 4, 16)


def test_many_pages_given_back():
    """More pages laid on the stack than a workgroup has threads, some taken again at
    once, and a stack too small for all."""
    rng = np.random.default_rng(9)
    for B in (3, 600):
        note(f"many pages given back by {B}")
        s = list(state(rng, B, 16, 30000 if B == 3 else 600, 50, 0.2, ended=0.5))
        s[0][0], s[1][0], s[2][0] = 0, 0, s[3].shape[1] - 1      # the first gives back its whole row
        check(s, int(s[1].sum()), 16)
        few = s[4][:s[5] + 4].copy()
        check((*s[:4], few, s[5]), int(s[1].sum()), 16)
        check((*s[:4], s[4], 10**6), int(s[1].sum()), 16)        # a count past the stack
        check((*s[:4], s[4], -4), int(s[1].sum()), 16)


def test_counter_and_repeats():
    note("the workspace's counters are zero after a call, and a second call agrees")
    rng = np.random.default_rng(5)
    s = state(rng, 900, 16, 200, 30)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    rows = int(s[1].sum())
    for _ in range(2):
        check(s, rows, 16, workspace=ws)
        assert not ws.any()


def test_steps_in_place_as_captured():
    """Twelve steps of a batch on the same tensors, replayed from a graph: every step
    as the oracle's."""
    note("captured steps")
    rng = np.random.default_rng(7)
    B, page, rows = 300, 16, 1500
    s = state(rng, B, page, 60, 4, 30.0)
    t = [dev(s[0]), dev(s[1]), dev(s[2]), dev(s[3]), dev(s[4]), dev(np.asarray([s[5]]))]
    want_table = np.pad(s[3], ((0, 0), (0, 8)), constant_values=-7)
    t[3] = dev(want_table)
    outs = dict(cu_q=torch.empty(B + 1, dtype=torch.int32, device=DEV), slots=torch.empty(rows, dtype=torch.int64, device=DEV),
                positions=torch.empty(rows, dtype=torch.int32, device=DEV),
                sequence=torch.empty(rows, dtype=torch.int32, device=DEV), kv_lens=t[0], held_out=t[2], free_out=t[5],
                workspace=torch.zeros(1 << 20, dtype=torch.uint8, device=DEV))
    saved = [x.clone() for x in t]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        sp.spear_kv_plan(*t, rows, page_size=page, **outs)
    for x, y in zip(t, saved):
        x.copy_(y)
    lens, new, held, table, stack, free = s[0], s[1], s[2], want_table, s[4], s[5]
    for step in range(12):
        g.replay()
        torch.cuda.synchronize()
        w = ref.kv_plan(lens, new, held, table, stack, free, rows, page)
        got = [outs["cu_q"], t[0], outs["slots"], outs["positions"], outs["sequence"], t[2], t[5], t[3], t[4]]
        for name, x, y in zip(NAMES, got, w):
            assert np.array_equal(x.cpu().numpy(), y), (step, name)
        lens, held, free, table, stack = w[1].astype(np.int64), w[5], int(w[6][0]), w[7], w[8]
        new = rng.integers(0, 5, B)
        gone = rng.random(B) < 0.05
        back = np.minimum(lens, rng.integers(0, 3, B))           # refused drafts
        lens = np.where(gone, 0, lens - back)
        new = np.where(gone, 0, new)
        t[0].copy_(dev(lens))
        t[1].copy_(dev(new))


def test_refusals():
    note("refusals")
    s = state(np.random.default_rng(1), 4, 16, 30, 3)
    t = [dev(s[0]), dev(s[1]), dev(s[2]), dev(s[3]), dev(s[4]), dev(np.asarray([s[5]]))]
    for i in range(6):
        for wrong, error in ((t[i].long(), TypeError), (t[i].cpu(), ValueError), (t[i][None], ValueError)):
            with pytest.raises(error):
                sp.spear_kv_plan(*t[:i], wrong, *t[i + 1:], 9)
    with pytest.raises(ValueError):
        sp.spear_kv_plan(t[0][:3], *t[1:], 9)
    with pytest.raises(ValueError):
        sp.spear_kv_plan(*t, 9, slots=torch.empty(8, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        sp.spear_kv_plan(*t, -1)
    for page in (8, 24, 2048):
        with pytest.raises(sp.SpearError, match="UNSUPPORTED"):
            sp.spear_kv_plan(*t, 9, page_size=page)
    with pytest.raises(sp.SpearError, match="SHAPE"):
        sp.spear_kv_plan(*t, 9, page_size=0)
    with pytest.raises(sp.SpearError, match="WORKSPACE"):
        sp.spear_kv_plan(*t, 2000, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
