"""The draw of next tokens on the GPU against the oracle in 64 bits.

Which tokens are left: equal to the oracle's, except that top-p's cut may fall one way
or the other where the sum before it is within 2^-31 of its mass (weights enter the
sums to 2^-33 of themselves, and a selection's to 2^-40 of a bin's edge).

Probabilities: the weight is an fp32 power of two of an argument exact to 2^-25 (one
step of the hardware's exponential: 2^-23), the sum's reciprocal and the product are
rounded once each: together below 2^-21 of the value, or 2^-149 beneath the normal
numbers.

Tokens: the scores' weights are as near (2^-22 with the division), so the oracle's
score of the drawn token is within 2^-21 of its largest; it is the oracle's token
where no other is that near.
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import spear_step as ref
import w4_gemm_gated_amd as sp
from w4_gemm_gated_amd import _binding, serve
from w4_gemm_gated_amd._binding import SampleDesc

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-sample] {msg}", flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def logits(rng, B, V, dtype=np.float16, width=2.2):
    z = rng.normal(0, width, size=(B, V))
    z[:, rng.integers(0, V, 1 + V // 500)] += rng.exponential(3, size=1 + V // 500)
    return z.astype(dtype)


def check_row(b, l, noise, rules, token, probs):
    """One draw's results against the oracle's, with top-p's cut on either side of a
    sum that is as good as its mass."""
    for nudge in (0.0, 2.0 ** -31, -2.0 ** -31):
        want, scores, p = ref.sample(l, noise, *rules, nudge=nudge)
        if probs is None or np.array_equal(probs > 0, p > 2.0 ** -150):
            break
    if probs is not None:
        off = np.abs(probs.astype(np.float64) - p)
        assert (off <= p * 2.0 ** -21 + 2.0 ** -149).all(), (b, rules, int((probs > 0).sum()), int((p > 0).sum()),
                                                             float(off.max()))
    if token is None:
        return
    if scores is None or want < 0:
        assert token == want, (b, rules, token, want)
        return
    assert 0 <= token < len(l), (b, rules, token)
    best = scores[want]
    assert scores[token] >= best * (1 - 2.0 ** -21) or scores[token] == best, (b, rules, token, want)
    if (scores >= best * (1 - 2.0 ** -21)).sum() == 1 or best == scores[token] == np.inf:
        assert token == want, (b, rules, token, want)


def settings(rules):
    t, k, p, m = zip(*rules)
    return dict(temperature=dev(np.array(t, np.float32)), top_k=dev(np.array(k, np.int32)),
                top_p=dev(np.array(p, np.float32)), min_p=dev(np.array(m, np.float32)))


def check(l, noise, rules, rows=None, **more):
    """Tokens, probabilities, and both, of one call each; `rules`: (temperature, top_k,
    top_p, min_p) of each draw."""
    rules = [(np.float32(t), int(k), np.float32(p), np.float32(m)) for t, k, p, m in rules]
    d, n, s = dev(l), dev(noise), settings(rules)
    r = None if rows is None else dev(np.array(rows, np.int32))
    both = sp.spear_sample(d, n, rows=r, probs=True, **s, **more)
    tokens, none = sp.spear_sample(d, n, rows=r, **s, **more)
    assert none is None
    none, probs = sp.spear_sample(d, rows=r, probs=True, **s, **more)
    assert none is None
    torch.cuda.synchronize()
    assert torch.equal(both[0], tokens) and torch.equal(both[1], probs)
    tokens, probs = tokens.cpu().numpy(), probs.cpu().numpy()
    for b, rule in enumerate(rules):
        i = b if rows is None else rows[b]
        row = l[i] if 0 <= i < len(l) else np.full(l.shape[1], -np.inf, l.dtype)
        check_row(b, row, noise[b], rule, int(tokens[b]), probs[b])


RULES = [(1.0, 0, 1.0, 0.0), (0.7, 50, 1.0, 0.0), (0.9, 0, 0.9, 0.0), (1.2, 0, 1.0, 0.05), (0.8, 40, 0.95, 0.02),
         (0.0, 0, 1.0, 0.0), (1.0, 1, 0.5, 0.0), (1.3, 200, 0.3, 0.0), (0.5, 0, 0.999, 0.0), (2.5, 3, 0.99, 0.3),
         (1.0, 10**6, 0.6, 1e-6), (0.2, 7, 0.0, 0.0)]


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 63, 511, 1000, 8191, 8192, 8193, 32000, 50257, 131071])
def test_against_the_oracle(V, dtype):
    note(f"V {V} {np.dtype(dtype).name}")
    rng = np.random.default_rng(V)
    check(logits(rng, len(RULES), V, dtype), rng.exponential(size=(len(RULES), V)).astype(np.float32), RULES)


@pytest.mark.parametrize("seed", range(6))
def test_random_rules(seed):
    note(f"random rules, seed {seed}")
    rng = np.random.default_rng(100 + seed)
    B, V = 40, int(rng.integers(1000, 40000))
    rules = [(rng.uniform(0.3, 2), rng.choice([0, 1, 2, 20, 1000, 5000]), rng.choice([1.0, rng.uniform(0.01, 1)]),
              rng.choice([0.0, rng.uniform(0.0001, 0.5)])) for _ in range(B)]
    l = logits(rng, B, V, [np.float16, np.float32][seed % 2], rng.uniform(0.1, 4))
    l[rng.random(l.shape) < 0.3 * (seed % 3)] = -np.inf
    check(l, rng.exponential(size=(B, V)).astype(np.float32), rules)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("V", [5000, 40001])
def test_equal_logits(V, dtype):
    """Rows of one value, or of two: cuts go by the index, in bins that hold more tokens
    than any list."""
    note(f"equal logits, V {V}")
    rng = np.random.default_rng(2)
    rules = [(1.0, 5, 1.0, 0.0), (0.5, 0, 0.5, 0.0), (1.0, 4500, 1.0, 0.0), (1.0, 4500, 0.25, 0.5), (3.0, V - 1, 0.999, 0.0),
             (1.0, 0, 1.0, 1.0), (0.0, 0, 1.0, 0.0), (1.0, 0, 1.0, 0.0)]
    noise = rng.exponential(size=(len(rules), V)).astype(np.float32)
    for value in (0.0, -7.25, 30000.0):
        check(np.full((len(rules), V), value, dtype), noise, rules)
    l = np.where(rng.random((len(rules), V)) < 0.5, 1.5, 1.25).astype(dtype)
    check(l, noise, rules)
    l[:, ::3] = -0.0                                    # as +0
    l[:, 1::3] = 0.0
    l[:, 2::3] = -1.0
    check(l, noise, rules)


@pytest.mark.parametrize("V", [6517, 9000, 40000])
def test_tokens_too_light_to_count(V):
    """A few tokens so far above all others that these weigh nothing, with a top-k
    that reaches into them; the others are many, and alone in most of the row."""
    note(f"tokens that weigh nothing, V {V}")
    rng = np.random.default_rng(V)
    rules = [(0.05, 1000, 1.0, 1e-6), (0.05, 1000, 0.999, 0.9), (0.05, 1000, 0.01, 0.0), (0.05, 5, 0.5, 0.0),
             (0.05, 2, 1.0, 0.0), (0.05, V - 1, 0.9, 0.0), (0.02, 300, 0.95, 0.0), (0.001, 100, 1.0, 0.0)]
    for dtype in (np.float16, np.float32):
        l = rng.normal(0, 0.1, size=(len(rules), V)).astype(dtype)
        l[:, rng.permutation(min(V, 4096))[:4]] += np.array([6.3, 6.0, 3.9, 3.2], dtype)
        check(l, rng.exponential(size=l.shape).astype(np.float32), rules)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_many_light_tokens_count_in_the_sum(dtype):
    """One heavy token, and more equal light ones than any list holds, cut by top-k: each is
    next to nothing, all of them a millionth or more of what is kept."""
    note(f"many light tokens {np.dtype(dtype).name}")
    V = 1 << 22
    rng = np.random.default_rng(11)
    l = np.full((3, V), -27.0378, dtype)          # weights of 1.99 2^-40, then of 2^-41, then of both
    l[1] = -28.4
    l[2, ::2] = -28.4
    l[:, 12345] = 0
    check(l, rng.exponential(size=l.shape).astype(np.float32), [(1.0, V - 1, 1.0, 0.0)] * 3)


@pytest.mark.parametrize("light", [-12.3, -17.1, -20.4, -22.9])
@pytest.mark.parametrize("V", [3000, 131072])
def test_top_p_among_light_tokens_below_a_heavy_one(V, light):
    """Top-k ends among equal light tokens, top-p before or within them: its cut is looked
    for from the heavy token's bin on, and the light ones enter the sums whole.

    The sum before the cut may be off by 2^-31 of its mass, which is 2^-31 of the heavy
    token (its own weight enters to 2^-33): that is one token's weight or less down to a
    logit of -21.5, and four tokens' at -22.9, so the count lies between the oracle's for
    masses 2^-31 below and above.  Given the count, the light tokens kept are the first
    ones and the probabilities follow, as near as the others' are.
    """
    note(f"top-p among light tokens, V {V} logit {light}")
    rng = np.random.default_rng(12)
    w = np.exp(np.float64(np.float32(light)))
    rules = []
    for part in (0.1, 0.35, 0.6, 0.85):
        p = np.float32((1 + part * (V - 2) * w) / (1 + (V - 2) * w))       # (V - 2 light tokens are left by top-k)
        rules.append((1.0, V - 1, p, 0.0))
    l = np.full((len(rules), V), light, np.float32)
    l[:, 7] = 0
    noise = rng.exponential(size=l.shape).astype(np.float32)
    tokens, probs = sp.spear_sample(dev(l), dev(noise), probs=True, **settings(rules))
    tokens, probs = tokens.cpu().numpy(), probs.cpu().numpy()
    for b, rule in enumerate(rules):
        least, most = (len(ref.kept_tokens(l[b], *rule, nudge=x)[0]) for x in (-2.0 ** -31, 2.0 ** -31))
        kept = int((probs[b] > 0).sum())
        assert least <= kept <= most, (b, rule, kept, least, most)
        check_row(b, l[b], noise[b], (1.0, kept, 1.0, 0.0), int(tokens[b]), probs[b])


def test_flat_rows():
    """Distinct logits in a few bins: a selection over the row, step by step."""
    note("flat rows")
    rng = np.random.default_rng(3)
    V = 70001
    rules = [(50.0, 1234, 1.0, 0.0), (50.0, 0, 0.777, 0.0), (50.0, 30000, 0.5, 0.0), (1e30, 0, 0.3, 0.0), (np.inf, 17, 1.0, 0.0),
             (20.0, 0, 0.6, 0.95), (9.0, 60000, 0.97, 0.0), (5.0, 0, 0.2, 0.0)]
    check(rng.normal(size=(len(rules), V)).astype(np.float32), rng.exponential(size=(len(rules), V)).astype(np.float32), rules)


def test_special_values():
    note("infinities, NaN, masked rows, extreme temperatures")
    rng = np.random.default_rng(4)
    V = 9001
    for dtype in (np.float16, np.float32):
        for rule in RULES + [(1e-30, 0, 0.9, 0.1), (1e-45, 30, 1.0, 0.0), (np.nan, 3, 0.4, 0.0), (-2.0, 0, 1.0, 0.0),
                             (np.inf, 0, 0.5, 0.0), (1.0, -5, np.nan, np.nan), (1.0, 2, 1e-40, 7.0)]:
            l = logits(rng, 8, V, dtype)
            l[0] = -np.inf
            l[1] = np.nan
            l[2, ::2] = np.nan
            l[3, [5, 70, 8999]] = np.inf
            l[4] = -np.inf
            l[4, 8500] = -3.0
            l[5, :8192] = -np.inf
            l[6] = np.finfo(dtype).min
            l[6, 77] = np.finfo(dtype).max
            l[7] *= dtype(1000) if dtype == np.float32 else dtype(100)
            check(l, rng.exponential(size=(8, V)).astype(np.float32), [rule] * 8)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("V", [3, 5000])
def test_extreme_settings(V, dtype):
    """Settings at the ends of their types, over logits of every size.  (No min-p of 1:
    the oracle's weights round to 1 there, and the logits' order decides here.)"""
    note(f"extreme settings, V {V} {np.dtype(dtype).name}")
    rng = np.random.default_rng(V)
    rules = [(np.inf, 0, 0.9, 0), (1e-45, 0, 0.9, 0), (1e-38, 50, 0.9, 0.1), (1e30, 5, 0.5, 0.1), (3e38, 0, 1, 0.99),
             (1, -4, 1.5, -1), (1, 2**31 - 1, 1, 0.5), (-1, 0, 1, 0), (np.nan, 3, 0.5, 0), (1, 0, 1e-45, 0),
             (1, 0, 1 - 2**-24, 0), (1, 0, 1, 1e-45), (1, 0, 1, 1e-38), (100, V - 1, 0.99999, 0)]
    n, info = len(rules), np.finfo(dtype)
    noise = rng.exponential(size=(n, V)).astype(np.float32)
    alone = np.full((n, V), -np.inf, dtype)
    alone[:, V // 2] = 3
    wide = np.full((n, V), info.max, dtype)
    wide[:, ::2] *= -1
    small = np.full((n, V), info.tiny, dtype)
    small[:, ::2] = info.smallest_subnormal
    small[:, ::3] = -0.0
    for l in (logits(rng, n, V, dtype), alone, np.full((n, V), np.inf, dtype), wide, small):
        check(l, noise, rules)


@pytest.mark.parametrize("offset", [-3e4, 1000.0, 65000.0])
def test_logits_far_from_zero(offset):
    """Rows whose logits share a large offset: their place on the bins' grid is a product
    rounded to 64 bits, 2^-53 |l| / temperature of a weight, which 2^-33 of itself holds up
    to a quotient of 2^20.  (Steps of fp32 there: 2^-8; of the weights at 0.07: 5 %.)"""
    note(f"offset {offset}")
    rng = np.random.default_rng(14)
    rules = [(0.07, 0, 0.9, 0.0), (0.07, 40, 0.6, 0.0), (0.5, 3000, 0.95, 0.01), (1.0, 0, 0.3, 0.0), (2.0, 7000, 0.999, 0.0)]
    l = (logits(rng, len(rules), 9001, np.float32) + np.float32(offset)).astype(np.float32)
    check(l, rng.exponential(size=l.shape).astype(np.float32), rules)


def test_noise_values():
    """Zero noise wins, infinite noise loses to any other, NaN takes no part; ties go to
    the lowest index."""
    note("noise")
    V = 20000
    rng = np.random.default_rng(5)
    l = np.zeros((6, V), np.float32)
    noise = np.ones((6, V), np.float32)
    noise[0, 12345] = noise[0, 17000] = 0.0
    noise[1] = np.inf
    noise[2, :] = np.nan
    noise[3, :15000] = np.nan
    noise[4] = -1.0
    noise[5] = rng.exponential(size=V)
    tokens, _ = sp.spear_sample(dev(l), dev(noise))
    assert tokens.tolist()[:5] == [12345, 0, -1, 15000, -1]
    tokens, _ = sp.spear_sample(dev(l), dev(noise), top_k=13000)
    assert tokens.tolist()[:5] == [12345, 0, -1, -1, -1]
    assert tokens[5] == int(noise[5, :13000].argmin())


def test_numbers_for_all_and_greedy_without_noise():
    note("settings as numbers")
    rng = np.random.default_rng(6)
    l = logits(rng, 9, 12345)
    noise = rng.exponential(size=l.shape).astype(np.float32)
    rule = (0.8, 30, 0.9, 0.01)
    want = sp.spear_sample(dev(l), dev(noise), probs=True, **settings([rule] * 9))
    got = sp.spear_sample(dev(l), dev(noise), 0.8, 30, 0.9, 0.01, probs=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    first = torch.from_numpy(l.argmax(1).astype(np.int32)).to(DEV)
    for one in (dict(temperature=0), dict(top_k=1), dict(top_p=0.0)):
        tokens, probs = sp.spear_sample(dev(l), probs=True, **one)
        assert torch.equal(tokens, first) and torch.equal(probs.argmax(1).int(), first)
        assert torch.equal(probs.sum(1), torch.ones(9, device=DEV))
    assert sp.spear_sample(dev(l), top_k=2**32 + 1, probs=True)[0] is None


def test_numbers_that_change_from_call_to_call():
    """What is kept for a call's sizes does not grow with its settings (NaN, which equals
    nothing, among them), and each call goes by its own."""
    note("settings that change")
    rng = np.random.default_rng(13)
    l = logits(rng, 5, 777)
    noise = rng.exponential(size=l.shape).astype(np.float32)
    d, n = dev(l), dev(noise)
    sp.spear_sample(d, n)
    kept = len(serve._plans)
    calls = [dict(temperature=0.5 + i / 16, top_k=3 + i, top_p=0.5 + i / 64, min_p=i / 256) for i in range(20)]
    for rule in calls + calls[::-1] + [dict(temperature=float("nan"))] * 2 + [dict(top_p=float("nan"))]:
        got = sp.spear_sample(d, n, probs=True, **rule)
        full = (rule.get("temperature", 1.0), rule.get("top_k", 0), rule.get("top_p", 1.0), rule.get("min_p", 0.0))
        want = sp.spear_sample(d, n, probs=True, **settings([full] * 5))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert len(serve._plans) == kept


def test_rows_and_strides():
    """Draws from some rows of a wider tensor, one of them twice, two outside it."""
    note("rows and strides")
    rng = np.random.default_rng(7)
    rows = [3, 0, 3, -1, 6, 5, 2**31 - 1]
    rules = [RULES[i % 5] for i in range(len(rows))]
    for dtype in (np.float16, np.float32):
        for V, width, at in ((8200, 8205, 3), (500, 501, 1), (16384, 16400, 0)):
            l = logits(rng, 6, V, dtype)
            noise = rng.exponential(size=(len(rows), V)).astype(np.float32)
            wide = torch.full((6, width), 9e4 if dtype == np.float32 else 6e4, dtype=dev(l).dtype, device=DEV)
            wide[:, at:at + V] = dev(l)
            s = settings(rules)
            tokens, probs = sp.spear_sample(wide[:, at:at + V], dev(noise), rows=dev(np.array(rows, np.int32)), probs=True, **s)
            for b, (i, rule) in enumerate(zip(rows, rules)):
                row = l[i] if 0 <= i < 6 else np.full(V, -np.inf, dtype)
                r = (np.float32(rule[0]), rule[1], np.float32(rule[2]), np.float32(rule[3]))
                check_row(b, row, noise[b], r, int(tokens[b]), probs[b].cpu().numpy())


@pytest.mark.parametrize("B,V", [(5000, 40), (700, 60000), (3, 1 << 22), (1, 131072)])
def test_many_draws_and_long_rows(B, V):
    """More rows than one launch takes, and the longest vocabulary: some of them against
    the oracle, all against calls of a row each where they are few."""
    note(f"{B} draws of {V}")
    g = torch.Generator(device=DEV)
    g.manual_seed(B)
    l = torch.empty(B, V, dtype=torch.float16, device=DEV).normal_(0, 2, generator=g)
    noise = torch.empty(B, V, device=DEV).exponential_(generator=g)
    rules = [RULES[b % 5] for b in range(B)]
    s = settings(rules)
    tokens, _ = sp.spear_sample(l, noise, **s)
    out = torch.full((B, V), 3.0, device=DEV)
    _, probs = sp.spear_sample(l, probs=out, **s)
    assert probs is out
    assert bool(((probs.double().sum(1) - 1).abs() < 1e-5).all())
    for b in sorted({0, 1, 2, B // 2, B - 1} & set(range(B))):
        t, k, p, m = rules[b]
        check_row(b, l[b].cpu().numpy(), noise[b].cpu().numpy(), (np.float32(t), k, np.float32(p), np.float32(m)),
                  int(tokens[b]), probs[b].cpu().numpy())


def test_the_draw_follows_the_distribution():
    """4000 draws from one row: frequencies within five standard deviations."""
    note("frequencies")
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    l = torch.tensor([[0.3, -1.0, 1.2, 0.0, 2.0, -float("inf")]], device=DEV)
    n = 4000
    noise = torch.empty(n, 6, device=DEV).exponential_(generator=g)
    tokens, probs = sp.spear_sample(l, noise, 0.8, 4, 0.95, rows=torch.zeros(n, dtype=torch.int32, device=DEV), probs=True)
    want = probs[0].double().cpu().numpy()
    got = np.bincount(tokens.cpu().numpy(), minlength=6) / n
    assert (np.abs(got - want) <= 5 * np.sqrt(want * (1 - want) / n)).all() and got[5] == 0


def test_counters_repeats_and_streams():
    note("workspace counters, another stream")
    rng = np.random.default_rng(8)
    l, noise = dev(logits(rng, 12, 33000)), dev(rng.exponential(size=(12, 33000)).astype(np.float32))
    s = settings(RULES)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    want = sp.spear_sample(l, noise, probs=True, workspace=ws, **s)
    for _ in range(3):
        got = sp.spear_sample(l, noise, probs=True, workspace=ws, **s)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert not ws[:1 << 20].any()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        got = sp.spear_sample(l, noise, probs=True, **s)
    stream.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("B,V", [(40, 1000), (300, 4096), (300, 4097), (20, 16385), (4100, 50)])
def test_a_workspace_of_just_the_bytes_asked_for(B, V):
    """What stays within a workgroup has no place in the workspace: a call works in the
    bytes that it asks for, and leaves what lies behind them."""
    note(f"workspace of {B} draws of {V}")
    rng = np.random.default_rng(V)
    l, noise = dev(logits(rng, B, V)), dev(rng.exponential(size=(B, V)).astype(np.float32))
    s = settings([RULES[b % len(RULES)] for b in range(B)])
    want = sp.spear_sample(l, noise, probs=True, **s)
    need = ctypes.c_size_t(0)
    d = SampleDesc(B, V, B, 0, 0.0, 0, 0.0, 0.0)
    assert _binding.load().spear_sample_workspace_bytes(ctypes.byref(d), ctypes.byref(need)) == 0
    ws = torch.full((need.value + (4 << 20),), 77, dtype=torch.uint8, device=DEV)
    ws[:need.value] = 0
    got = sp.spear_sample(l, noise, probs=True, workspace=ws[:need.value], **s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((ws[need.value:] == 77).all()) and not ws[:1 << 20].any()


def test_graph_replays():
    note("captured draws")
    rng = np.random.default_rng(9)
    B, V = 12, 20000
    first = [(logits(rng, B, V), rng.exponential(size=(B, V)).astype(np.float32)) for _ in range(2)]
    l, noise = dev(first[0][0]), dev(first[0][1])
    s = settings(RULES)
    ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
    tokens, probs = torch.zeros(B, dtype=torch.int32, device=DEV), torch.zeros(B, V, device=DEV)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        sp.spear_sample(l, noise, tokens=tokens, probs=probs, workspace=ws, **s)
    for i in (1, 0, 1, 1):
        l.copy_(dev(first[i][0]))
        noise.copy_(dev(first[i][1]))
        want = sp.spear_sample(l, noise, probs=True, **s)
        tokens.fill_(-9)
        probs.fill_(-9)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(tokens, want[0]) and torch.equal(probs, want[1])


def test_refusals():
    note("refusals")
    l, noise = torch.zeros(3, 50, dtype=torch.float16, device=DEV), torch.ones(3, 50, device=DEV)
    for bad in (l.bfloat16(), l.double(), l.int()):
        with pytest.raises(TypeError):
            sp.spear_sample(bad, noise)
    for bad in (l.cpu(), l[0], l.t()):
        with pytest.raises(ValueError):
            sp.spear_sample(bad, noise)
    for bad in (noise[:2], noise[:, :49], noise.t()):
        with pytest.raises(ValueError):
            sp.spear_sample(l, bad)
    with pytest.raises(TypeError):
        sp.spear_sample(l, noise.half())
    for name, good in (("temperature", torch.ones(3, device=DEV)), ("top_p", torch.ones(3, device=DEV)),
                       ("min_p", torch.ones(3, device=DEV)), ("top_k", torch.ones(3, dtype=torch.int32, device=DEV))):
        with pytest.raises(TypeError):
            sp.spear_sample(l, noise, **{name: good.double()})
        with pytest.raises(ValueError):
            sp.spear_sample(l, noise, **{name: good[:2]})
        with pytest.raises(ValueError):
            sp.spear_sample(l, noise, **{name: good.cpu()})
    with pytest.raises(TypeError):
        sp.spear_sample(l, noise, rows=torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        sp.spear_sample(l, noise, rows=torch.zeros(2, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        sp.spear_sample(l, noise, probs=torch.zeros(3, 49, device=DEV))
    with pytest.raises(ValueError):
        sp.spear_sample(l, noise, tokens=torch.zeros(4, dtype=torch.int32, device=DEV))
    with pytest.raises(sp.SpearError, match="NULL"):
        sp.spear_sample(l, tokens=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(sp.SpearError, match="WORKSPACE"):
        sp.spear_sample(l, noise, workspace=torch.zeros(1 << 20, dtype=torch.uint8, device=DEV))
    with pytest.raises(sp.SpearError, match="UNSUPPORTED"):
        sp.spear_sample(torch.zeros(1, (1 << 22) + 1, dtype=torch.float16, device=DEV), probs=True)
    tokens, probs = sp.spear_sample(l[:0], noise[:0], probs=True)
    assert tokens.shape == (0,) and probs.shape == (0, 50)
    none = sp.spear_sample(l[:0], noise[:2], rows=torch.zeros(2, dtype=torch.int32, device=DEV), probs=True)
    assert none[0].tolist() == [-1, -1] and not none[1].any()
