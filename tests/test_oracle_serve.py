"""Pins of the serving oracle (CPU): facts from outside it."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import spear_serve as ref


def cache_of(rows, page, pages, rng, fill=np.nan):
    """rows [n, heads, dim] laid into random pages: (cache, table row)."""
    n, heads, dim = rows.shape
    cache = np.full((pages, heads, page, dim), fill, dtype=rows.dtype)
    order = rng.permutation(pages)
    table = np.full(pages, -1, dtype=np.int32)
    for i in range(n):
        table[i // page] = order[i // page]
        cache[order[i // page], :, i % page] = rows[i]
    return cache, table


def test_codes_are_the_nearest_and_ties_are_even():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(50, 64)).astype(np.float16)
    codes, s = ref.quantise_kv(x)
    assert s.dtype == np.float32 and codes.dtype == np.int8
    for r in range(50):
        assert s[r] == np.float32(np.abs(x[r]).max()) / np.float32(127)
        for i in range(64):
            exact = Fraction(float(x[r, i])) / Fraction(float(s[r]))
            assert abs(int(codes[r, i]) - exact) <= Fraction(1, 2) + Fraction(1, 2 ** 16)
    tie = np.zeros((1, 64), dtype=np.float16)
    tie[0, :4] = [127, 2.5, 3.5, -2.5]
    codes, s = ref.quantise_kv(tie)
    assert s[0] == 1 and codes[0, :4].tolist() == [127, 2, 4, -2]


def test_special_rows_of_the_quantiser():
    x = np.zeros((4, 64), dtype=np.float16)
    x[1, 3] = np.inf
    x[2, 5] = np.nan
    x[3, 0] = 6e-8
    codes, s = ref.quantise_kv(x)
    assert s[0] == 0 and not codes[0].any()
    assert np.isinf(s[1]) and np.isnan(s[2])
    assert codes[3, 0] == 127 and s[3] > 0
    with np.errstate(all="ignore"):
        assert not np.isfinite(codes[1].astype(np.float32) * s[1]).any()
        assert not np.isfinite(codes[2].astype(np.float32) * s[2]).any()


@pytest.mark.parametrize("page", [16, 32])
def test_attention_closed_forms(page):
    rng = np.random.default_rng(1)
    n, heads, dim = 37, 2, 64
    v = rng.normal(size=(n, heads, dim)).astype(np.float16)
    k = np.zeros_like(v)
    kc, table = cache_of(k, page, 4, rng)
    vc = np.full_like(kc, np.nan)
    for i in range(n):
        vc[table[i // page], :, i % page] = v[i]
    q = rng.normal(size=(3, 4, dim)).astype(np.float16)
    # equal keys: the mean of the visible values
    out, spread, reach = ref.paged_attention(q, kc, vc, table[None], [0, 3], [n], 0.125)
    for i in range(3):
        for h in range(4):
            want = v[: n - 2 + i, h // 2].astype(np.float64).mean(0)
            np.testing.assert_allclose(out[i, h], want, rtol=1e-13)
    assert not reach.any() and (spread >= np.abs(out) - 1e-15).all()
    # one key far above the others: its value
    k[11] = 100 * q[2, 0]
    for i in range(n):
        kc[table[i // page], :, i % page] = k[i]
    out, _, _ = ref.paged_attention(q, kc, vc, table[None], [0, 3], [n], 0.125)
    np.testing.assert_allclose(out[2, 0], v[11, 0].astype(np.float64), rtol=1e-12)


def test_attention_brute_force_and_empty_rows():
    rng = np.random.default_rng(2)
    n, heads, dim = 9, 1, 64
    k, v = (rng.normal(size=(n, heads, dim)).astype(np.float16) for _ in range(2))
    kc, table = cache_of(k, 16, 2, rng)
    vc = np.full_like(kc, np.nan)
    vc[table[0], :, :n] = v.transpose(1, 0, 2)
    q = rng.normal(size=(12, 1, dim)).astype(np.float16)
    out, _, _ = ref.paged_attention(q, kc, vc, table[None], [0, 12], [n], 0.2)
    for i in range(12):
        seen = n - 12 + i + 1
        if seen <= 0:
            assert not out[i].any()
            continue
        z = [math.fsum(float(a) * float(b) for a, b in zip(q[i, 0], k[j, 0])) * 0.2 for j in range(seen)]
        w = [math.exp(x - max(z)) for x in z]
        for d in range(0, dim, 7):
            want = math.fsum(a * float(v[j, 0, d]) for j, a in enumerate(w)) / math.fsum(w)
            assert abs(out[i, 0, d] - want) < 1e-13


def test_attention_over_codes_is_attention_over_what_they_stand_for():
    rng = np.random.default_rng(3)
    x = rng.normal(size=(20, 1, 64)).astype(np.float16)
    codes, s = ref.quantise_kv(x)
    kc, table = cache_of(codes, 16, 3, rng, fill=0)
    sc = np.zeros((3, 1, 16), dtype=np.float32)
    for i in range(20):
        sc[table[i // 16], 0, i % 16] = s[i, 0]
    stood = (codes.astype(np.float64) * s[..., None])
    q = rng.normal(size=(1, 1, 64)).astype(np.float16)
    out, _, _ = ref.paged_attention(q, kc, kc, table[None], [0, 1], [20], 0.3, sc, sc)
    z = stood[:, 0] @ q[0, 0].astype(np.float64) * 0.3
    p = np.exp(z - z.max())
    np.testing.assert_allclose(out[0, 0], p @ stood[:, 0] / p.sum(), rtol=1e-12)


def test_verify_hand_worked():
    f = np.float32
    target = np.array([[[.5, .5, 0, 0], [.25, .25, .5, 0], [0, 0, 0, 1]]], dtype=f)
    draft = np.array([[[.5, .25, .25, 0], [.5, .25, .25, 0]]], dtype=f)
    noise = np.ones((1, 4), dtype=f)
    # both kept: 0.9 * 0.5 < 0.5, then 0.4 * 0.5 < 0.25; next from the last row
    a, t = ref.verify_draft(target, draft, np.array([[0, 0]]), np.array([[.9, .4]], dtype=f), noise)
    assert a.tolist() == [2] and t.tolist() == [[0, 0, 3]]
    # the second refused: residual max(p - q, 0) = [0, 0, .25, 0]
    a, t = ref.verify_draft(target, draft, np.array([[0, 0]]), np.array([[.9, .6]], dtype=f), noise)
    assert a.tolist() == [1] and t.tolist() == [[0, 2, -1]]
    # equality refuses; a zero residual draws from the target's own row
    a, t = ref.verify_draft(target, target[:, :2], np.array([[2, 0]]), np.array([[0., 0.]], dtype=f),
                            np.array([[4, 1, 1, 1]], dtype=f))
    assert a.tolist() == [0] and t.tolist() == [[1, -1, -1]]
    # copied drafts; lengths; a token outside the vocabulary
    a, t = ref.verify_draft(target, None, np.array([[1, 2]]), np.array([[.4, .4]], dtype=f), noise, [1])
    assert a.tolist() == [1] and t.tolist() == [[1, 2, -1]]
    a, t = ref.verify_draft(target, None, np.array([[7, 2]]), np.array([[.4, .4]], dtype=f), noise)
    assert a.tolist() == [0] and t.tolist() == [[0, -1, -1]]


def test_verified_tokens_follow_the_target():
    """First token's distribution over many trials: within five standard errors
    of the target's, whatever the draft proposes."""
    rng = np.random.default_rng(5)
    V, N = 6, 20000
    p = rng.dirichlet(np.ones(V), size=2).astype(np.float32)
    q = rng.dirichlet(np.ones(V)).astype(np.float32)
    drafted = rng.choice(V, size=(N, 1), p=q / q.sum()).astype(np.int32)
    target = np.broadcast_to(p, (N, 2, V))
    draft = np.broadcast_to(q, (N, 1, V))
    _, t = ref.verify_draft(target, draft, drafted, rng.random((N, 1), dtype=np.float32),
                            rng.exponential(size=(N, V)).astype(np.float32))
    got = np.bincount(t[:, 0], minlength=V) / N
    assert (np.abs(got - p[0]) < 5 * np.sqrt(p[0] * (1 - p[0]) / N) + 1e-9).all()
