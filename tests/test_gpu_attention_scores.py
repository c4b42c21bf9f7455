"""Attention whose scores lie far outside the usual range, where a score's neighbours
in fp32 are whole numbers apart."""
import numpy as np
import pytest
import torch

from test_gpu_paged_attention import make, note, run

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

BATCHES = [([1], [200]), ([1, 3], [3000, 40]), ([40], [3000]), ([50], [100]), ([129], [400])]


def keys(c, int8, values):
    """Every cached key's first channels (those beyond: zero), scales one."""
    held = np.isfinite(c["k_scale"] if int8 else c["k"][..., 0])
    c["k"][held] = 0
    for d, x in enumerate(values):
        c["k"][..., d][held] = x
    if int8:
        c["k_scale"][held] = 1
        c["v_scale"][held] = 1


def worst(c, got, weights):
    """Largest error over its bound; weights(positions) are the exact ones.  They or
    their sums lose nothing here (powers of two), so sums in fp32 and a result in fp16
    are all that rounds."""
    most = 0.0
    for b, (n, length) in enumerate(zip(np.diff(c["cu"]), c["lens"])):
        v = np.stack([c["v"][c["table"][b, i // 16], 0, i % 16].astype(np.float64) for i in range(length)])
        for i in range(n):
            w = weights(np.arange(length - n + i + 1))
            w = w / w.sum()
            want, spread = w @ v[:len(w)], w @ np.abs(v[:len(w)])
            tol = 2.0 ** -11 * np.abs(want) + 2.0 ** -17 * spread + 2.0 ** -24
            d = np.abs(got[c["cu"][b] + i].astype(np.float64) - want) / tol
            most = max(most, float(np.nan_to_num(d, nan=np.inf).max()))
    return most


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("score", [1e9, 1e31])
@pytest.mark.parametrize("q_lens,lens", BATCHES)
def test_equal_large_scores_give_the_mean(int8, dim, score, q_lens, lens):
    note(f"scores of {score:g} int8 {int8} dim {dim} q {q_lens} kv {lens}")
    c = make(np.random.default_rng(3), q_lens, lens, 1, 4, dim, 16, int8)
    c["q"][:] = 0
    c["q"][:, :, 0] = 10.5
    keys(c, int8, [3])
    got = run(c, scale=score / 31.5)
    assert worst(c, got, lambda at: np.ones(len(at))) <= 1


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,lens", BATCHES)
def test_a_step_of_sixteen_at_large_scores(int8, dim, q_lens, lens):
    """Scores (in powers of two) of 1500 * 2^17 for the first 128 keys and 16 more, the
    next number in fp32, for the others: these weigh 2^16 times as much."""
    note(f"neighbouring scores int8 {int8} dim {dim} q {q_lens} kv {lens}")
    c = make(np.random.default_rng(4), q_lens, lens, 1, 4, dim, 16, int8)
    c["q"][:] = 0
    c["q"][:, :, 0] = 12 if int8 else 1
    c["q"][:, :, 1] = 2.0 ** -13
    keys(c, int8, [125 if int8 else 1500])
    for b, length in enumerate(lens):
        for i in range(128, length):
            c["k"][c["table"][b, i // 16], :, i % 16, 1] = 1
    scale = np.float32(2.0 ** 17) / np.float32(1.44269504088896341)
    assert scale * np.float32(1.44269504088896341) == 2.0 ** 17
    got = run(c, scale=float(scale))
    assert worst(c, got, lambda at: np.where(at < 128, 1.0, 2.0 ** 16)) <= 1


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("score", [-1e9, -1e31, -1e33])
@pytest.mark.parametrize("q_lens,lens", BATCHES)
def test_equal_scores_far_below_zero_give_the_mean(int8, dim, score, q_lens, lens):
    note(f"scores of {score:g} int8 {int8} dim {dim} q {q_lens} kv {lens}")
    c = make(np.random.default_rng(5), q_lens, lens, 1, 4, dim, 16, int8)
    c["q"][:] = 0
    c["q"][:, :, 0] = 1050
    keys(c, int8, [-3])
    got = run(c, scale=-score / 3150)
    assert worst(c, got, lambda at: np.ones(len(at))) <= 1


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("score", [1.0, 2.4e8, 5e8])
@pytest.mark.parametrize("power", [-36, -30, -24, -18, -10, 9])
@pytest.mark.parametrize("q_lens,lens", BATCHES[1:4])
def test_scales_of_values_beside_large_scores(dim, score, power, q_lens, lens):
    """The exponent of the values' scales cannot be held beside a large score; the
    result is the values' mean all the same (or zero where fp16 holds no such value)."""
    note(f"scores of {score:g}, scales of 2^{power}, dim {dim} q {q_lens} kv {lens}")
    c = make(np.random.default_rng(6), q_lens, lens, 1, 4, dim, 16, True)
    c["q"][:] = 0
    c["q"][:, :, 0] = 10.5
    keys(c, True, [3])
    c["v_scale"][np.isfinite(c["v_scale"])] = 2.0 ** power
    got = run(c, scale=score / 31.5)
    v = c["v"]
    c["v"] = v.astype(np.float64) * 2.0 ** power
    assert worst(c, got, lambda at: np.ones(len(at))) <= 1
