"""Verification of drafted tokens on the GPU against the oracle: whole numbers,
every one equal."""
import numpy as np
import pytest
import torch

from oracle import spear_serve as ref
import w4_gemm_gated_amd as sp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-verify] {msg}", flush=True)


def softmax(z):
    e = np.exp(z - z.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def case(rng, B, K, V, given=True):
    z = rng.normal(0, 2.5, size=(B, K + 1, V))
    target = softmax(z)
    draft = softmax(z[:, :K] + rng.normal(0, 0.6, size=(B, K, V))) if given else None
    base = draft if given else target[:, :K]
    drafted = (base / rng.exponential(size=(B, K, V))).argmax(-1).astype(np.int32) if K else \
        np.zeros((B, 0), dtype=np.int32)
    u = rng.random(size=(B, K), dtype=np.float32)
    noise = rng.exponential(size=(B, V)).astype(np.float32)
    return target, draft, drafted, u, noise


def run(target, draft, drafted, u, noise, n=None):
    d = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    n = None if n is None else np.asarray(n, dtype=np.int32)
    a, t = sp.spear_verify_draft(d(target), d(draft), d(drafted), d(u), d(noise), d(n))
    torch.cuda.synchronize()
    return a.cpu().numpy(), t.cpu().numpy()


@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("B,K,V", [(1, 0, 1), (1, 1, 2), (3, 4, 63), (5, 3, 4096), (4, 2, 4097), (2, 5, 32000),
                                   (7, 8, 50257), (1, 70, 300), (300, 1, 130), (1, 3, 131071)])
def test_against_the_oracle(B, K, V, given):
    note(f"B {B} K {K} V {V} given {given}")
    rng = np.random.default_rng(B * 7 + K + V)
    c = case(rng, B, K, V, given)
    n = rng.integers(-1, K + 2, size=B)          # clamped to [0, K]
    for lens in (None, n):
        got, want = run(*c, lens), ref.verify_draft(*c, lens)
        assert np.array_equal(got[0], want[0])
        assert np.array_equal(got[1], want[1])


def test_special_values():
    note("ties, zeros, infinities, NaN")
    V = 9000
    rng = np.random.default_rng(3)
    target, draft, drafted, u, noise = case(rng, 8, 2, V)
    noise[0] = 1.0
    target[0] = 1.0 / V                          # every score equal: the lowest index
    draft[0] = 0.0
    u[0] = 0.5                                   # u * 0 < p: kept
    target[1] = draft[1, 0]                      # residual zero: the target's own row
    u[1, 0] = 1.0
    target[2] = 0.0                              # nothing to draw: -1
    noise[3, :] = np.inf                         # every score zero: the lowest index of positive weight
    noise[4, 4321] = 0.0                         # an infinite score wins
    target[4, :, 4321] = 0.5
    draft[4, :, 4321] = 0.1
    target[5, :, ::3] = np.nan                   # not drawn, not kept
    drafted[6] = [V, 0]                          # outside the vocabulary
    drafted[7] = [-5, 0]
    got, want = run(target, draft, drafted, u, noise), ref.verify_draft(target, draft, drafted, u, noise)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert got[1][2, 0] == -1 and got[0][6] == 0 and got[0][7] == 0


def test_strides_repeat_and_counters():
    """Rows of larger tensors; a second call on the same workspace; the
    workspace's counters back at zero."""
    note("strides")
    rng = np.random.default_rng(4)
    target, draft, drafted, u, noise = case(rng, 6, 3, 20001)
    big = torch.zeros(6, 5, 20011, device=DEV)
    big[:, 1:, 7:20008] = torch.from_numpy(target).to(DEV)
    small = torch.zeros(3, 6, 20001, device=DEV)
    small.copy_(torch.from_numpy(draft).transpose(0, 1))
    ws = torch.zeros(2 << 20, dtype=torch.uint8, device=DEV)
    d = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    want = ref.verify_draft(target, draft, drafted, u, noise)
    for _ in range(2):
        a, t = sp.spear_verify_draft(big[:, 1:, 7:20008], small.transpose(0, 1), d(drafted), d(u), d(noise),
                                     workspace=ws)
        assert np.array_equal(a.cpu().numpy(), want[0]) and np.array_equal(t.cpu().numpy(), want[1])
        assert not ws[:1 << 20].any()


def test_graph_replays():
    note("captured verification")
    rng = np.random.default_rng(6)
    first, second = case(rng, 4, 3, 33000), case(rng, 4, 3, 33000)
    t = [torch.from_numpy(x).to(DEV) for x in first]
    ws = torch.zeros(2 << 20, dtype=torch.uint8, device=DEV)
    out = (torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(4, 4, dtype=torch.int32, device=DEV))
    call = lambda: sp.spear_verify_draft(*t, accepted=out[0], tokens=out[1], workspace=ws)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for c in (second, first, second):
        for x, y in zip(t, c):
            x.copy_(torch.from_numpy(y))
        g.replay()
        torch.cuda.synchronize()
        want = ref.verify_draft(*c)
        assert np.array_equal(out[0].cpu().numpy(), want[0]) and np.array_equal(out[1].cpu().numpy(), want[1])


def test_refusals():
    rng = np.random.default_rng(5)
    c = [torch.from_numpy(x).to(DEV) for x in case(rng, 2, 3, 100)]
    target, draft, drafted, u, noise = c
    with pytest.raises(TypeError):
        sp.spear_verify_draft(target.half(), draft, drafted, u, noise)
    with pytest.raises(ValueError):
        sp.spear_verify_draft(target, draft[:, :2], drafted, u, noise)
    with pytest.raises(ValueError):
        sp.spear_verify_draft(target, draft, drafted[:1], u, noise)
    with pytest.raises(ValueError):
        sp.spear_verify_draft(target.transpose(1, 2), draft, drafted, u, noise)
    with pytest.raises(TypeError):
        sp.spear_verify_draft(target, draft, drafted.long(), u, noise)
    with pytest.raises(sp.SpearError, match="WORKSPACE"):
        big = [torch.zeros(1, 1, 9000, device=DEV), None, drafted[:1, :0].contiguous(), u[:1, :0].contiguous(),
               torch.ones(1, 9000, device=DEV)]
        sp.spear_verify_draft(*big, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    a, t = sp.spear_verify_draft(target[:0], draft[:0], drafted[:0], u[:0], noise[:0])
    assert a.shape == (0,) and t.shape == (0, 4)


@pytest.mark.parametrize("lost", [False, True])
@pytest.mark.parametrize("V", [5, 63, 4097, 9001, 33002])
def test_draft_entries_below_zero_count_where_they_are(V, lost):
    """A draft row that is no distribution (entries below zero, as a clipped one may
    hold) still draws by p - q, and only from the vocabulary, also where the target
    is NaN."""
    note(f"draft entries below zero, V {V}, target NaN there: {lost}")
    rng = np.random.default_rng(V)
    target, draft, drafted, u, noise = case(rng, 6, 2, V)
    u[:] = 1.0                                    # (nothing is kept)
    draft += np.float32(1e-3) + target[:, :2]
    for b in range(6):
        draft[b, :, V - 1 - b % 5] = -0.5         # the largest residual, near the end
        draft[b, :, V // 2] = -0.01
        if lost:
            target[b, :, V - 1 - b % 5] = np.nan
    drafted[:] = 0
    got, want = run(target, draft, drafted, u, noise), ref.verify_draft(target, draft, drafted, u, noise)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert (got[1] < V).all()
