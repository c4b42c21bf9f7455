"""Adapters of many requests on the GPU against the oracle in 64 bits.

Tolerance: the oracle's slack (its sums' roundings) and the one rounding of Y to fp16,
half a step: 2^-11 of the result, or 2^-25 below the normal numbers.  The slack itself
moves the value that is rounded, so it counts once more beside that step.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import spear_step as ref
import w4_gemm_gated_amd as sp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-adapter] {msg}", flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def batch(rng, lens, adapters, bare=0.2, rows=None):
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    of = np.where(rng.random(len(lens)) < bare, -1, rng.integers(0, adapters, len(lens))).astype(np.int32)
    return cu, of, int(cu[-1]) if rows is None else rows


def tensors(rng, rows, K, N, rank, adapters):
    X = rng.normal(size=(rows, K)).astype(np.float16)
    if K >= 64:
        X[:, rng.integers(0, K, 1 + K // 100)] *= np.float16(20)
    A = (rng.normal(size=(adapters, rank, K)) * K ** -0.5).astype(np.float16)
    B = (rng.normal(size=(adapters, N, rank)) * rank ** -0.5).astype(np.float16)
    return X, A, B, rng.normal(size=(rows, N)).astype(np.float16)


def compare(got, want, slack, Y, cu, of, adapters):
    got = got.astype(np.float64)
    tol = slack * (1 + 2.0 ** -11) + np.abs(want) * 2.0 ** -11 + 2.0 ** -25
    off = np.abs(got - want)
    assert (off <= tol).all(), float((off / tol).max())
    for b, a in enumerate(of):
        if not 0 <= a < adapters:
            assert np.array_equal(got[cu[b]:cu[b + 1]], Y[cu[b]:cu[b + 1]].astype(np.float64))
    assert np.array_equal(got[cu[-1]:], Y[cu[-1]:].astype(np.float64))


def check(rng, lens, K, N, rank, adapters, bare=0.2, scale=True, rows=None):
    cu, of, rows = batch(rng, lens, adapters, bare, rows)
    X, A, B, Y = tensors(rng, rows, K, N, rank, adapters)
    s = rng.normal(size=adapters).astype(np.float32) if scale else None
    plan = sp.spear_adapter_plan(dev(cu), dev(of), adapters, rows)
    got = sp.spear_adapter_add(dev(Y), dev(X), dev(A), dev(B), plan, None if s is None else dev(s))
    torch.cuda.synchronize()
    want, slack = ref.adapter_add(Y, X, A, B, cu, of, s)
    compare(got.cpu().numpy(), want, slack, Y, cu, of, adapters)


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128, 136, 256])
@pytest.mark.parametrize("lens", [[1], [1] * 37, [17, 1, 0, 1, 130, 1, 64]])
def test_ranks(rank, lens):
    note(f"rank {rank} lens {lens[:8]}")
    rng = np.random.default_rng(rank)
    check(rng, lens, 640, 320, rank, 5)


@pytest.mark.parametrize("K,N", [(8, 1), (8, 64), (16, 65), (40, 1000), (136, 15), (504, 16), (520, 17), (1032, 257),
                                 (2048, 2048), (4104, 511), (14336, 256)])
@pytest.mark.parametrize("lens", [[1, 1, 1], [70, 5, 33]])
def test_shapes(K, N, lens):
    note(f"K {K} N {N} lens {lens}")
    rng = np.random.default_rng(K + N)
    check(rng, lens, K, N, 16, 3, scale=False)
    check(rng, lens, K, N, 48, 2, bare=0.0)


@pytest.mark.parametrize("lens,adapters", [([1] * 200, 200), ([1] * 200, 1), ([1] * 1500, 7), ([3] * 50 + [200, 1], 4096),
                                           ([64, 64, 64], 1), ([65, 63, 1], 2), ([0, 0, 0], 2), ([1025], 1),
                                           ([0, 5] * 700, 3)])
def test_batches(lens, adapters):
    note(f"{len(lens)} sequences, {adapters} adapters")
    check(np.random.default_rng(len(lens)), lens, 64, 72, 8, adapters, rows=sum(lens) + 3)


def test_all_or_none_have_adapters():
    note("all, none")
    rng = np.random.default_rng(2)
    check(rng, [1, 9, 20], 128, 96, 16, 3, bare=1.0)
    check(rng, [1, 9, 20], 128, 96, 16, 3, bare=0.0, rows=40)
    cu, _, rows = batch(rng, [2, 3], 2)
    X, A, B, Y = tensors(rng, rows, 64, 64, 8, 2)
    for of in ([2, -7], [2**31 - 1, -2**31]):           # indices of no adapter
        plan = sp.spear_adapter_plan(dev(cu), dev(np.array(of, np.int32)), 2, rows)
        assert np.array_equal(sp.spear_adapter_add(dev(Y), dev(X), dev(A), dev(B), plan).cpu().numpy(), Y)


def test_offsets_that_do_not_rise_do_nothing():
    note("offsets that do not rise")
    rng = np.random.default_rng(3)
    X, A, B, Y = tensors(rng, 20, 64, 64, 8, 2)
    for cu in ([0, 9, 4, 12], [-3, 2, 4, 6], [0, 5, 9, 21], [0, 2**31 - 1, 3, 4]):
        plan = sp.spear_adapter_plan(dev(np.array(cu, np.int32)), dev(np.array([0, 1, 0], np.int32)), 2, 20)
        assert np.array_equal(sp.spear_adapter_add(dev(Y), dev(X), dev(A), dev(B), plan).cpu().numpy(), Y)


def test_parts_of_joint_tensors():
    """Y and X as parts of wider tensors, at odd places; what lies beside them stays."""
    note("strides")
    rng = np.random.default_rng(4)
    cu, of, rows = batch(rng, [1, 40, 7], 3, 0.0)
    for K, N, xw, yw, y0 in ((256, 96, 400, 300, 8), (256, 96, 400, 301, 3), (64, 33, 64, 33, 0), (64, 128, 72, 136, 1)):
        X, A, B, Y = tensors(rng, rows, K, N, 16, 3)
        wide, x = torch.full((rows, yw), 7.0, dtype=torch.float16, device=DEV), torch.zeros(rows, xw, dtype=torch.float16, device=DEV)
        wide[:, y0:y0 + N] = dev(Y)
        x[:, :K] = dev(X)
        plan = sp.spear_adapter_plan(dev(cu), dev(of), 3, rows)
        sp.spear_adapter_add(wide[:, y0:y0 + N], x[:, :K], dev(A), dev(B), plan)
        got = wide.cpu().numpy()
        want, slack = ref.adapter_add(Y, X, A, B, cu, of)
        compare(got[:, y0:y0 + N], want, slack, Y, cu, of, 3)
        got[:, y0:y0 + N] = 7
        assert (got == 7).all()


def test_magnitudes():
    """Rows far larger and far smaller than fp16 holds in between (H up to 2^40 and
    down to 2^-40), and a row of zeros."""
    note("magnitudes")
    rng = np.random.default_rng(5)
    cu, of, rows = batch(rng, [1, 1, 1, 20], 2, 0.0)
    X, A, B, Y = tensors(rng, rows, 512, 64, 16, 2)
    X = np.clip(X, -4, 4)
    X[0] *= np.float16(2.0 ** 12)
    X[1] = np.float16(2.0 ** -20) * np.sign(X[1])
    X[2] = 0
    A = (A.astype(np.float32) * 2.0 ** 12).astype(np.float16)
    s = np.array([2.0 ** -20, 2.0 ** -24], np.float32)
    plan = sp.spear_adapter_plan(dev(cu), dev(of), 2, rows)
    got = sp.spear_adapter_add(dev(Y), dev(X), dev(A), dev(B), plan, dev(s)).cpu().numpy()
    want, slack = ref.adapter_add(Y, X, A, B, cu, of, s)
    compare(got, want, slack, Y, cu, of, 2)


@pytest.mark.parametrize("rank", [16, 64])
def test_infinities_and_nan_stay_in_their_rows(rank):
    note(f"infinities and NaN, rank {rank}")
    rng = np.random.default_rng(6)
    cu, of, rows = batch(rng, [1, 30, 2, 1], 2, 0.0)
    of[:] = 1
    X, A, B, Y = tensors(rng, rows, 256, 80, rank, 2)
    X[3, 5], X[9, 0], Y[12, 7] = np.inf, np.nan, -np.inf
    A[0, 0, 0], B[0, 0, 0] = np.nan, np.inf          # of an adapter that nobody has
    plan = sp.spear_adapter_plan(dev(cu), dev(of), 2, rows)
    got = sp.spear_adapter_add(dev(Y), dev(X), dev(A), dev(B), plan).cpu().numpy()
    bad = np.zeros(rows, bool)
    bad[[3, 9]] = True
    assert not np.isfinite(got[bad]).any() and np.isnan(got[9]).all()
    assert got[12, 7] == -np.inf
    keep = np.isfinite(Y) & ~bad[:, None]
    with np.errstate(all="ignore"):
        want, slack = ref.adapter_add(Y, X, A, B, cu, of)
    tol = slack * (1 + 2.0 ** -11) + np.abs(want) * 2.0 ** -11 + 2.0 ** -25
    assert (np.abs(got[keep].astype(np.float64) - want[keep]) <= tol[keep]).all()


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 48, 64])
@pytest.mark.parametrize("K,N", [(2048, 1000), (520, 4100)])
def test_rows_that_fall_to_one_adapter(rank, K, N):
    """A decode step with many adapters to choose from, whose requests want one of them
    (tiles of 64, of 17 and of one row), or nearly all of them."""
    note(f"one adapter of many, rank {rank} K {K} N {N}")
    rng = np.random.default_rng(rank + K)
    adapters = 40
    X, A, B, Y = tensors(rng, 100, K, N, rank, adapters)
    scale = rng.normal(size=adapters).astype(np.float32)
    cu = np.arange(101, dtype=np.int32)
    for of in (np.full(100, 7), np.where(np.arange(100) < 81, 7, 3), np.where(np.arange(100) % 5 == 0, -1, np.arange(100) % 40)):
        of = of.astype(np.int32)
        plan = sp.spear_adapter_plan(dev(cu), dev(of), adapters, 100)
        got = sp.spear_adapter_add(dev(Y), dev(X), dev(A), dev(B), plan, dev(scale))
        torch.cuda.synchronize()
        want, slack = ref.adapter_add(Y, X, A, B, cu, of, scale)
        compare(got.cpu().numpy(), want, slack, Y, cu, of, adapters)


@pytest.mark.parametrize("rank", [16, 72, 136])
def test_more_tiles_than_there_are_counters(rank):
    """Nearly as many adapters as a plan holds, so that there can be more tiles than the
    workspace has counters.  Past rank 64 all of K and all ranks are then one workgroup's, 64
    ranks at a time; up to it one launch does both products.  Most tiles are of one or two
    rows, some of 16 and more and one of 64."""
    note(f"many tiles, rank {rank}")
    rng = np.random.default_rng(rank)
    adapters = 4096
    of = np.concatenate([rng.permutation(adapters), np.repeat([5, 9, 4001], [103, 16, 15]), [-1, adapters],
                         rng.integers(0, adapters, 764)]).astype(np.int32)
    rows = len(of)
    cu = np.arange(rows + 1, dtype=np.int32)
    for K, N in ((64, 72), (1096, 17)):
        if K > 64 and rank > 72:
            continue
        X, A, B, Y = tensors(rng, rows, K, N, rank, adapters)
        scale = rng.normal(size=adapters).astype(np.float32)
        plan = sp.spear_adapter_plan(dev(cu), dev(of), adapters, rows)
        got = sp.spear_adapter_add(dev(Y), dev(X), dev(A), dev(B), plan, dev(scale))
        torch.cuda.synchronize()
        want, slack = ref.adapter_add(Y, X, A, B, cu, of, scale)
        compare(got.cpu().numpy(), want, slack, Y, cu, of, adapters)


def test_a_row_does_not_depend_on_its_batch():
    """The same row alone, among others of its adapter, and among other adapters'
    (where K is cut alike)."""
    note("rows alone and in a batch")
    rng = np.random.default_rng(7)
    X, A, B, Y = tensors(rng, 90, 1024, 200, 32, 4)
    one = lambda rows, of: sp.spear_adapter_add(  # noqa: E731
        dev(Y[rows]), dev(X[rows]), dev(A), dev(B),
        sp.spear_adapter_plan(dev(np.arange(len(rows) + 1, dtype=np.int32)), dev(np.array(of, np.int32)), 4, len(rows)))
    rows = list(range(90))
    all_same = one(rows, [2] * 90)
    mixed = one(rows, [i % 4 for i in rows])
    for i in (0, 2, 6, 42, 62):
        alone = one([i], [2])
        assert torch.equal(alone[0], all_same[i])
        if i % 4 == 2:
            assert torch.equal(alone[0], mixed[i])


def test_beside_the_layer_captured():
    """The W4 layer and its requests' adapters as a step runs them, on one workspace,
    eager and replayed from a graph: the counters end at zero, and every replay gives
    the eager result's bits."""
    note("layer and adapters, captured")
    rng = np.random.default_rng(8)
    K, N, r, adapters = 1024, 768, 32, 5
    lens = [1, 1, 90, 1, 3]
    cu, of, rows = batch(rng, lens, adapters, 0.2)
    X, W, EA, EB, w_g = workloads.random_layer(rows, K, N, r, seed=3)
    Wq, s = sp.spear_pack_w4(dev(W))
    layer = (Wq, s, dev(EA), dev(EB), dev(w_g), -0.5)
    _, A, B, _ = tensors(rng, rows, K, N, 16, adapters)
    A, B, x = dev(A), dev(B), dev(X)
    cu_d, of_d = dev(cu), dev(of)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
    plan = sp.spear_adapter_plan(cu_d, of_d, adapters, rows)
    Y = torch.empty(rows, N, dtype=torch.float16, device=DEV)

    def step():
        sp.spear_adapter_plan(cu_d, of_d, adapters, rows, plan=plan)
        sp.spear_w4ec_linear(x, *layer, Y=Y, workspace=ws)
        sp.spear_adapter_add(Y, x, A, B, plan, workspace=ws)

    step()
    torch.cuda.synchronize()
    first = Y.clone()
    base = sp.spear_w4ec_linear(x, *layer, workspace=ws).cpu().numpy()
    want, slack = ref.adapter_add(base, X, A.cpu().numpy(), B.cpu().numpy(), cu, of)
    compare(first.cpu().numpy(), want, slack, base, cu, of, adapters)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        step()
    for i in range(4):
        of2 = np.roll(of, i)
        of_d.copy_(dev(of2))
        x.copy_(dev(np.roll(X, i, 0)))
        step()
        torch.cuda.synchronize()
        eager = Y.clone()
        Y.fill_(3)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, eager)


def test_counters_and_streams():
    note("workspace counters, another stream")
    rng = np.random.default_rng(9)
    cu, of, rows = batch(rng, [1] * 30, 4, 0.0)
    X, A, B, Y = tensors(rng, rows, 4096, 512, 16, 4)
    t = [dev(Y), dev(X), dev(A), dev(B)]
    plan = sp.spear_adapter_plan(dev(cu), dev(of), 4, rows)
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device=DEV)
    want = sp.spear_adapter_add(t[0].clone(), *t[1:], plan, workspace=ws)
    assert not ws[:1 << 20].any()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        again = sp.spear_adapter_add(t[0].clone(), *t[1:], plan)
    stream.synchronize()
    assert torch.equal(again, want)


def test_refusals():
    note("refusals")
    rng = np.random.default_rng(10)
    cu, of, rows = batch(rng, [1, 2], 2)
    X, A, B, Y = (dev(t) for t in tensors(rng, rows, 64, 32, 8, 2))
    plan = sp.spear_adapter_plan(dev(cu), dev(of), 2, rows)
    with pytest.raises(TypeError):
        sp.spear_adapter_plan(dev(cu).long(), dev(of), 2, rows)
    with pytest.raises(ValueError):
        sp.spear_adapter_plan(dev(cu), dev(of[:1]), 2, rows)
    with pytest.raises(ValueError):
        sp.spear_adapter_plan(dev(cu), dev(of), 3, rows, plan=plan)
    with pytest.raises(TypeError):
        sp.spear_adapter_plan(dev(cu), dev(of), 2, rows, plan=plan.data)
    for n in (0, -1):
        with pytest.raises(sp.SpearError, match="SHAPE"):
            sp.spear_adapter_plan(dev(cu), dev(of), n, rows)
    with pytest.raises(sp.SpearError, match="UNSUPPORTED"):
        sp.spear_adapter_plan(dev(cu), dev(of), 4097, rows)
    with pytest.raises(TypeError):
        sp.spear_adapter_add(Y.float(), X, A, B, plan)
    with pytest.raises(TypeError):
        sp.spear_adapter_add(Y, X, A, B, plan.data)
    with pytest.raises(TypeError):
        sp.spear_adapter_add(Y, X, A, B, plan, scale=torch.ones(2, dtype=torch.float16, device=DEV))
    for bad in ((Y[:, :31], X, A, B), (Y, X[:2], A, B), (Y, X, A[:1], B), (Y, X, A, B[:, :, :4]), (Y.t(), X, A, B),
                (Y, X.cpu(), A, B), (Y, X, A.transpose(1, 2), B), (Y, X, A, B.transpose(1, 2)),
                (torch.empty(32, 3, dtype=torch.float16, device=DEV).t(), X, A, B)):
        with pytest.raises(ValueError):
            sp.spear_adapter_add(*bad, plan)
    odd = [torch.zeros(2, 4, 64, dtype=torch.float16, device=DEV), torch.zeros(2, 32, 4, dtype=torch.float16, device=DEV)]
    with pytest.raises(sp.SpearError, match="SHAPE"):
        sp.spear_adapter_add(Y, X, *odd, plan)
    shifted = torch.zeros(rows, 68, dtype=torch.float16, device=DEV)
    with pytest.raises(sp.SpearError, match="MISALIGNED"):
        sp.spear_adapter_add(Y, torch.zeros(rows, 72, dtype=torch.float16, device=DEV)[:, 4:68], A, B, plan)
    with pytest.raises(sp.SpearError, match="SHAPE"):
        sp.spear_adapter_add(Y, shifted[:, :64], A, B, plan)
    with pytest.raises(sp.SpearError, match="WORKSPACE"):
        sp.spear_adapter_add(Y, X, A, B, plan, workspace=torch.zeros(1 << 20, dtype=torch.uint8, device=DEV))
