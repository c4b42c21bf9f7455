"""Attention over the paged cache on the GPU against the float64 oracle.

Tolerance, per element, from the arithmetic the operator states.  With
A = sum_j p_j |v_j| (the weighted mean of |v|):
  - the weights are rounded to fp16 (2^-11 relative each, the sum of weights is
    not): 2^-11 A, and below fp16's normal range an absolute 2^-25 against a
    largest weight of at least 2^6, at most 2^-29 max|v| per key for codes whose
    common scale is up to four times a value's own;
  - scores in fp32: head_dim products and a scale or two, 2^-17 of the sum of
    |q_d k_d| scale, and the exponential's argument and result; each moves a
    weight by that much relative, numerator and sum: 2 (2^-17 reach + 2^-18) A;
  - the result is rounded to fp16: 2^-11 |out|, 2^-24 below the normal range.
"""
import math

import numpy as np
import pytest
import torch

from oracle import spear_serve as ref
import w4_gemm_gated_amd as sp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-attention] {msg}", flush=True)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def make(rng, q_lens, kv_lens, kv_heads, group, dim, page, int8, sharp=1.3, fill=None):
    """Inputs on the host: random pages; what no sequence holds is `fill` (NaN and
    infinities in turn when None)."""
    need = [-(-n // page) for n in kv_lens]
    pages = sum(need) + 2
    order = rng.permutation(pages)
    table = np.full((len(kv_lens), max(need + [1]) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pages, kv_heads, page, dim)
    held = np.zeros((pages, page), dtype=bool)
    for b, n in enumerate(kv_lens):
        for i in range(n):
            held[table[b, i // page], i % page] = True
    held = np.broadcast_to(held[:, None, :], shape[:3])
    junk = np.where(np.arange(page) % 2, np.nan, np.inf)
    c = {}
    for n in ("k", "v"):
        if int8:
            c[n] = np.clip(np.rint(rng.normal(0, 40, size=shape)), -127, 127).astype(np.int8)
            s = (0.02 * np.exp(0.5 * rng.normal(size=shape[:3]))).astype(np.float32)
            c[n + "_scale"] = np.where(held, s, junk if fill is None else fill).astype(np.float32)
        else:
            x = rng.normal(size=shape)
            c[n] = np.where(held[..., None], x, junk[:, None] if fill is None else fill).astype(np.float16)
            c[n + "_scale"] = None
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    c["q"] = rng.normal(0, sharp, size=(int(cu[-1]), kv_heads * group, dim)).astype(np.float16)
    c["table"], c["cu"], c["lens"] = table, cu, np.asarray(kv_lens, dtype=np.int32)
    c["max_q"] = max(list(q_lens) + [1])
    return c


def run(c, scale=None, joint=False, **more):
    q = dev(c["q"])
    if joint:      # the queries as a part of a wider projection, heads not adjacent
        total, heads, dim = q.shape
        wide = torch.full((total, heads, dim + 8), float("nan"), dtype=torch.float16, device=DEV)
        wide[:, :, :dim] = q
        q = wide[:, :, :dim]
    args = dict(k_scale=dev(c["k_scale"]), v_scale=dev(c["v_scale"]), scale=scale)
    args.update(more)
    out = sp.spear_paged_attention(q, dev(c["k"]), dev(c["v"]), dev(c["table"]), dev(c["cu"]), dev(c["lens"]),
                                   args.pop("max_q", c["max_q"]), **args)
    torch.cuda.synchronize()
    return out.cpu().numpy()


def check(c, got, scale=None):
    scale = 1 / math.sqrt(c["q"].shape[2]) if scale is None else scale
    want, spread, reach = ref.paged_attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["lens"], scale,
                                              c["k_scale"], c["v_scale"])
    ok = np.isfinite(want)
    big = 0.0
    for b, n in enumerate(c["lens"]):
        if n and c["cu"][b + 1] > c["cu"][b]:
            v = np.abs(ref.cached(c["v"], c["v_scale"], c["table"][b], int(n)))
            big = max(big, float(v[np.isfinite(v)].max(initial=0.0)) * int(n))
    tol = (2.0 ** -11 * np.abs(want) + (2.0 ** -11 + 2 * (2.0 ** -17 * np.abs(reach)[..., None] + 2.0 ** -18)) * spread
           + 2.0 ** -29 * big + 2.0 ** -24)
    d = np.abs(got.astype(np.float64) - want)
    assert np.array_equal(np.isfinite(got), ok)
    worst = float((d[ok] / tol[ok]).max(initial=0.0))
    rel = float(np.linalg.norm(d[ok]) / max(np.linalg.norm(want[ok]), 1e-300))
    note(f"  worst error {worst:.2f} of the bound, relative L2 {rel:.1e}")
    assert (d[ok] <= tol[ok]).all()
    return want


SHAPES = [(1, 1, 128, 16), (8, 4, 128, 32), (2, 8, 64, 16), (4, 1, 64, 64), (2, 3, 128, 16), (1, 16, 128, 1024),
          (3, 5, 64, 32)]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kv_heads,group,dim,page", SHAPES)
def test_decode(int8, kv_heads, group, dim, page):
    """One new token for each sequence, at every edge of a tile and a page."""
    lens = [1, 0, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 255, 256, 257, 700]
    note(f"decode int8 {int8} kv_heads {kv_heads} group {group} dim {dim} page {page}")
    c = make(np.random.default_rng(dim + page + group), [1] * len(lens), lens, kv_heads, group, dim, page, int8)
    got = run(c, joint=True)
    check(c, got)
    assert not got[1].any()                       # nothing cached: zeros


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("kv_heads,group,dim,page", SHAPES)
def test_ragged_chunks(int8, kv_heads, group, dim, page):
    """No new token, one, a few drafted ones, prompts' chunks; also more new
    tokens than cached ones, whose first see nothing."""
    q_lens = [3, 0, 1, 17, 5, 40, 33, 2, 130]
    lens = [3, 9, 300, 17, 64, 20, 260, 0, 135]
    note(f"chunks int8 {int8} kv_heads {kv_heads} group {group} dim {dim} page {page}")
    c = make(np.random.default_rng(7 + dim + page), q_lens, lens, kv_heads, group, dim, page, int8)
    got = run(c)
    check(c, got)
    empty = c["cu"][5]
    assert not got[empty:empty + 20].any() and got[empty + 20].any()
    for hint in (1, 1000):                        # the hint changes the speed, not what is computed
        check(c, run(c, max_q=hint))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("q_lens,lens,kv_heads,group,dim", [
    ([1], [9001], 2, 4, 128), ([1, 1], [5000, 37], 1, 1, 64), ([6], [7003], 2, 5, 128), ([1] * 70, [1500] * 3 + [40] * 67, 1, 2, 64),
    ([65, 1], [4100, 6000], 1, 2, 128)])
def test_long_sequences_are_split(int8, q_lens, lens, kv_heads, group, dim):
    note(f"split int8 {int8} q {q_lens[:4]} kv {lens[:4]}")
    c = make(np.random.default_rng(11), q_lens, lens, kv_heads, group, dim, 16, int8)
    got = run(c)
    check(c, got)
    assert np.array_equal(got.view(np.uint16), run(c).view(np.uint16))     # the same bits each time


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_masked_infinities_and_nan(int8, dim):
    """Infinities and NaN in a sequence's later tokens reach the tokens that see
    them and no earlier one."""
    note(f"masked values int8 {int8} dim {dim}")
    rng = np.random.default_rng(5)
    q_lens, lens = [4, 20, 70, 3], [40, 20, 200, 2000]
    c = make(rng, q_lens, lens, 2, 3, dim, 16, int8)

    def spoil(name, b, i, value):
        p, o = c["table"][b, i // 16], i % 16
        if int8:
            c[name + "_scale"][p, :, o] = value
        else:
            c[name][p, :, o, 3] = value
    spoil("v", 0, 38, np.inf)
    spoil("k", 0, 39, np.nan)
    spoil("v", 1, 10, np.nan)
    spoil("v", 2, 150, np.inf)
    spoil("v", 2, 190, -np.inf)
    spoil("k", 3, 1998, np.nan)
    spoil("v", 3, 1999, np.nan)
    got = run(c)
    scale = 1 / math.sqrt(dim)
    with np.errstate(all="ignore"):
        want, _, _ = ref.paged_attention(c["q"], c["k"], c["v"], c["table"], c["cu"], c["lens"], scale, c["k_scale"],
                                         c["v_scale"])
    # which elements are finite follows from the definition
    assert np.array_equal(np.isfinite(got), np.isfinite(want))
    assert np.isfinite(want[0]).all() and not np.isfinite(want[3]).all()
    ok = np.isfinite(want)
    # the spoiled channel apart, the rows are ordinary: relative L2 of fp16 weights and results
    rel = np.linalg.norm(got[ok] - want[ok]) / np.linalg.norm(want[ok])
    note(f"  relative L2 of the finite elements {rel:.1e}")
    assert rel <= 2.0 ** -10


@pytest.mark.parametrize("int8", [False, True])
def test_extreme_scores_and_values(int8):
    """Scores far apart, one dominating key, values near fp16's ends, zeros."""
    note(f"extreme values int8 {int8}")
    rng = np.random.default_rng(9)
    c = make(rng, [1, 1, 2, 1], [100, 500, 64, 90], 1, 4, 128, 16, int8, sharp=12.0)
    p = c["table"][1, 3]
    if int8:
        c["v_scale"][c["table"][0]] *= np.float32(1e4)
        c["v_scale"][p] = np.float32(1e-6)
        c["v_scale"][c["table"][3, 0]] = 0
        c["k_scale"][c["table"][2, 1]] = 0
    else:
        c["v"][c["table"][0, 0]] = (60000 * np.sign(rng.normal(size=c["v"][0].shape))).astype(np.float16)
        c["v"][p] = np.float16(6e-8)
        c["v"][c["table"][3, 0]] = 0
        c["k"][c["table"][2, 1]] = 0
    check(c, run(c))
    check(c, run(c, scale=2.0), scale=2.0)
    check(c, run(c, scale=0.0), scale=0.0)
    check(c, run(c, scale=-0.1), scale=-0.1)


def test_minus_infinity_scores_give_zeros():
    note("every visible score -inf")
    c = make(np.random.default_rng(10), [1, 1], [20, 20], 1, 1, 64, 16, False)
    c["q"][0] = 0
    c["q"][0, 0, 0] = 1
    c["k"][c["table"][0, :2]] = 0
    c["k"][c["table"][0, :2], :, :, 0] = -np.inf
    got = run(c)
    assert not got[0].any()
    assert np.isfinite(got[1]).all()


def test_offsets_past_32_bits():
    heads, dim, page = 8, 128, 64
    pages = (1 << 31) // (heads * dim * page) + 8
    for dtype in (torch.float16, torch.int8):
        note(f"large cache {dtype}")
        c = make(np.random.default_rng(12), [1, 2], [200, 130], heads, 2, dim, page, dtype is torch.int8)
        n = c["k"].shape[0]
        big = {}
        for name in ("k", "v"):
            big[name] = torch.empty(pages, heads, page, dim, dtype=dtype, device=DEV)
            big[name][pages - n:] = dev(c[name])
            s = c[name + "_scale"]
            big[name + "_scale"] = None
            if s is not None:
                big[name + "_scale"] = torch.empty(pages, heads, page, device=DEV)
                big[name + "_scale"][pages - n:] = dev(s)
        table = np.where(c["table"] >= 0, c["table"] + pages - n, -1).astype(np.int32)
        out = sp.spear_paged_attention(dev(c["q"]), big["k"], big["v"], dev(table), dev(c["cu"]), dev(c["lens"]), 2,
                                       k_scale=big["k_scale"], v_scale=big["v_scale"])
        check(c, out.cpu().numpy())
        del big


def test_lengths_outside_the_tensors_stay_inside():
    """Lengths, offsets and pages that break the contract are clamped: the call
    ends, and sequences that keep it are right."""
    note("clamped lengths")
    c = make(np.random.default_rng(13), [1, 1, 2], [40, 30, 50], 2, 2, 64, 16, False, fill=0.0)
    want = run(c)
    bad = dict(c)
    bad["lens"] = np.array([40, 10 ** 6, -7], dtype=np.int32)
    bad["table"] = c["table"].copy()
    bad["table"][1, 0] = 10 ** 8
    got = run(bad)
    assert np.array_equal(got[0], want[0]) and not got[2:].any()
    bad = dict(c)
    bad["cu"] = np.array([0, 1, 900, 2], dtype=np.int32)
    assert np.array_equal(run(bad)[0], want[0])


def test_other_stream_workspace_and_out():
    note("stream, workspace, out")
    c = make(np.random.default_rng(14), [1, 3], [3000, 900], 2, 4, 128, 16, True)
    want = run(c)
    ws = torch.full((256 << 20,), 255, dtype=torch.uint8, device=DEV)
    ws[:1 << 20] = 0
    out = torch.empty(c["q"].shape, dtype=torch.float16, device=DEV)
    args = [dev(c[n]) for n in ("q", "k", "v", "table", "cu", "lens")]
    ks, vs = dev(c["k_scale"]), dev(c["v_scale"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = sp.spear_paged_attention(*args, 3, k_scale=ks, v_scale=vs, out=out, workspace=ws)
    s.synchronize()
    assert got is out and np.array_equal(out.cpu().numpy(), want)
    assert not ws[:1 << 20].any()                     # the header's counters are back at zero


@pytest.mark.parametrize("int8", [False, True])
def test_graph_replays_follow_the_lengths(int8):
    """A captured call reads lengths, tables and queries anew at each replay."""
    note(f"captured attention int8 {int8}")
    rng = np.random.default_rng(15)
    c = make(rng, [1, 2, 1], [2500, 77, 300], 2, 4, 64, 16, int8, fill=0.0)
    t = {n: dev(c[n]) for n in ("q", "k", "v", "table", "cu", "lens", "k_scale", "v_scale")}
    out = torch.empty(c["q"].shape, dtype=torch.float16, device=DEV)
    ws = torch.zeros(256 << 20, dtype=torch.uint8, device=DEV)
    call = lambda: sp.spear_paged_attention(t["q"], t["k"], t["v"], t["table"], t["cu"], t["lens"], 2,  # noqa: E731
                                            k_scale=t["k_scale"], v_scale=t["v_scale"], out=out, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([2500, 77, 300], [100, 50, 299], [1, 2, 0], [2400, 77, 1]):
        c["lens"] = np.asarray(lens, dtype=np.int32)
        c["q"] = rng.normal(size=c["q"].shape).astype(np.float16)
        t["lens"].copy_(torch.from_numpy(c["lens"]))
        t["q"].copy_(torch.from_numpy(c["q"]))
        g.replay()
        torch.cuda.synchronize()
        got = out.cpu().numpy()
        check(c, got)
        assert np.array_equal(got, run(c))


def test_refusals():
    c = make(np.random.default_rng(16), [1, 2], [20, 30], 2, 2, 64, 16, False, fill=0.0)
    a = {n: dev(c[n]) for n in ("q", "k", "v", "table", "cu", "lens")}

    def call(max_q=2, scale=None, workspace=None, **other):
        b = {**a, **other}
        return sp.spear_paged_attention(b["q"], b["k"], b["v"], b["table"], b["cu"], b["lens"], max_q, scale=scale,
                                        workspace=workspace)
    call()
    for other, error in (({"q": a["q"].float()}, TypeError), ({"table": a["table"].long()}, TypeError),
                         ({"cu": a["cu"][:2]}, ValueError), ({"lens": a["lens"][:1]}, ValueError),
                         ({"q": a["q"][:, :, :32]}, ValueError), ({"v": a["v"][:1]}, ValueError),
                         ({"q": a["q"].transpose(1, 2)}, ValueError), ({"k": a["k"].cpu()}, ValueError),
                         ({"table": a["table"].cpu()}, ValueError)):
        with pytest.raises(error):
            call(**other)
    with pytest.raises(sp.SpearError, match="INVALID_SHAPE"):
        call(q=a["q"][:, :3])                       # heads not a multiple of the kv heads
    with pytest.raises(sp.SpearError, match="INVALID_SHAPE"):
        call(max_q=0)
    for scale in (float("nan"), float("inf")):
        with pytest.raises(sp.SpearError, match="INVALID_ARGUMENT"):
            call(scale=scale)
    big = torch.zeros(2, 100, dtype=torch.int32, device=DEV)
    with pytest.raises(sp.SpearError, match="WORKSPACE"):
        call(table=big, workspace=torch.zeros(1 << 20, dtype=torch.uint8, device=DEV))
    assert call(q=a["q"][:0]).shape == (0, 4, 64)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("batch,kv_heads,group,dim,q_most,kv_most", [
    (150, 2, 4, 64, 1, 300), (300, 1, 1, 128, 1, 40), (90, 3, 20, 64, 1, 200), (70, 1, 40, 128, 1, 150),
    (100, 2, 3, 128, 4, 120), (80, 1, 20, 64, 3, 90)])
def test_large_batches(int8, batch, kv_heads, group, dim, q_most, kv_most):
    """More sequences than one scan step takes; more query heads to a kv head than
    16 and 32 rows; sequences without new tokens or without cached ones between."""
    note(f"batch {batch} int8 {int8} kv_heads {kv_heads} group {group} dim {dim}")
    rng = np.random.default_rng(batch + group)
    q_lens = rng.integers(0 if batch != 90 else 1, q_most + 1, size=batch).tolist()
    lens = np.exp(rng.uniform(0, math.log(kv_most), size=batch)).astype(int) + rng.integers(0, 2, size=batch)
    lens[::17] = 0
    c = make(rng, q_lens, lens.tolist(), kv_heads, group, dim, 16, int8)
    check(c, run(c))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("q_lens,lens,kv_heads,group,dim", [
    ([300, 1, 1, 5, 1], [900, 2000, 30, 400, 1], 1, 2, 64),       # both kernels, the long one in pieces
    ([300, 1, 1], [300, 700, 64], 2, 24, 64),                     # .. 32 rows for one token's heads
    ([130, 90], [2500, 1300], 1, 1, 128),                         # row tiles in pieces, two lengths
    ([64, 64, 64], [64, 1000, 129], 3, 4, 128),                   # tiles alone
    ([33], [4000], 1, 1, 128), ([500], [500], 1, 5, 64)])
def test_tiles_and_pieces(int8, q_lens, lens, kv_heads, group, dim):
    note(f"tiles int8 {int8} q {q_lens} kv {lens} group {group} dim {dim}")
    c = make(np.random.default_rng(sum(lens)), q_lens, lens, kv_heads, group, dim, 32, int8)
    got = run(c)
    check(c, got)
    assert np.array_equal(got.view(np.uint16), run(c).view(np.uint16))


def test_calls_on_one_workspace_do_not_meet():
    """Calls of other shapes one after the other on the stream's workspace, which
    the linear layer and the verification use too: counters are left at zero."""
    note("shared workspace")
    rng = np.random.default_rng(21)
    cases = [make(rng, [1, 1], [4000, 90], 2, 4, 128, 16, True), make(rng, [200, 1], [1500, 2600], 1, 2, 64, 16, False),
             make(rng, [6], [5000], 2, 4, 64, 16, True)]
    want = [run(c) for c in cases]
    for _ in range(3):
        for c, w in zip(cases, want):
            assert np.array_equal(run(c).view(np.uint16), w.view(np.uint16))
