"""Calls on the stream's cached workspace under graph capture: refused where it would
have to be made or grown, right in every replay where it is there, also after a
larger eager call has replaced it."""
import numpy as np
import pytest
import torch

import workloads
import w4_gemm_gated_amd as sp
from test_gpu_paged_attention import dev, make

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-workspace] {msg}", flush=True)


def attention(rng, q_lens, lens):
    c = make(rng, q_lens, lens, 2, 4, 128, 16, False)
    t = [dev(c[n]) for n in ("q", "k", "v", "table", "cu", "lens")]
    return lambda out=None: sp.spear_paged_attention(*t, c["max_q"], out=out)


def linear(rng, M, K, N, r, variant="auto"):
    X, W, A, B, w_g = workloads.random_layer(M, K, N, r, seed=5, outliers=True)
    Wq, s = sp.spear_pack_w4(dev(W))
    args = (dev(X), Wq, s, dev(A), dev(B), dev(w_g), -0.5)
    return lambda out=None: sp.spear_w4ec_linear(*args, variant=variant, Y=out)


def verification(rng, B, K, V):
    p = rng.exponential(size=(B, K + 1, V)).astype(np.float32)
    p /= p.sum(-1, keepdims=True)
    a = [dev(p), dev(p[:, :K]), dev(rng.integers(0, V, size=(B, K)).astype(np.int32)),
         dev(rng.random(size=(B, K), dtype=np.float32)), dev(rng.exponential(size=(B, V)).astype(np.float32))]
    return lambda out=None: sp.spear_verify_draft(*a, tokens=out)[1]


@pytest.fixture
def fresh(monkeypatch):
    monkeypatch.setattr(sp, "_workspaces", {})
    torch.cuda.synchronize()
    yield torch.cuda.Stream()
    torch.cuda.synchronize()


def capture(stream, call, out):
    g = torch.cuda.CUDAGraph()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=stream):
        call(out)
    return g


@pytest.mark.parametrize("kind", ["attention", "linear", "verification"])
def test_capture_without_a_workspace_is_refused(fresh, kind):
    note(f"refused: {kind}")
    rng = np.random.default_rng(1)
    call = {"attention": lambda: attention(rng, [1, 1], [3000, 40]), "linear": lambda: linear(rng, 4, 1024, 2048, 32, "fused"),
            "verification": lambda: verification(rng, 2, 2, 33000)}[kind]()
    out = torch.empty_like(call())
    torch.cuda.synchronize()
    refused = False
    try:
        capture(fresh, call, out)
    except Exception as e:      # the refusal (ending an empty capture may raise on top of it)
        refused = any("workspace=" in str(x) for x in (e, e.__context__) if x is not None)
    assert refused
    torch.cuda.synchronize()
    want = call().clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(fresh):
        got = call()
    fresh.synchronize()
    assert torch.equal(got, want)


def test_replays_after_a_larger_call(fresh):
    """Decode, verification and layer captured on a stream's workspace; then a prompt's
    chunk replaces that workspace, and memory is handed to other tensors."""
    note("replays after the workspace grew")
    rng = np.random.default_rng(2)
    calls = [attention(rng, [1, 1, 1], [3000, 40, 700]), verification(rng, 3, 2, 33000), linear(rng, 4, 1024, 2048, 32)]
    chunk = attention(rng, [300, 1], [2500, 900])
    want = [call().clone() for call in calls]
    torch.cuda.synchronize()
    with torch.cuda.stream(fresh):
        for call in calls:
            call()
    fresh.synchronize()
    outs = [torch.empty_like(w) for w in want]
    graphs = [capture(fresh, call, out) for call, out in zip(calls, outs)]
    torch.cuda.synchronize()
    with torch.cuda.stream(fresh):
        before = {n: w.data_ptr() for n, w in sp._workspaces.items()}
        chunk()
    fresh.synchronize()
    assert any(sp._workspaces[n].data_ptr() != at for n, at in before.items()), "the workspace did not grow"
    with torch.cuda.stream(fresh):
        others = [torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV) for _ in range(64)]
    fresh.synchronize()
    for _ in range(4):
        for g, out, w, call in zip(graphs, outs, want, calls):
            out.fill_(7)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w)
            with torch.cuda.stream(fresh):
                assert torch.equal(call(), w)
            fresh.synchronize()
    assert all(bool((x == 255).all()) for x in others)
    del graphs
