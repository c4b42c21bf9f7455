"""The layer, attention and verification one after the other on one workspace: the
counters, flags and epoch of its header serve all of them, so every call gives the
same bits as on a workspace of its own, in any order."""
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
    print(f"[gpu-shared] {msg}", flush=True)


def layer(M, K, N, r, variant):
    X, W, A, B, w_g = workloads.random_layer(M, K, N, r, seed=M + K, outliers=True)
    Wq, s = sp.spear_pack_w4(dev(W))
    args = (dev(X), Wq, s, dev(A), dev(B), dev(w_g), -0.5)
    return lambda ws: sp.spear_w4ec_linear(*args, variant=variant, workspace=ws)


def attention(q_lens, lens, int8):
    c = make(np.random.default_rng(sum(lens)), q_lens, lens, 2, 4, 64, 16, int8)
    t = [dev(c[n]) for n in ("q", "k", "v", "table", "cu", "lens")]
    ks, vs = dev(c["k_scale"]), dev(c["v_scale"])
    return lambda ws: sp.spear_paged_attention(*t, c["max_q"], k_scale=ks, v_scale=vs, workspace=ws)


def verification(B, K, V):
    rng = np.random.default_rng(V)
    p = rng.exponential(size=(B, K + 1, V)).astype(np.float32)
    p /= p.sum(-1, keepdims=True)
    a = [dev(p), dev(p[:, :K]), dev(rng.integers(0, V, size=(B, K)).astype(np.int32)),
         dev(rng.random(size=(B, K), dtype=np.float32)), dev(rng.exponential(size=(B, V)).astype(np.float32))]
    return lambda ws: sp.spear_verify_draft(*a, workspace=ws)[1]


@pytest.mark.parametrize("given", [True, False])
def test_all_operators_share_a_workspace(given, monkeypatch):
    note("given" if given else "the stream's")
    calls = {
        "fused decode": layer(4, 4096, 1024, 32, "fused"), "split decode": layer(16, 2048, 1024, 32, "split"),
        "fused tiles": layer(200, 1024, 2048, 32, "fused"), "split tiles": layer(300, 2048, 1024, 64, "split"),
        "decode": attention([1, 1, 1], [4000, 40, 900], True), "chunk and decode": attention([300, 1], [2500, 3000], False),
        "verification": verification(3, 2, 50000),
    }
    monkeypatch.setattr(sp, "_workspaces", {})
    own = {n: call(torch.zeros(256 << 20, dtype=torch.uint8, device=DEV)).clone() for n, call in calls.items()}
    torch.cuda.synchronize()
    ws = torch.zeros(256 << 20, dtype=torch.uint8, device=DEV) if given else None
    rng = np.random.default_rng(7)
    order = [n for _ in range(6) for n in rng.permutation(list(calls))]
    got = [(n, calls[n](ws)) for n in order]        # (no wait between them)
    torch.cuda.synchronize()
    for n, x in got:
        assert torch.equal(x, own[n]), n
    assert sp.spear_take_error(ws) == 0
