"""Tensors of a device other than the current one are refused: the library launches on
the current device.  (The other device is played by torch's answer, so one GPU or
none is enough.)"""
import types

import pytest
import torch

import w4_gemm_gated_amd as sp
from w4_gemm_gated_amd import serve

DEV = "cuda:0"


def test_a_stream_is_taken_on_the_current_device_only(monkeypatch):
    asked = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: asked.append(d) or types.SimpleNamespace(cuda_stream=7))
    monkeypatch.setattr(serve, "_raw_stream", None)
    for stream in (sp._stream, serve._stream):
        with pytest.raises(ValueError, match="current device is cuda:0"):
            stream(torch.device("cuda", 1))
        assert not asked
        at = stream(torch.device("cuda", 0))
        assert getattr(at, "value", at) == 7 and asked.pop() == torch.device("cuda", 0)
    assert sp._stream(torch.device("cuda")).value == 7      # "cuda" alone is the current one


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
def test_every_call_refuses_another_device(monkeypatch):
    f16 = dict(dtype=torch.float16, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    X, W = torch.zeros(4, 256, **f16), torch.zeros(256, 512, **f16)
    Wq, s = sp.spear_pack_w4(W)
    A, w_g = torch.zeros(256, 16, **f16), torch.zeros(256, **f16)
    kc, vc, _, _ = sp.spear_kv_cache(4, 2, 64, 16, torch.float16, DEV)
    x = torch.ones(3, 2, 64, **f16)
    table, cu = torch.zeros(1, 4, **i32), torch.tensor([0, 3], **i32)
    lens = torch.tensor([3], **i32)
    p = torch.ones(1, 2, 9000, device=DEV)
    word = torch.zeros(256, dtype=torch.int32, device=DEV)
    calls = {
        "pack": lambda: sp.spear_pack_w4(W), "pack_grouped": lambda: sp.spear_pack_w4_grouped(W),
        "unpack": lambda: sp.spear_debug_unpack_w4(Wq, 256, 512), "init": lambda: sp.spear_ec_init(W, Wq, s, 16),
        "linear": lambda: sp.spear_w4ec_linear(X, Wq, s, None, None, None, 0.0),
        "noalloc": lambda: sp.spear_w4ec_linear_noalloc(X, Wq, s, None, None, None, 0.0),
        "project": lambda: sp.spear_ec_project(X, A, w_g, 0.0),
        "error": lambda: sp.spear_take_error(torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)),
        "read": lambda: sp.spear_debug_stream_read(W, 256, word),
        "append": lambda: sp.spear_kv_append(x, x, torch.arange(3, device=DEV), kc, vc),
        "gather": lambda: sp.spear_kv_gather(kc, vc, table, cu, 3),
        "attention": lambda: sp.spear_paged_attention(x, kc, vc, table, cu, lens, 3),
        "verify": lambda: sp.spear_verify_draft(p, None, torch.zeros(1, 1, **i32), torch.zeros(1, 1, device=DEV),
                                                torch.ones(1, 9000, device=DEV)),
    }
    for call in calls.values():
        call()
    torch.cuda.synchronize()
    kc.zero_()
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1)
        for name, call in calls.items():
            print(f"[gpu-device] {name}", flush=True)
            with pytest.raises(ValueError, match="current device is cuda:1"):
                call()
    torch.cuda.synchronize()
    assert not kc.any()                         # nothing was launched
