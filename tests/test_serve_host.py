"""The serving operators' C ABI on the host (no GPU): exports, argument checks in
the order in which they are documented, workspace sizes.  No call reaches a kernel."""
import ctypes
import os
import re

import pytest

from w4_gemm_gated_amd import _binding

REPO = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(REPO, "include", "spear_serve.h")
OK, NULL, SHAPE, UNSUPPORTED, MISALIGNED, SMALL, ARGUMENT = 0, 1, 2, 3, 4, 5, 8

pytestmark = pytest.mark.skipif(not os.path.exists(_binding.LIB_PATH),
                                reason="libspear_w4ec.so not built (run __graft_entry__.build())")


@pytest.fixture(scope="module")
def lib():
    return _binding.load()


@pytest.fixture(scope="module")
def buf():
    raw = ctypes.create_string_buffer(1 << 12)
    at = (ctypes.addressof(raw) + 63) // 64 * 64
    return raw, at


def test_header_and_binding_agree(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(spear_[a-z0-9_]+)\s*\(", text))
    assert names == set(_binding.SERVE_EXPORTS)
    for n in names:
        assert ctypes.cast(getattr(lib, n), ctypes.c_void_p).value
    assert not names & set(_binding.EXPORTS)


def kv(dtype=0, pages=4, heads=2, dim=64, page=16):
    return _binding.KvDesc(dtype, pages, heads, dim, page)


def append(lib, p, d=None, tokens=1, k=True, ts=128, hs=64, slots=True, cache=True, ks=True, off=0):
    d = kv() if d is None else d
    f = lambda on: p + off if on else None  # noqa: E731
    return lib.spear_kv_append(ctypes.byref(d), tokens, f(k), ts, hs, f(k), ts, hs, f(slots), f(cache), f(cache), f(ks),
                               f(ks), None)


def test_append_checks(lib, buf):
    p = buf[1]
    assert lib.spear_kv_append(None, 1, p, 128, 64, p, 128, 64, p, p, p, p, p, None) == NULL
    for d in (kv(pages=0), kv(heads=0), kv(dim=0), kv(page=0)):
        assert append(lib, p, d) == SHAPE
    assert append(lib, p, kv(dtype=2)) == ARGUMENT
    for d in (kv(dim=96), kv(page=8), kv(page=24), kv(page=2048), kv(heads=1025)):
        assert append(lib, p, d) == UNSUPPORTED
    assert append(lib, p, tokens=-1) == SHAPE
    assert append(lib, p, ts=130) == SHAPE and append(lib, p, hs=-8) == SHAPE
    assert append(lib, p, tokens=0, k=False, slots=False, cache=False) == OK
    assert append(lib, p, k=False) == NULL and append(lib, p, slots=False) == NULL and append(lib, p, cache=False) == NULL
    assert append(lib, p, kv(dtype=1), ks=False) == NULL
    assert append(lib, p, off=8) == MISALIGNED
    assert append(lib, p, kv(heads=1024), tokens=(1 << 17) + 1) == UNSUPPORTED     # more than a launch's threads


def test_gather_checks(lib, buf):
    p = buf[1]

    def gather(d=None, batch=1, rows=1, table=p, stride=4, cu=p, c=p, s=p, o=p):
        d = kv() if d is None else d
        return lib.spear_kv_gather(ctypes.byref(d), batch, rows, table, stride, cu, c, c, s, s, o, o, None)
    assert lib.spear_kv_gather(None, 1, 1, p, 4, p, p, p, p, p, p, p, None) == NULL
    assert gather(kv(dim=32)) == UNSUPPORTED and gather(kv(dtype=9)) == ARGUMENT
    assert gather(batch=-1) == SHAPE and gather(rows=-1) == SHAPE and gather(stride=0) == SHAPE
    assert gather(rows=0, table=None, cu=None, c=None, o=None) == OK
    assert gather(table=None) == NULL and gather(cu=None) == NULL and gather(c=None) == NULL and gather(o=None) == NULL
    assert gather(kv(dtype=1), s=None) == NULL
    assert gather(kv(heads=1024), rows=(1 << 18) + 1) == UNSUPPORTED
    assert gather(o=p + 2) == MISALIGNED and gather(cu=p + 2) == MISALIGNED and gather(c=p + 8) == MISALIGNED


def attention(**o):
    a = dict(kv=kv(), batch=2, total_q=2, max_q=1, max_pages=4, q_heads=4, scale=0.1, device_cus=256)
    a.update(o)
    return _binding.AttentionDesc(*a.values())


def test_attention_checks(lib, buf):
    p = buf[1]
    n = ctypes.c_size_t(0)

    def size(d):
        return lib.spear_attention_workspace_bytes(ctypes.byref(d), ctypes.byref(n))

    def call(d, q=p, ts=256, hs=64, cu=p, table=p, stride=4, c=p, s=p, out=p, ws=p, bytes_=1 << 40):
        return lib.spear_paged_attention(ctypes.byref(d), q, ts, hs, cu, cu, table, stride, c, c, s, s, out, ws, bytes_,
                                         None)
    assert lib.spear_attention_workspace_bytes(None, ctypes.byref(n)) == NULL
    assert lib.spear_attention_workspace_bytes(ctypes.byref(attention()), None) == NULL
    for d, want in ((attention(batch=-1), SHAPE), (attention(total_q=-1), SHAPE), (attention(max_q=0), SHAPE),
                    (attention(max_pages=0), SHAPE), (attention(q_heads=3), SHAPE), (attention(q_heads=0), SHAPE),
                    (attention(scale=float("nan")), ARGUMENT), (attention(scale=float("-inf")), ARGUMENT),
                    (attention(scale=1e31), ARGUMENT), (attention(device_cus=-1), ARGUMENT),
                    (attention(kv=kv(dim=80)), UNSUPPORTED), (attention(max_pages=1 << 27), UNSUPPORTED),
                    (attention(total_q=1 << 29), UNSUPPORTED), (attention(batch=1 << 21), UNSUPPORTED)):
        assert size(d) == want and call(d) == want
    for d in (attention(batch=0), attention(total_q=0)):
        assert size(d) == OK and n.value == 0
        assert call(d, q=None, cu=None, table=None, c=None, out=None, ws=None, bytes_=0) == OK
    d = attention()
    assert size(d) == OK and n.value > 1 << 20
    assert lib.spear_paged_attention(None, p, 256, 64, p, p, p, 4, p, p, p, p, p, p, 1 << 40, None) == NULL
    assert call(d, ts=252) == SHAPE and call(d, stride=3) == SHAPE
    for o in ({"q": None}, {"cu": None}, {"table": None}, {"c": None}, {"out": None}, {"ws": None}):
        assert call(d, **o) == NULL
    assert call(attention(kv=kv(dtype=1)), s=None) == NULL
    for o in ({"q": p + 2}, {"out": p + 8}, {"cu": p + 1}, {"c": p + 4}, {"ws": p + 8}):
        assert call(d, **o) == MISALIGNED
    assert call(d, bytes_=n.value - 1) == SMALL


def test_workspaces_follow_the_launch_shape(lib):
    """Room for two partial results of 16 or 32 rows for each workgroup, which are
    as many as the GPU holds or as there can be steps of 128 keys, and of 128 rows
    for two pieces of each item aimed at: whatever the lengths turn out to be, they
    fit (the kernels' own bound)."""
    n = ctypes.c_size_t(0)

    def size(**o):
        assert lib.spear_attention_workspace_bytes(ctypes.byref(attention(**o)), ctypes.byref(n)) == OK
        return n.value - (1 << 20)
    item = lambda rows, dim: rows * (dim + 2) * 4  # noqa: E731
    assert size() == 2 * 4 * item(16, 64)                          # 2 sequences x 2 heads, 64 keys at most
    assert size(max_pages=9) == 2 * 2 * 4 * item(16, 64)           # 144 keys: two steps
    assert size(max_pages=10000) == 2 * 3 * 256 * item(16, 64)
    assert size(max_pages=10000, max_q=9, total_q=18, kv=kv(dim=128)) == 2 * 2 * 256 * item(32, 128)
    assert size(max_q=100, total_q=200) == 2 * 2 * 256 * item(128, 64)                      # tiles alone
    assert size(max_q=100, total_q=101) == 2 * 2 * 256 * item(128, 64) + 2 * 4 * item(16, 64)
    assert size(max_pages=10000, device_cus=4096) == 2 * 3 * 512 * item(16, 64)   # no more than the counters allow
    v = _binding.VerifyDesc(2, 3, 100, 256)
    assert lib.spear_verify_workspace_bytes(ctypes.byref(v), ctypes.byref(n)) == OK and n.value == 0
    v = _binding.VerifyDesc(2, 3, 100000, 256)
    assert lib.spear_verify_workspace_bytes(ctypes.byref(v), ctypes.byref(n)) == OK
    assert n.value == (1 << 20) + 2 * 25 * 8
    v = _binding.VerifyDesc(5000, 3, 100000, 256)                   # more sequences than counters: no sharing
    assert lib.spear_verify_workspace_bytes(ctypes.byref(v), ctypes.byref(n)) == OK and n.value == 0


def test_verify_checks(lib, buf):
    p = buf[1]

    def call(batch=1, K=2, V=5000, cus=256, target=p, draft=p, drafted=p, u=p, noise=p, acc=p, tok=p, ws=p,
             bytes_=1 << 40, stride=5000):
        d = _binding.VerifyDesc(batch, K, V, cus)
        return lib.spear_verify_draft(ctypes.byref(d), target, stride, stride, draft, stride, stride, drafted, u, noise,
                                      None, acc, tok, ws, bytes_, None)
    assert lib.spear_verify_draft(None, p, 1, 1, p, 1, 1, p, p, p, p, p, p, p, 0, None) == NULL
    assert call(batch=-1) == SHAPE and call(K=-1) == SHAPE and call(V=0) == SHAPE and call(stride=-1) == SHAPE
    assert call(cus=-1) == ARGUMENT
    assert call(V=(1 << 30) + 1) == UNSUPPORTED and call(K=1 << 21) == UNSUPPORTED
    assert call(batch=0, target=None, noise=None, acc=None, tok=None, ws=None, bytes_=0) == OK
    for o in ({"target": None}, {"noise": None}, {"acc": None}, {"tok": None}, {"drafted": None}, {"u": None}, {"ws": None}):
        assert call(**o) == NULL
    for o in ({"target": p + 2}, {"draft": p + 1}, {"noise": p + 2}, {"tok": p + 2}, {"ws": p + 8}):
        assert call(**o) == MISALIGNED
    assert call(bytes_=(1 << 20) + 8) == SMALL


def test_gather_of_no_sequences_needs_no_table(lib, buf):
    p = buf[1]
    d = kv()

    def gather(batch, table, stride, out, cu=p):
        return lib.spear_kv_gather(ctypes.byref(d), batch, 1, table, stride, cu, p, p, p, p, out, out, None)
    # (the outputs' alignment is looked at after the table)
    assert gather(0, None, 4, p + 2) == MISALIGNED and gather(0, None, 0, p + 2) == MISALIGNED
    assert gather(1, None, 4, p + 2) == NULL and gather(1, p, 0, p) == SHAPE
    assert gather(0, None, 0, p, cu=None) == NULL


def test_verification_takes_no_more_sequences_than_a_launch_holds(lib, buf):
    n = ctypes.c_size_t(0)

    def size(batch):
        return lib.spear_verify_workspace_bytes(ctypes.byref(_binding.VerifyDesc(batch, 1, 100, 256)), ctypes.byref(n))
    assert size(1 << 24) == UNSUPPORTED             # 2^24 workgroups of 256: 2^32 threads
    assert size((1 << 24) - 1) == OK and n.value == 0
