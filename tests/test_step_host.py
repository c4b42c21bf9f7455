"""The C ABI of a serving step's other operators (block tables, adapters, sampling) on the
host (no GPU): argument checks in the order in which they are documented, workspace
sizes.  No call reaches a kernel."""
import ctypes
import os
import re

import pytest
import torch

from w4_gemm_gated_amd import _binding
from w4_gemm_gated_amd._binding import AdapterDesc, KvPlanDesc, SampleDesc

OK, NULL, SHAPE, UNSUPPORTED, MISALIGNED, SMALL, ARGUMENT = 0, 1, 2, 3, 4, 5, 8
HEADER = 1 << 20

pytestmark = pytest.mark.skipif(not os.path.exists(_binding.LIB_PATH),
                                reason="libspear_w4ec.so not built (run __graft_entry__.build())")


@pytest.fixture(scope="module")
def lib():
    return _binding.load()


@pytest.fixture(scope="module")
def buf():
    raw = ctypes.create_string_buffer(1 << 12)
    return raw, (ctypes.addressof(raw) + 63) // 64 * 64


def size_of(fn, d):
    n = ctypes.c_size_t(0)
    return fn(ctypes.byref(d), ctypes.byref(n)), n.value


# ---------------------------------------------------------------- block tables

NAMES = ("lens", "new", "held", "table", "stack", "count", "cu", "kv_lens", "slots", "positions", "sequence", "held_out",
         "free_out")


def kv_plan(lib, p, batch=3, rows=3000, pages=8, page=16, free=9, stride=8, ws=True, bytes_=HEADER, **at):
    a = {n: p for n in NAMES}
    a.update(at)
    v = [a[n] for n in NAMES]
    return lib.spear_kv_plan(ctypes.byref(KvPlanDesc(batch, rows, pages, page, free)), *v[:4], stride, *v[4:],
                             p if ws is True else ws, bytes_, None)


def test_kv_plan_checks(lib, buf):
    p = buf[1]
    assert lib.spear_kv_plan(None, p, p, p, p, 8, p, p, p, p, p, p, p, p, p, p, 0, None) == NULL
    for o in ({"batch": -1}, {"rows": -1}, {"pages": 0}, {"page": 0}, {"free": -1}, {"stride": 7}, {"stride": -8},
              {"stride": (1 << 31) + 1}):
        assert kv_plan(lib, p, **o) == SHAPE, o
    for o in ({"batch": (1 << 20) + 1}, {"rows": (1 << 30) + 1}, {"page": 8}, {"page": 24}, {"page": 2048},
              {"pages": (1 << 26) + 1}):
        assert kv_plan(lib, p, **o) == UNSUPPORTED, o
    for n in NAMES:
        assert kv_plan(lib, p, **{n: None}) == NULL, n
        assert kv_plan(lib, p, **{n: p + 2}) == MISALIGNED, n
    assert kv_plan(lib, p, slots=p + 4) == MISALIGNED
    assert kv_plan(lib, p, ws=None) == NULL and kv_plan(lib, p, ws=p + 8) == MISALIGNED
    assert kv_plan(lib, p, bytes_=HEADER - 1) == SMALL
    # what a call of nothing does not read may be NULL, what it writes may not
    none = dict(lens=None, new=None, held=None, table=None, kv_lens=None, held_out=None)
    assert kv_plan(lib, p, batch=0, **none, cu=None) == NULL
    assert kv_plan(lib, p, batch=0, **none, free_out=p + 1) == MISALIGNED
    assert kv_plan(lib, p, rows=0, slots=None, positions=None, sequence=None, count=None) == NULL
    assert kv_plan(lib, p, rows=0, slots=None, positions=None, sequence=None, count=p + 1) == MISALIGNED


def test_kv_plan_workspace(lib):
    f = lib.spear_kv_plan_workspace_bytes
    assert f(None, None) == NULL and f(ctypes.byref(KvPlanDesc(1, 1, 1, 16, 1)), None) == NULL
    # counters, where more than one workgroup has rows to fill
    for batch, rows, want in ((0, 0, 0), (1, 256, 0), (1, 257, HEADER), (1024, 256, 0), (1025, 512, 0), (1025, 513, HEADER),
                              (1 << 20, 1 << 30, HEADER)):
        assert size_of(f, KvPlanDesc(batch, rows, 4, 16, 0)) == (OK, want)
    assert size_of(f, KvPlanDesc(1, 1, 4, 8, 0))[0] == UNSUPPORTED
    assert size_of(f, KvPlanDesc(1, 1, 0, 16, 0))[0] == SHAPE


# -------------------------------------------------------------------- adapters

def test_adapter_plan_checks(lib, buf):
    p = buf[1]
    n = ctypes.c_size_t(0)

    def call(batch=2, adapters=3, rows=5, cu=p, of=p, plan=p, bytes_=1 << 12):
        return lib.spear_adapter_plan(batch, adapters, rows, cu, of, plan, bytes_, None)
    size = lambda *a: lib.spear_adapter_plan_bytes(*a, ctypes.byref(n))  # noqa: E731
    assert lib.spear_adapter_plan_bytes(1, 1, 1, None) == NULL
    for o, want in (({"batch": -1}, SHAPE), ({"adapters": 0}, SHAPE), ({"rows": -1}, SHAPE),
                    ({"batch": (1 << 20) + 1}, UNSUPPORTED), ({"adapters": 4097}, UNSUPPORTED),
                    ({"rows": (1 << 24) + 1}, UNSUPPORTED)):
        a = dict(batch=2, adapters=3, rows=5)
        a.update(o)
        assert size(*a.values()) == want and call(**o) == want
    assert call(plan=None) == NULL and call(cu=None) == NULL and call(of=None) == NULL
    assert call(batch=0, cu=None, of=None, plan=None) == NULL
    assert size(2, 3, 5) == OK
    assert call(bytes_=n.value - 1) == SMALL
    assert call(cu=p + 2) == MISALIGNED and call(of=p + 1) == MISALIGNED and call(plan=p + 8) == MISALIGNED
    # a list of the rows and a tile for each 64 of an adapter
    for batch, adapters, rows, tiles in ((1, 1, 1, 1), (1, 1, 64, 1), (1, 1, 65, 2), (9, 9, 9, 9), (9, 2, 9, 2),
                                         (4, 4, 2048, 35), (5000, 4096, 5000, 4110)):
        assert size(batch, adapters, rows) == OK and 16 * tiles + 4 * rows <= n.value <= 16 * tiles + 4 * rows + 64
    assert size(0, 1, 0) == OK and n.value > 0


def adapter(batch=2, adapters=3, rows=5, K=64, N=32, rank=16, cus=256):
    return AdapterDesc(batch, adapters, rows, K, N, rank, cus)


def test_adapter_add_checks(lib, buf):
    p = buf[1]
    f = lib.spear_adapter_workspace_bytes

    def call(d, x=p, xs=64, a=p, b=p, scale=p, plan=p, bytes_=1 << 12, y=p, ys=32, ws=p, ws_bytes=1 << 40):
        return lib.spear_adapter_add(ctypes.byref(d), x, xs, a, b, scale, plan, bytes_, y, ys, ws, ws_bytes, None)
    assert f(None, None) == NULL and f(ctypes.byref(adapter()), None) == NULL
    assert lib.spear_adapter_add(None, p, 64, p, p, p, p, 64, p, 32, p, 0, None) == NULL
    for o, want in (({"batch": -1}, SHAPE), ({"rows": -1}, SHAPE), ({"adapters": 0}, SHAPE), ({"K": 0}, SHAPE),
                    ({"K": 60}, SHAPE), ({"N": 0}, SHAPE), ({"rank": 0}, SHAPE), ({"rank": 12}, SHAPE),
                    ({"rank": 264}, UNSUPPORTED), ({"K": (1 << 24) + 8}, UNSUPPORTED), ({"N": (1 << 24) + 1}, UNSUPPORTED),
                    ({"adapters": 4097}, UNSUPPORTED), ({"rows": 1 << 24, "N": 1 << 24}, UNSUPPORTED),
                    ({"cus": -1}, ARGUMENT)):
        d = adapter(**o)
        assert size_of(f, d)[0] == want and call(d, ys=1 << 24) == want, o
    d = adapter()
    st, need = size_of(f, d)
    assert st == OK and need > HEADER
    for o in ({"xs": -8}, {"xs": 60}, {"xs": (1 << 31) + 8}, {"ys": 31}, {"ys": (1 << 31) + 1}):
        assert call(d, **o) == SHAPE, o
    for none in (adapter(batch=0), adapter(rows=0)):
        assert size_of(f, none) == (OK, 0)
        assert call(none, x=None, a=None, b=None, scale=None, plan=None, y=None, ws=None, ws_bytes=0) == OK
    for n in ("x", "a", "b", "plan", "y", "ws"):
        assert call(d, **{n: None}) == NULL, n
    for o in ({"x": p + 8}, {"a": p + 2}, {"b": p + 8}, {"scale": p + 2}, {"plan": p + 8}, {"y": p + 1}, {"ws": p + 8}):
        assert call(d, **o) == MISALIGNED, o
    assert call(d, bytes_=16) == SMALL and call(d, ws_bytes=need - 1) == SMALL


@pytest.mark.parametrize("cus", [1, 80, 256, 1 << 20])
def test_adapter_workspaces_hold_what_the_products_exchange(lib, cus):
    """H as two fp16 numbers a value and a factor, for as many tiles as there can be."""
    for batch, adapters, rows, K, N, rank in ((1, 1, 1, 8, 8, 8), (64, 24, 64, 8192, 2048, 16), (41, 12, 740, 14336, 4096, 32),
                                              (5, 4, 2048, 4096, 14336, 64), (3, 2, 700, 40, 9, 256),
                                              (100000, 4096, 1 << 20, 512, 512, 128)):
        tiles = (rows + 63 * min(batch, adapters, rows)) // 64
        st, need = size_of(lib.spear_adapter_workspace_bytes, adapter(batch, adapters, rows, K, N, rank, cus))
        assert st == OK and need >= HEADER + tiles * 64 * (4 * rank + 4)


# -------------------------------------------------------------------- sampling

def test_sample_checks(lib, buf):
    p = buf[1]
    f = lib.spear_sample_workspace_bytes

    def call(batch=2, V=100, rows_=3, dtype=0, T=1.0, k=0, top_p=1.0, m=0.0, z=p, stride=100, rows=p, noise=p, t=p, ks=p,
             ps=p, ms=p, tok=p, probs=p, ws=p, bytes_=1 << 40):
        d = SampleDesc(batch, V, rows_, dtype, T, k, top_p, m)
        return lib.spear_sample(ctypes.byref(d), z, stride, rows, noise, t, ks, ps, ms, tok, probs, ws, bytes_, None)
    assert f(None, None) == NULL and f(ctypes.byref(SampleDesc(1, 1, 1, 0, 1, 0, 1, 0)), None) == NULL
    assert lib.spear_sample(None, p, 1, p, p, p, p, p, p, p, p, p, 0, None) == NULL
    for o, want in (({"batch": -1}, SHAPE), ({"V": 0}, SHAPE), ({"rows_": -1}, SHAPE), ({"dtype": 2}, ARGUMENT),
                    ({"dtype": -1}, ARGUMENT), ({"batch": (1 << 20) + 1}, UNSUPPORTED), ({"V": (1 << 22) + 1}, UNSUPPORTED)):
        a = dict(batch=2, V=100, rows_=3, dtype=0)
        a.update(o)
        assert size_of(f, SampleDesc(*a.values(), 1.0, 0, 1.0, 0.0))[0] == want and call(**o) == want, o
    assert call(stride=-1) == SHAPE and call(stride=(1 << 31) + 1) == SHAPE
    assert call(batch=4, rows=None) == SHAPE                        # more draws than rows
    assert call(batch=0, z=None, noise=None, ws=None, bytes_=0) == OK
    assert call(tok=None, probs=None, z=None, ws=None, bytes_=0) == OK
    assert call(z=None) == NULL and call(noise=None) == NULL and call(ws=None) == NULL
    # no noise is needed where the settings of all draws leave one token, or none is drawn
    for o in ({"t": None, "T": 0.0}, {"t": None, "T": float("nan")}, {"ks": None, "k": 1}, {"ps": None, "top_p": 0.0},
              {"tok": None}):
        assert call(noise=None, bytes_=0, **o) == SMALL, o
    assert call(noise=None, T=0.0, k=1, top_p=0.0) == NULL          # (arrays are given: they count)
    for o in ({"z": p + 1}, {"rows": p + 2}, {"noise": p + 1}, {"t": p + 2}, {"ks": p + 2}, {"ps": p + 2}, {"ms": p + 2},
              {"tok": p + 2}, {"probs": p + 2}, {"ws": p + 8}):
        assert call(**o) == MISALIGNED, o
    assert call(dtype=1, z=p + 2) == MISALIGNED
    st, need = size_of(f, SampleDesc(2, 100, 3, 0, 1.0, 0, 1.0, 0.0))
    assert st == OK and need > HEADER and call(bytes_=need - 1) == SMALL


def test_sample_workspaces_stay_bounded(lib):
    """A large batch goes in groups: its workspace does not grow with it."""
    f = lib.spear_sample_workspace_bytes
    assert size_of(f, SampleDesc(0, 100, 3, 0, 1.0, 0, 1.0, 0.0)) == (OK, 0)
    for V in (1, 1000, 50257, 128001, 1 << 22):
        st, most = size_of(f, SampleDesc(1 << 20, V, 1, 0, 1.0, 0, 1.0, 0.0))
        assert st == OK and HEADER < most < (2 << 30)
        for batch in (1, 7, 64, 1000):
            st, need = size_of(f, SampleDesc(batch, V, 1, 1, 1.0, 0, 1.0, 0.0))
            assert st == OK and HEADER < need <= most, (batch, V)


def test_sample_workspaces_hold_only_what_leaves_a_workgroup(lib):
    """A row of one share (up to 16384 tokens) has its bins in LDS, one of one part (up to
    4096) its list too: neither has a place in the workspace.  The groups of rows that go
    together bound the rest: 4096 shares' bins, and a list of 48 KiB a row."""
    f = lib.spear_sample_workspace_bytes
    size = lambda batch, V: size_of(f, SampleDesc(batch, V, batch, 0, 1.0, 0, 1.0, 0.0))[1] - HEADER  # noqa: E731
    for V in (1, 40, 1000, 4096):
        assert size(1000, V) <= 1000 * 512 and size(1 << 20, V) <= 4096 * 512
    for V in (4097, 8000):                                      # (1000 rows of these go as single shares)
        assert 1000 * (48 << 10) < size(1000, V) < 1000 * (49 << 10)
    for V in (32000, 128001, 1 << 22):
        assert size(1 << 20, V) < 4096 * ((32 << 10) + (48 << 10) + 1024) + (1 << 20)


def documented_rows(text):
    """The expression that a document's usage gives spear_sample for its rows: the argument
    itself, or what the variable of that name is set to."""
    call = re.search(r"sp\.spear_sample\((.*?)\n```", text, re.S).group(1)
    given = re.search(r"\brows=(.*?), \w+=", re.sub(r" #.*", "", call)).group(1)
    found = re.search(r"^%s = (.*?)(?: +#.*)?$" % re.escape(given), text, re.M)
    return found.group(1) if found else given


def test_documented_rows_leave_out_sequences_without_tokens(repo_root):
    """Sequences that a plan gives nothing (they wait, have ended, or found no pages) own no
    row of the logits: the usage shown maps them outside, not to a neighbour's row."""
    with open(os.path.join(repo_root, "README.md")) as f:
        rows = documented_rows(f.read())
    for n in ([1, 0, 2], [0, 0, 1, 1, 0], [0], [3, 4, 5], [2, 0, 0]):
        cu_q = torch.tensor([0] + n, dtype=torch.int32).cumsum(0, dtype=torch.int32)
        got = eval(rows, {"torch": torch, "cu_q": cu_q})
        assert got.dtype == torch.int32
        assert got.tolist() == [sum(n[:b + 1]) - 1 if n[b] else -1 for b in range(len(n))]
