"""What a serving step does around the W4 layers and the paged cache: its pages,
block tables and slots planned on the GPU, the low-rank adapters of its requests
added beside a shared projection, and the draw of its next tokens.

Python names mirror the C ABI in include/spear_serve.h, which states the
definitions; only arguments are marshalled here, as in serve.py.
"""
import ctypes
import functools

import torch

from . import _binding
from ._binding import AdapterDesc, KvPlanDesc, SampleDesc
from .serve import _check, _dense, _p, _plan, _scratch, _stream

__all__ = ["spear_kv_plan", "spear_adapter_plan", "spear_adapter_add", "spear_sample"]


def _out(t, name, shape, dtype, device):
    """The caller's output tensor, or a new one."""
    if t is None:
        return torch.empty(shape if len(shape) > 1 else shape[0], dtype=dtype, device=device)
    _dense(t, name, dtype, len(shape), device)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}")
    return t


def _gpu(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.device


def _space(workspace, nbytes, device, stream):
    """(address, bytes) of the caller's workspace, or of the stream's cached one."""
    if workspace is None:
        workspace = _scratch(nbytes, device, stream)
    else:
        _dense(workspace, "workspace", torch.uint8, 1, device)
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())


_PLANNED = ("cu_q", "kv_lens", "positions", "sequence", "held_out", "free_out")


def spear_kv_plan(lens, new_tokens, held, block_table, free_pages, free_count, rows, page_size=16, cu_q=None,
                  kv_lens=None, slots=None, positions=None, sequence=None, held_out=None, free_out=None,
                  workspace=None):
    """(cu_q [B + 1], kv_lens [B], slots int64 [rows], positions [rows], sequence
    [rows], held [B], free_count [1]) of a step in which sequence b, with lens[b]
    cached tokens in held[b] pages, gets new_tokens[b] more as far as pages and
    rows last; pages that it no longer needs are laid on the stack of free ones.

    lens, new_tokens, held int32 [B]; block_table int32 [B, max_pages] (updated in
    place); free_pages int32 [any] with free_count int32 [1] entries used, the stack
    of free pages (updated in place); rows: the most new tokens that the step may
    have.  Outputs are int32 where nothing else is said and may be given; kv_lens,
    held_out and free_out may be lens, held and free_count themselves.  Rows past the
    last new token hold -1.  `workspace` as in spear_paged_attention.
    """
    dev = _gpu(lens, "lens")
    i32 = torch.int32
    _dense(lens, "lens", i32, 1, dev)
    _dense(new_tokens, "new_tokens", i32, 1, dev)
    _dense(held, "held", i32, 1, dev)
    _dense(block_table, "block_table", i32, 2, dev)
    _dense(free_pages, "free_pages", i32, 1, dev)
    _dense(free_count, "free_count", i32, 1, dev)
    B, pages = block_table.shape
    if lens.numel() != B or new_tokens.numel() != B or held.numel() != B or free_count.numel() != 1:
        raise ValueError("need lens, new_tokens and held [B], block_table [B, max_pages], free_count [1]")
    rows = int(rows)
    if rows < 0:
        raise ValueError("rows must not be negative")
    if slots is None:
        slots = torch.empty(rows, dtype=torch.int64, device=dev)
    else:
        _out(slots, "slots", (rows,), torch.int64, dev)
    given = (cu_q, kv_lens, positions, sequence, held_out, free_out)
    sizes = (B + 1, B, rows, rows, B, 1)
    if cu_q is kv_lens is positions is sequence is held_out is free_out is None:     # (one allocation, a microsecond each)
        given = torch.empty(sum(sizes), dtype=i32, device=dev).unsafe_split_with_sizes(sizes)
    else:
        given = [_out(t, name, (n,), i32, dev) for t, name, n in zip(given, _PLANNED, sizes)]
    cu_q, kv_lens, positions, sequence, held_out, free_out = given
    lib, stream = _binding.load(), _stream(dev)
    page_size, free_slots = int(page_size), free_pages.numel()
    d = _plan(("kv_plan", B, rows, pages, page_size, free_slots), lambda: (
        KvPlanDesc(B, rows, pages, page_size, free_slots), lib.spear_kv_plan_workspace_bytes, "spear_kv_plan"))
    ws = _space(workspace, d[2], dev, stream)
    st = lib.spear_kv_plan(d[1], lens.data_ptr(), new_tokens.data_ptr(), held.data_ptr(), block_table.data_ptr(), pages,
                           free_pages.data_ptr(), free_count.data_ptr(), cu_q.data_ptr(), kv_lens.data_ptr(),
                           slots.data_ptr(), positions.data_ptr(), sequence.data_ptr(), held_out.data_ptr(),
                           free_out.data_ptr(), *ws, stream)
    _binding.check(st, "spear_kv_plan")
    return cu_q, kv_lens, slots, positions, sequence, held_out, free_out


class AdapterPlan:
    """The rows of a batch by adapter: what spear_adapter_plan makes for a step and
    spear_adapter_add reads."""
    __slots__ = ("data", "device", "batch", "adapters", "rows")

    def __init__(self, data, batch, adapters, rows):
        self.data, self.device, self.batch, self.adapters, self.rows = data, data.device, batch, adapters, rows


@functools.lru_cache(maxsize=4096)
def _plan_bytes(batch, adapters, rows):
    n = ctypes.c_size_t(0)
    _binding.check(_binding.load().spear_adapter_plan_bytes(batch, adapters, rows, ctypes.byref(n)), "spear_adapter_plan")
    return n.value


def spear_adapter_plan(cu_q, adapter, adapters, rows, plan=None):
    """The plan of a step's adapters: sequence b has rows cu_q[b] .. cu_q[b + 1] - 1 and
    adapter adapter[b] (outside [0, adapters): none).

    cu_q int32 [B + 1], rising from 0 to at most rows; adapter int32 [B].  `plan`: one
    of the same sizes to be filled again (a captured graph's).
    """
    dev = _gpu(cu_q, "cu_q")
    _dense(cu_q, "cu_q", torch.int32, 1, dev)
    _dense(adapter, "adapter", torch.int32, 1, dev)
    B, adapters, rows = adapter.numel(), int(adapters), int(rows)
    if cu_q.numel() != B + 1:
        raise ValueError("cu_q must have one entry more than adapter")
    lib, stream = _binding.load(), _stream(dev)
    if plan is None:
        plan = AdapterPlan(torch.empty(_plan_bytes(B, adapters, rows), dtype=torch.uint8, device=dev), B, adapters, rows)
    elif not isinstance(plan, AdapterPlan):
        raise TypeError("plan must come from spear_adapter_plan")
    elif (plan.batch, plan.adapters, plan.rows) != (B, adapters, rows) or plan.device != dev:
        raise ValueError("plan was made for other sizes")
    st = lib.spear_adapter_plan(B, adapters, rows, cu_q.data_ptr(), adapter.data_ptr(), plan.data.data_ptr(),
                                plan.data.numel(), stream)
    _binding.check(st, "spear_adapter_plan")
    return plan


def spear_adapter_add(Y, X, A, B, plan, scale=None, workspace=None):
    """Y fp16 [rows, N], updated in place and returned: each row of a sequence with
    adapter a gets scale[a] * (X . A[a]^T) . B[a]^T more.

    X fp16 [rows, K]; A fp16 [adapters, rank, K]; B fp16 [adapters, N, rank]; X's and
    Y's last dimension contiguous (Y may be a part of a joint projection's output);
    scale fp32 [adapters] or None (1); plan from spear_adapter_plan; `workspace` as in
    spear_paged_attention.
    """
    dev = _gpu(Y, "Y")
    f16 = torch.float16
    _check(Y, "Y", f16, 2, dev)
    _check(X, "X", f16, 2, dev)
    _dense(A, "A", f16, 3, dev)
    _dense(B, "B", f16, 3, dev)
    if not isinstance(plan, AdapterPlan):
        raise TypeError("plan must come from spear_adapter_plan")
    if plan.device != dev:
        raise ValueError(f"plan must be on {dev}")
    n, rank, K = A.shape
    rows, N = Y.shape
    if B.shape != (n, N, rank) or X.shape != (rows, K) or plan.adapters != n or plan.rows != rows:
        raise ValueError("need Y [rows, N], X [rows, K], A [adapters, rank, K], B [adapters, N, rank] and a plan of "
                         "these rows and adapters")
    (xs, x1), (ys, y1) = X.stride(), Y.stride()
    if (x1 != 1 and K > 1) or (y1 != 1 and N > 1):
        raise ValueError("X and Y must be contiguous in their last dimension")
    if scale is not None:
        _dense(scale, "scale", torch.float32, 1, dev)
        if scale.numel() != n:
            raise ValueError("scale must be [adapters]")
    lib, stream = _binding.load(), _stream(dev)
    d = _plan(("adapter", dev.index, plan.batch, n, rows, K, N, rank), lambda: (
        AdapterDesc(plan.batch, n, rows, K, N, rank, 0), lib.spear_adapter_workspace_bytes, "spear_adapter_add"))
    ws = _space(workspace, d[2], dev, stream)
    if rows == 1:       # (the strides of a single row say nothing)
        xs, ys = K, N
    st = lib.spear_adapter_add(d[1], X.data_ptr(), xs, A.data_ptr(), B.data_ptr(), _p(scale), plan.data.data_ptr(),
                               plan.data.numel(), Y.data_ptr(), ys, *ws, stream)
    _binding.check(st, "spear_adapter_add")
    return Y


_LOGITS = {torch.float16: 0, torch.float32: 1}


def _setting(x, name, dtype, batch, device):
    """(address, value for all): an array of a value for each draw, or one for all."""
    if not isinstance(x, torch.Tensor):
        return None, x
    _dense(x, name, dtype, 1, device)
    if x.shape[0] != batch:
        raise ValueError(f"{name} must have an entry for each draw")
    return x.data_ptr(), 0


# The last call's descriptor (never written to again): what a call needs beside it follows
# from its sizes alone, and settings may change from one to the next.
_last = ((), None)


def _with_settings(fields):
    global _last
    last = _last
    if last[0] != fields:
        _last = last = (fields, ctypes.byref(SampleDesc(*fields)))
    return last[1]


def spear_sample(logits, noise=None, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, rows=None, probs=False,
                 tokens=None, workspace=None):
    """(tokens int32 [B], probs fp32 [B, V]): one token drawn for each row of the
    logits, and the distribution that it is drawn from.

    logits fp16 or fp32 [R, V] (last dimension contiguous); rows int32 [B]: the row of
    each draw, or None: all in order (outside [0, R): token -1 and no distribution, for
    sequences that a plan gave no rows); noise fp32 [B, V] from Exp(1): None if no tokens
    are wanted (tokens is then None, unless the settings below, given as numbers,
    leave a single token).  Settings are numbers, or a tensor [B] with one for each
    draw: temperature (0: the largest logit's token), top_k (int32; 0: off), top_p
    (1: off), min_p (0: off).  probs: True, or the tensor to be filled, for the
    distribution; else None is returned.  `workspace` as in spear_paged_attention.
    """
    dev = _gpu(logits, "logits")
    dt = logits.dtype
    if dt not in _LOGITS:
        raise TypeError(f"logits must be torch.float16 or torch.float32, got {dt}")
    _check(logits, "logits", dt, 2, dev)
    R, V = logits.shape
    if logits.stride(1) != 1 and V > 1:
        raise ValueError("logits must be contiguous in its last dimension")
    B = R
    if rows is not None:
        _dense(rows, "rows", torch.int32, 1, dev)
        B = rows.shape[0]
    if noise is not None:
        _dense(noise, "noise", torch.float32, 2, dev)
        if noise.shape != (B, V):
            raise ValueError("noise must be [B, V]")
    f32 = torch.float32
    t_at, t = _setting(temperature, "temperature", f32, B, dev)
    k_at, k = _setting(top_k, "top_k", torch.int32, B, dev)
    p_at, p = _setting(top_p, "top_p", f32, B, dev)
    m_at, m = _setting(min_p, "min_p", f32, B, dev)
    t, k, p, m = float(t), min(max(int(k), 0), V), float(p), float(m)
    one = (t_at is None and not t > 0) or (k_at is None and k == 1) or (p_at is None and p <= 0)
    if noise is not None or one or tokens is not None:
        tokens = _out(tokens, "tokens", (B,), torch.int32, dev)
    if probs is True or isinstance(probs, torch.Tensor):
        probs = _out(None if probs is True else probs, "probs", (B, V), f32, dev)
    else:
        probs = None
    lib, stream = _binding.load(), _stream(dev)
    d = _plan(("sample", B, V, R, dt), lambda: (
        SampleDesc(B, V, R, _LOGITS[dt], 0.0, 0, 0.0, 0.0), lib.spear_sample_workspace_bytes, "spear_sample"))
    ws = _space(workspace, d[2], dev, stream)
    st = lib.spear_sample(_with_settings((B, V, R, _LOGITS[dt], t, k, p, m)), logits.data_ptr(), V if R == 1 else logits.stride(0), _p(rows), _p(noise), t_at, k_at,
                          p_at, m_at, _p(tokens), _p(probs), *ws, stream)
    _binding.check(st, "spear_sample")
    return tokens, probs
