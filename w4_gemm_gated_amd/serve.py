"""Serving operators beside the W4 linear layer: a paged key/value cache (fp16
or 8-bit), attention of new tokens over it, and the verification of drafted
tokens.

Python names mirror the C ABI in include/spear_serve.h, which states the
definitions.  As in the package's other wrappers only arguments are
marshalled here: every step runs in the HIP kernels of libspear_w4ec.so on the
current stream.

The cache is four tensors that the caller owns:
    k_cache, v_cache   [num_pages, kv_heads, page_size, head_dim], fp16 or int8
    k_scale, v_scale   fp32 [num_pages, kv_heads, page_size] with int8, else None
"""
import ctypes
import math

import torch

import w4_gemm_gated_amd as _pkg

from . import _binding
from ._binding import AttentionDesc, KvDesc, VerifyDesc

__all__ = ["spear_kv_cache", "spear_kv_append", "spear_kv_gather", "spear_paged_attention", "spear_verify_draft"]

_KV_DTYPES = {torch.float16: 0, torch.int8: 1}


def _refuse(t, name, dtype, dims, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    raise ValueError(f"{name} must be contiguous")


# Small calls take about as long on the host as on the GPU: the checks look at
# each tensor once, and only a failing one asks what is wrong with it.
def _check(t, name, dtype, dims, device):
    """A GPU tensor of this type."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == dims and t.device == device):
        _refuse(t, name, dtype, dims, device)


def _dense(t, name, dtype, dims, device):
    """.. that is contiguous."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == dims and t.device == device
            and t.is_contiguous()):
        _refuse(t, name, dtype, dims, device)


def _rows(t, name, dtype, device):
    """A 3-D tensor whose last dimension is contiguous: its first two strides."""
    _check(t, name, dtype, 3, device)
    s0, s1, s2 = t.stride()
    if s2 != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return s0, s1


def _kv_desc(k_cache, v_cache, k_scale, v_scale):
    """The cache's (type, num_pages, kv_heads, page_size, head_dim), its device, and
    its tensors' addresses."""
    if not isinstance(k_cache, torch.Tensor) or not k_cache.is_cuda:
        raise ValueError("k_cache must be a GPU tensor")
    dev, dt = k_cache.device, k_cache.dtype
    if dt not in _KV_DTYPES:
        raise TypeError(f"k_cache must be torch.float16 or torch.int8, got {dt}")
    _dense(k_cache, "k_cache", dt, 4, dev)
    _dense(v_cache, "v_cache", dt, 4, dev)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    at = (k_cache.data_ptr(), v_cache.data_ptr(), None, None)
    if dt is torch.int8:
        for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if s is None:
                raise ValueError(f"{name} must be given with an int8 cache")
            _dense(s, name, torch.float32, 3, dev)
            if s.shape != shape[:3]:
                raise ValueError(f"{name} must be [num_pages, kv_heads, page_size]")
        at = (at[0], at[1], k_scale.data_ptr(), v_scale.data_ptr())
    return (_KV_DTYPES[dt], *shape), dev, at


def _p(t):
    return t.data_ptr() if t is not None else None


# torch.cuda.current_stream() makes an object of the stream; only its handle is
# needed, which this gives in a thirtieth of the time where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device):
    index = device.index
    if index != torch.cuda.current_device():
        _pkg._on_current(device)                # refuses
    return _raw_stream(index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream


# What follows from a call's sizes alone is made once for them: the descriptor
# (never written to again), and the bytes of workspace that it needs.
_plans = {}


def _plan(key, make):
    p = _plans.get(key)
    if p is None:
        if len(_plans) >= 4096:
            _plans.clear()
        d, ask, where = make()
        nb = ctypes.c_size_t(0)
        if ask is not None:
            _binding.check(ask(ctypes.byref(d), ctypes.byref(nb)), where)
        p = _plans[key] = (d, ctypes.byref(d), nb.value)
    return p


def _kv_struct(kv):
    return KvDesc(kv[0], kv[1], kv[2], kv[4], kv[3])


def _scratch(n, device, stream):
    """The cached workspace of the stream, as the linear layer's."""
    if n == 0:
        return None
    ws = _pkg._workspaces.get((device.index, stream))
    return ws if ws is not None and ws.numel() >= n else _pkg._workspace(n, device)


def spear_kv_cache(num_pages, kv_heads, head_dim, page_size=16, dtype=torch.float16, device="cuda"):
    """Zeroed cache tensors (k_cache, v_cache, k_scale, v_scale); the scales are
    None with fp16."""
    shape = (num_pages, kv_heads, page_size, head_dim)
    k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
    if dtype is not torch.int8:
        return k, v, None, None
    ks, vs = (torch.zeros(shape[:3], dtype=torch.float32, device=device) for _ in range(2))
    return k, v, ks, vs


def spear_kv_append(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None):
    """Write new tokens into the cache in place.

    k, v fp16 [T, kv_heads, head_dim] (last dimension contiguous, e.g. parts of
    a joint projection); slots int64 [T]: page * page_size + place, or -1 for
    rows that are not written.
    """
    kv, dev, at = _kv_desc(k_cache, v_cache, k_scale, v_scale)
    kt, kh = _rows(k, "k", torch.float16, dev)
    vt, vh = _rows(v, "v", torch.float16, dev)
    _dense(slots, "slots", torch.int64, 1, dev)
    T = slots.shape[0]
    if k.shape != (T, kv[2], kv[4]) or v.shape != k.shape:
        raise ValueError("k and v must be [T, kv_heads, head_dim] with T slots")
    d = _plan(kv, lambda: (_kv_struct(kv), None, None))
    st = _binding.load().spear_kv_append(d[1], T, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh,
                                         slots.data_ptr(), *at, _stream(dev))
    _binding.check(st, "spear_kv_append")


def spear_kv_gather(k_cache, v_cache, block_table, cu_kv, rows, k_scale=None, v_scale=None, k_out=None, v_out=None):
    """(k, v) fp16 [rows, kv_heads, head_dim]: rows cu_kv[b] .. cu_kv[b + 1] - 1
    are sequence b's cached tokens in order; rows past the last are zero.

    block_table int32 [B, max_pages]; cu_kv int32 [B + 1].
    """
    kv, dev, at = _kv_desc(k_cache, v_cache, k_scale, v_scale)
    _dense(block_table, "block_table", torch.int32, 2, dev)
    _dense(cu_kv, "cu_kv", torch.int32, 1, dev)
    B, rows = block_table.shape[0], int(rows)
    if cu_kv.shape[0] != B + 1:
        raise ValueError("cu_kv must have one entry more than block_table has rows")
    shape = (rows, kv[2], kv[4])
    out = []
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        if t is None:
            t = torch.empty(shape, dtype=torch.float16, device=dev)
        else:
            _dense(t, name, torch.float16, 3, dev)
            if t.shape != shape:
                raise ValueError(f"{name} must be [rows, kv_heads, head_dim]")
        out.append(t)
    d = _plan(kv, lambda: (_kv_struct(kv), None, None))
    st = _binding.load().spear_kv_gather(d[1], B, rows, block_table.data_ptr(), block_table.shape[1],
                                         cu_kv.data_ptr(), *at, out[0].data_ptr(), out[1].data_ptr(), _stream(dev))
    _binding.check(st, "spear_kv_gather")
    return out[0], out[1]


def spear_paged_attention(q, k_cache, v_cache, block_table, cu_q, kv_lens, max_q, scale=None, k_scale=None,
                          v_scale=None, out=None, workspace=None):
    """out fp16 [total_q, q_heads, head_dim]: attention of every sequence's new
    tokens over its cached ones, causal within the new tokens.

    q fp16 [total_q, q_heads, head_dim] (last dimension contiguous); cu_q int32
    [B + 1]: rows of sequence b; kv_lens int32 [B]: its cached tokens, the new
    ones among them; block_table int32 [B, max_pages]; max_q: the longest
    sequence's new tokens; scale defaults to 1 / sqrt(head_dim).  `workspace`
    (uint8, zero-filled before first use) defaults to the cached one of the current
    stream, as spear_w4ec_linear's, also under graph capture.
    """
    kv, dev, at = _kv_desc(k_cache, v_cache, k_scale, v_scale)
    qt, qh = _rows(q, "q", torch.float16, dev)
    _dense(block_table, "block_table", torch.int32, 2, dev)
    _dense(cu_q, "cu_q", torch.int32, 1, dev)
    _dense(kv_lens, "kv_lens", torch.int32, 1, dev)
    B, pages = block_table.shape
    total, heads, dim = q.shape
    if dim != kv[4] or kv_lens.shape[0] != B or cu_q.shape[0] != B + 1:
        raise ValueError("need q [total_q, q_heads, head_dim], block_table [B, max_pages], cu_q [B + 1], kv_lens [B]")
    if out is None:
        out = torch.empty((total, heads, dim), dtype=torch.float16, device=dev)
    else:
        _dense(out, "out", torch.float16, 3, dev)
        if out.shape != q.shape:
            raise ValueError("out must have the shape of q")
    if B == 0 or total == 0:
        return out
    lib, stream = _binding.load(), _stream(dev)
    max_q, scale = int(max_q), 1.0 / math.sqrt(dim) if scale is None else float(scale)
    d = _plan((kv, dev.index, B, total, max_q, pages, heads, scale), lambda: (
        AttentionDesc(_kv_struct(kv), B, total, max_q, pages, heads, scale, 0),
        lib.spear_attention_workspace_bytes, "spear_paged_attention"))
    if workspace is None:
        workspace = _scratch(d[2], dev, stream)
    else:
        _dense(workspace, "workspace", torch.uint8, 1, dev)
    st = lib.spear_paged_attention(d[1], q.data_ptr(), qt, qh, cu_q.data_ptr(), kv_lens.data_ptr(),
                                   block_table.data_ptr(), pages, *at, out.data_ptr(), workspace.data_ptr(),
                                   workspace.numel(), stream)
    _binding.check(st, "spear_paged_attention")
    return out


def spear_verify_draft(target, draft, drafted, u, noise, num_drafts=None, accepted=None, tokens=None, workspace=None):
    """(accepted int32 [B], tokens int32 [B, K + 1]): the number of drafted tokens
    kept, and the kept tokens followed by the drawn one and then -1.

    target fp32 [B, K + 1, V] and draft fp32 [B, K, V]: probabilities (last
    dimension contiguous), draft None where each drafted token was certain;
    drafted int32 [B, K]; u fp32 [B, K] uniform in [0, 1); noise fp32 [B, V] from
    Exp(1); num_drafts int32 [B] or None (K each); `workspace` as in
    spear_paged_attention.
    """
    if not isinstance(target, torch.Tensor) or not target.is_cuda:
        raise ValueError("target must be a GPU tensor")
    dev = target.device
    tb, tr = _rows(target, "target", torch.float32, dev)
    B, K1, V = target.shape
    K = K1 - 1
    if K < 0:
        raise ValueError("target must be [B, K + 1, V]")
    db = dr = 0
    if draft is not None:
        db, dr = _rows(draft, "draft", torch.float32, dev)
        if draft.shape != (B, K, V):
            raise ValueError("draft must be [B, K, V] for target [B, K + 1, V]")
    _dense(drafted, "drafted", torch.int32, 2, dev)
    _dense(u, "u", torch.float32, 2, dev)
    _dense(noise, "noise", torch.float32, 2, dev)
    if drafted.shape != (B, K) or u.shape != (B, K) or noise.shape != (B, V):
        raise ValueError("need drafted [B, K], u [B, K], noise [B, V] for target [B, K + 1, V]")
    if num_drafts is not None:
        _dense(num_drafts, "num_drafts", torch.int32, 1, dev)
        if num_drafts.shape[0] != B:
            raise ValueError("num_drafts must be [B]")
    for t, name, shape in ((accepted, "accepted", (B,)), (tokens, "tokens", (B, K1))):
        if t is not None:
            _dense(t, name, torch.int32, len(shape), dev)
            if t.shape != shape:
                raise ValueError(f"{name} must be {list(shape)}")
    accepted = torch.empty(B, dtype=torch.int32, device=dev) if accepted is None else accepted
    tokens = torch.empty((B, K1), dtype=torch.int32, device=dev) if tokens is None else tokens
    lib, stream = _binding.load(), _stream(dev)
    d = _plan(("verify", dev.index, B, K, V),
              lambda: (VerifyDesc(B, K, V, 0), lib.spear_verify_workspace_bytes, "spear_verify_draft"))
    if workspace is None:
        workspace = _scratch(d[2], dev, stream)
    else:
        _dense(workspace, "workspace", torch.uint8, 1, dev)
    st = lib.spear_verify_draft(d[1], target.data_ptr(), tb, tr, _p(draft), db, dr, drafted.data_ptr(),
                                u.data_ptr(), noise.data_ptr(), _p(num_drafts), accepted.data_ptr(),
                                tokens.data_ptr(), _p(workspace), workspace.numel() if workspace is not None else 0,
                                stream)
    _binding.check(st, "spear_verify_draft")
    return accepted, tokens
