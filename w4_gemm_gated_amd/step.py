"""What a serving step does around the W4 layers and the paged cache: its pages,
block tables and slots planned on the GPU.

Python names mirror the C ABI in include/spear_serve.h, which states the
definitions; only arguments are marshalled here, as in serve.py.
"""
import torch

from . import _binding
from ._binding import KvPlanDesc
from .serve import _dense, _p, _plan, _scratch, _stream

__all__ = ["spear_kv_plan"]


def _out(t, name, shape, dtype, device):
    """The caller's output tensor, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
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
    if lens.shape[0] != B or new_tokens.shape[0] != B or held.shape[0] != B or free_count.shape[0] != 1:
        raise ValueError("need lens, new_tokens and held [B], block_table [B, max_pages], free_count [1]")
    rows = int(rows)
    if rows < 0:
        raise ValueError("rows must not be negative")
    cu_q = _out(cu_q, "cu_q", (B + 1,), i32, dev)
    kv_lens = _out(kv_lens, "kv_lens", (B,), i32, dev)
    slots = _out(slots, "slots", (rows,), torch.int64, dev)
    positions = _out(positions, "positions", (rows,), i32, dev)
    sequence = _out(sequence, "sequence", (rows,), i32, dev)
    held_out = _out(held_out, "held_out", (B,), i32, dev)
    free_out = _out(free_out, "free_out", (1,), i32, dev)
    lib, stream = _binding.load(), _stream(dev)
    d = _plan(("kv_plan", B, rows, pages, int(page_size), free_pages.shape[0]), lambda: (
        KvPlanDesc(B, rows, pages, int(page_size), free_pages.shape[0]), lib.spear_kv_plan_workspace_bytes,
        "spear_kv_plan"))
    ws = _space(workspace, d[2], dev, stream)
    st = lib.spear_kv_plan(d[1], lens.data_ptr(), new_tokens.data_ptr(), held.data_ptr(), block_table.data_ptr(), pages,
                           free_pages.data_ptr(), free_count.data_ptr(), cu_q.data_ptr(), kv_lens.data_ptr(),
                           slots.data_ptr(), positions.data_ptr(), sequence.data_ptr(), held_out.data_ptr(),
                           free_out.data_ptr(), *ws, stream)
    _binding.check(st, "spear_kv_plan")
    return cu_q, kv_lens, slots, positions, sequence, held_out, free_out
