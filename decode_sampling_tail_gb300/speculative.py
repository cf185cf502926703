"""Verification of drafted tokens on torch CUDA tensors (tail_verify, tail_verify_logits).

A speculative decode step runs the tail on the rows of the drafted positions
(``Tail.run`` with ``params=None``, its top-k or its logits as outputs) and then
calls one of these: which drafts stand, and the token after them.  ``include/tail.h``
states the rule.

The tensors are checked here (type, shape, device, contiguity; ValueError); the
library checks sizes and pointers.  Calls are asynchronous on ``stream`` (None: the
current stream of the tensors' device).
"""
from __future__ import annotations

import contextlib
import ctypes

from . import TAIL_BF16, TAIL_ERR_UNSUPPORTED, TAIL_F16, TAIL_F32, TAIL_OK, TailError, _ptr, _stream_ptr, lib


def _dtype_code(t, what):
    import torch
    codes = {torch.float32: TAIL_F32, torch.float16: TAIL_F16, torch.bfloat16: TAIL_BF16}
    if t.dtype not in codes:
        raise ValueError(f"{what} must be float32, float16 or bfloat16, not {t.dtype}")
    return codes[t.dtype]


def _need(t, what, dtype, shape, device):
    """A contiguous tensor of this type and shape on this device."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}; "
                         f"got {t.dtype}, {tuple(t.shape)}, strides {t.stride()}, {t.device}")


def _need_matrix(t, what, rows, device):
    """[rows, n] with unit stride along the columns; returns (n, leading dimension)."""
    if t.dim() != 2 or int(t.shape[0]) != rows or t.device != device or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be [{rows}, n] on {device} with contiguous rows; got {tuple(t.shape)}, "
                         f"strides {t.stride()}, {t.device}")
    n = int(t.shape[1])
    if rows > 1 and t.stride(0) < n:
        raise ValueError(f"{what}: rows overlap (strides {t.stride()})")
    return n, int(t.stride(0)) if rows > 1 else n


def _on(device, stream):
    """Makes `device` current and the call's stream the one that allocations belong to."""
    import torch
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(device))
    if stream is not None:
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=device)
        stack.enter_context(torch.cuda.stream(stream))
    return stack


def _sequences(cu_rows, drafts, u_accept, rows, device):
    import torch
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a CUDA device, not {device}")
    if cu_rows.dim() != 1 or cu_rows.shape[0] < 1:
        raise ValueError("cu_rows must be [nseq + 1]")
    _need(cu_rows, "cu_rows", torch.int32, cu_rows.shape, device)
    _need(drafts, "drafts", torch.int32, (rows,), device)
    _need(u_accept, "u_accept", torch.float32, (rows,), device)
    return int(cu_rows.shape[0]) - 1


def _outputs(out_tokens, out_count, rows, nseq, device):
    import torch
    if out_tokens is None:
        out_tokens = torch.full((rows,), -1, dtype=torch.int32, device=device)
    if out_count is None:
        out_count = torch.empty((nseq,), dtype=torch.int32, device=device)
    _need(out_tokens, "out_tokens", torch.int32, (rows,), device)
    _need(out_count, "out_count", torch.int32, (nseq,), device)
    return out_tokens, out_count


def _fail(rc, what):
    if rc == TAIL_ERR_UNSUPPORTED:
        raise TailError(rc, what + " [" + lib().tail_last_error().decode() + "]")
    if rc != TAIL_OK:
        raise TailError(rc, what)


def verify(topk_vals, topk_idx, params, cu_rows, drafts, u_accept, draft_probs=None, out_tokens=None,
           out_count=None, stream=None):
    """Drafts against the tail's sorted top-k (tail_verify).

    topk_vals [rows, k] float32 and topk_idx [rows, k] int32 as the tail writes them, params [rows, 3|4]
    float32, cu_rows [nseq + 1] int32, drafts [rows] int32, u_accept [rows] float32, draft_probs [rows, V]
    float32, float16 or bfloat16 (rows may be strided) or None.  Returns (out_tokens [rows] int32, out_count
    [nseq] int32), allocated when not given."""
    import torch
    device = topk_vals.device
    rows, k = (int(d) for d in topk_vals.shape)
    nseq = _sequences(cu_rows, drafts, u_accept, rows, device)
    _need(topk_vals, "topk_vals", torch.float32, (rows, k), device)
    _need(topk_idx, "topk_idx", torch.int32, (rows, k), device)
    if params.dim() != 2 or int(params.shape[1]) not in (3, 4):
        raise ValueError("params must be [rows, 3] or [rows, 4]")
    _need(params, "params", torch.float32, (rows, int(params.shape[1])), device)
    V, ld, code = 0, 0, TAIL_F32
    if draft_probs is not None:
        code = _dtype_code(draft_probs, "draft_probs")
        V, ld = _need_matrix(draft_probs, "draft_probs", rows, device)
    with _on(device, stream):
        out_tokens, out_count = _outputs(out_tokens, out_count, rows, nseq, device)
        rc = lib().tail_verify(rows, nseq, k, _ptr(topk_vals), _ptr(topk_idx), _ptr(params), int(params.shape[1]),
                               _ptr(cu_rows), _ptr(drafts), _ptr(u_accept), _ptr(draft_probs), code, ld, V,
                               _ptr(out_tokens), _ptr(out_count), _stream_ptr(stream, device))
    _fail(rc, "tail_verify")
    return out_tokens, out_count


def verify_logits_workspace(rows: int, nseq: int, V: int) -> int:
    """Bytes of workspace that ``verify_logits`` needs for these sizes."""
    n = ctypes.c_int64()
    _fail(lib().tail_verify_logits_workspace(rows, nseq, V, ctypes.byref(n)), "tail_verify_logits_workspace")
    return n.value


def verify_logits(logits, temperature, cu_rows, drafts, u_accept, u_draw, draft_probs=None, out_tokens=None,
                  out_count=None, workspace=None, stream=None):
    """Drafts against softmax(logits / temperature) over the whole vocabulary (tail_verify_logits).

    logits [rows, V] float32, float16 or bfloat16 (rows may be strided), temperature, u_accept and u_draw [rows]
    float32, cu_rows [nseq + 1] and drafts [rows] int32, draft_probs [rows, V] of any of the three types or None.
    ``workspace``: a uint8 tensor of at least ``verify_logits_workspace(rows, nseq, V)`` bytes that no call which
    may overlap this one uses; allocated when not given.  Returns (out_tokens [rows], out_count [nseq])."""
    import torch
    device = logits.device
    rows = int(logits.shape[0])
    nseq = _sequences(cu_rows, drafts, u_accept, rows, device)
    code = _dtype_code(logits, "logits")
    V, ld = _need_matrix(logits, "logits", rows, device)
    _need(temperature, "temperature", torch.float32, (rows,), device)
    _need(u_draw, "u_draw", torch.float32, (rows,), device)
    qcode, qld = TAIL_F32, 0
    if draft_probs is not None:
        qcode = _dtype_code(draft_probs, "draft_probs")
        qv, qld = _need_matrix(draft_probs, "draft_probs", rows, device)
        if qv != V:
            raise ValueError(f"draft_probs has {qv} columns, the logits {V}")
    need = verify_logits_workspace(rows, nseq, V)
    with _on(device, stream):
        out_tokens, out_count = _outputs(out_tokens, out_count, rows, nseq, device)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != device:
            raise ValueError("workspace must be a contiguous uint8 tensor on the logits' device")
        rc = lib().tail_verify_logits(rows, nseq, V, _ptr(logits), code, ld, _ptr(temperature), _ptr(cu_rows),
                                      _ptr(drafts), _ptr(u_accept), _ptr(u_draw), _ptr(draft_probs), qcode, qld,
                                      _ptr(workspace), int(workspace.numel()), _ptr(out_tokens), _ptr(out_count),
                                      _stream_ptr(stream, device))
    _fail(rc, "tail_verify_logits")
    return out_tokens, out_count
