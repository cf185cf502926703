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

import ctypes

from . import TAIL_F32, TAIL_OK, lib
from ._args import allocating_on, cuda_index, device_guard, fail, need, need_matrix, raw_stream


def _sequences(cu_rows, index):
    import torch
    if cu_rows.dim() != 1 or cu_rows.shape[0] < 1:
        raise ValueError("cu_rows must be [nseq + 1]")
    return need(cu_rows, "cu_rows", torch.int32, cu_rows.shape, index), cu_rows.shape[0] - 1


def _outputs(out_tokens, out_count, rows, nseq, stream, index):
    import torch
    if out_tokens is None or out_count is None:
        with allocating_on(stream, index):
            if out_tokens is None:
                out_tokens = torch.full((rows,), -1, dtype=torch.int32, device=index)
            if out_count is None:
                out_count = torch.empty((nseq,), dtype=torch.int32, device=index)
    return out_tokens, out_count


def verify(topk_vals, topk_idx, params, cu_rows, drafts, u_accept, draft_probs=None, out_tokens=None,
           out_count=None, stream=None):
    """Drafts against the tail's sorted top-k (tail_verify).

    topk_vals [rows, k] float32 and topk_idx [rows, k] int32 as the tail writes them, params [rows, 3|4]
    float32, cu_rows [nseq + 1] int32, drafts [rows] int32, u_accept [rows] float32, draft_probs [rows, V]
    float32, float16 or bfloat16 (rows may be strided) or None.  Returns (out_tokens [rows] int32, out_count
    [nseq] int32), allocated when not given."""
    import torch
    f32, i32 = torch.float32, torch.int32
    index = cuda_index(topk_vals, "topk_vals")
    rows, k = topk_vals.shape
    cu, nseq = _sequences(cu_rows, index)
    cols = params.shape[-1]
    if cols != 3 and cols != 4:
        raise ValueError("params must be [rows, 3] or [rows, 4]")
    q, code, V, ld = None, TAIL_F32, 0, 0
    if draft_probs is not None:
        q, code, V, ld = need_matrix(draft_probs, "draft_probs", rows, index)
    out_tokens, out_count = _outputs(out_tokens, out_count, rows, nseq, stream, index)
    args = (rows, nseq, k, need(topk_vals, "topk_vals", f32, (rows, k), index),
            need(topk_idx, "topk_idx", i32, (rows, k), index), need(params, "params", f32, (rows, cols), index), cols,
            cu, need(drafts, "drafts", i32, (rows,), index), need(u_accept, "u_accept", f32, (rows,), index), q, code,
            ld, V, need(out_tokens, "out_tokens", i32, (rows,), index),
            need(out_count, "out_count", i32, (nseq,), index), raw_stream(stream, index))
    with device_guard(index):
        rc = lib().tail_verify(*args)
    if rc != TAIL_OK:
        fail(rc, "tail_verify")
    return out_tokens, out_count


def verify_logits_workspace(rows: int, nseq: int, V: int) -> int:
    """Bytes of workspace that ``verify_logits`` needs for these sizes."""
    n = ctypes.c_int64()
    rc = lib().tail_verify_logits_workspace(rows, nseq, V, ctypes.byref(n))
    if rc != TAIL_OK:
        fail(rc, "tail_verify_logits_workspace")
    return n.value


def verify_logits(logits, temperature, cu_rows, drafts, u_accept, u_draw, draft_probs=None, out_tokens=None,
                  out_count=None, workspace=None, stream=None):
    """Drafts against softmax(logits / temperature) over the whole vocabulary (tail_verify_logits).

    logits [rows, V] float32, float16 or bfloat16 (rows may be strided), temperature, u_accept and u_draw [rows]
    float32, cu_rows [nseq + 1] and drafts [rows] int32, draft_probs [rows, V] of any of the three types or None.
    ``workspace``: a uint8 tensor of at least ``verify_logits_workspace(rows, nseq, V)`` bytes that no call which
    may overlap this one uses; allocated when not given.  Returns (out_tokens [rows], out_count [nseq])."""
    import torch
    f32, i32 = torch.float32, torch.int32
    index = cuda_index(logits, "logits")
    rows = logits.shape[0]
    cu, nseq = _sequences(cu_rows, index)
    l, code, V, ld = need_matrix(logits, "logits", rows, index)
    q, qcode, qld = None, TAIL_F32, 0
    if draft_probs is not None:
        q, qcode, qv, qld = need_matrix(draft_probs, "draft_probs", rows, index)
        if qv != V:
            raise ValueError(f"draft_probs has {qv} columns, the logits {V}")
    out_tokens, out_count = _outputs(out_tokens, out_count, rows, nseq, stream, index)
    if workspace is None:
        with allocating_on(stream, index):
            workspace = torch.empty(verify_logits_workspace(rows, nseq, V), dtype=torch.uint8, device=index)
    size = workspace.numel()
    args = (rows, nseq, V, l, code, ld, need(temperature, "temperature", f32, (rows,), index), cu,
            need(drafts, "drafts", i32, (rows,), index), need(u_accept, "u_accept", f32, (rows,), index),
            need(u_draw, "u_draw", f32, (rows,), index), q, qcode, qld,
            need(workspace, "workspace", torch.uint8, (size,), index), size,
            need(out_tokens, "out_tokens", i32, (rows,), index), need(out_count, "out_count", i32, (nseq,), index),
            raw_stream(stream, index))
    with device_guard(index):
        rc = lib().tail_verify_logits(*args)
    if rc != TAIL_OK:
        fail(rc, "tail_verify_logits")
    return out_tokens, out_count
