"""Training on vocabulary logits: losses with their gradients, on torch CUDA tensors.

``token_logprobs`` scores given tokens (a rollout's old and reference log-probabilities), ``token_logprobs_grad``
gives the gradient of any loss formed of them; ``policy_loss``, ``preference_loss`` and ``distill_topk`` form a
loss and its gradient in one call.  ``include/tail.h`` states the formulas.  A gradient is handed on with
``logits.backward(grad)``, or written over the logits themselves (``out_grad=logits``).  Outputs that the caller gives are
written through their pointers: autograd's version counters do not see it, so logits that some function has saved for its
backward pass must not be written over.

The tensors are checked here (type, shape, device, strides; ValueError); the library checks sizes, factors
and overlaps.  Calls are asynchronous on ``stream`` (None: the current stream of the tensors' device).
"""
from __future__ import annotations

import ctypes
import functools

from . import TAIL_OK, lib
from ._args import allocating_on, call, cuda_index, fail, need, need_matrix, need_opt, raw_stream


def _grad(out_grad, logits, rows, V, index):
    """(pointer, leading dimension) of the gradient's matrix; (None, 0) for none."""
    if out_grad is None:
        return None, 0
    if out_grad.dtype is not logits.dtype:
        raise ValueError(f"out_grad must be {logits.dtype} like the logits, not {out_grad.dtype}")
    p, _, n, ld = need_matrix(out_grad, "out_grad", rows, index)
    if n != V:
        raise ValueError(f"out_grad has {n} columns, the logits {V}")
    return p, ld


def _empty(t, shape, wanted, like):
    """An fp32 output that the caller did not give, where it is wanted."""
    if t is not None or not wanted:
        return t
    import torch
    return torch.empty(shape, dtype=torch.float32, device=like.device)


def set_training_wait_limit(ns: int):
    """Bounds the waits of later calls' CTAs for one another to ``ns`` nanoseconds (tail_training_set_wait_limit; 1e9 at
    first)."""
    if not 0 <= ns < 1 << 64:
        raise ValueError(f"ns must be 0 to 2^64 - 1, not {ns}")
    rc = lib().tail_training_set_wait_limit(ns)
    if rc != TAIL_OK:
        fail(rc, "tail_training_set_wait_limit")


def token_logprobs(logits, tokens, temperature=1.0, *, entropy=False, out_logprob=None, out_lse=None,
                   out_entropy=None, out_stats=None, stream=None):
    """Log-probabilities of ``tokens`` under softmax(logits / temperature) (tail_token_logprobs_ex).

    logits [rows, V] float32, float16 or bfloat16 (rows may be strided), tokens [rows] int32 (outside [0, V): an
    ignored row).  Returns (logprob, lse, entropy), each [rows] float32, allocated when not given; entropy is None
    unless asked for (``entropy=True`` or ``out_entropy``).  ``out_stats`` [rows, 2] float32 receives what
    ``token_logprobs_grad`` needs to give a likely token's gradient to all its digits."""
    import torch
    f32 = torch.float32
    index = cuda_index(logits, "logits")
    rows = logits.shape[0]
    l, code, V, ld = need_matrix(logits, "logits", rows, index)
    if out_logprob is None or out_lse is None or (entropy and out_entropy is None):
        with allocating_on(stream, index):
            out_logprob = _empty(out_logprob, rows, True, logits)
            out_lse = _empty(out_lse, rows, True, logits)
            out_entropy = _empty(out_entropy, rows, entropy, logits)
    n = (rows,)
    args = (rows, V, l, code, ld, need(tokens, "tokens", torch.int32, n, index), temperature,
            need(out_logprob, "out_logprob", f32, n, index), need(out_lse, "out_lse", f32, n, index),
            need_opt(out_entropy, "out_entropy", f32, n, index), need_opt(out_stats, "out_stats", f32, (rows, 2), index),
            raw_stream(stream, index))
    call("tail_token_logprobs_ex", args, index)
    return out_logprob, out_lse, out_entropy


def token_logprobs_grad(logits, tokens, lse, d_logprob, temperature=1.0, *, d_entropy=None, entropy=None,
                        stats=None, out_grad=None, stream=None):
    """The gradient of sum(d_logprob * logprob + d_entropy * entropy) by the logits (tail_token_logprobs_grad_ex).

    lse, entropy and stats as ``token_logprobs`` gave them, d_logprob and d_entropy [rows] float32 (d_entropy goes with
    entropy).  With ``stats`` lse is not read (None will do) and the gradient is exact to about 2^-16 of itself.  Without it
    every probability is off by lse's rounding, up to 2^-24 |lse| of itself: a token whose 1 - p is near that or below
    loses its gradient, and temperatures that make |logits| / temperature large lose the others'.  Returns out_grad,
    [rows, V] of the logits' type, allocated when not given (may be the logits)."""
    import torch
    f32 = torch.float32
    index = cuda_index(logits, "logits")
    rows = logits.shape[0]
    l, code, V, ld = need_matrix(logits, "logits", rows, index)
    if lse is None and stats is None:
        raise ValueError("lse or stats must be given")
    if out_grad is None:
        with allocating_on(stream, index):
            out_grad = torch.empty((rows, V), dtype=logits.dtype, device=logits.device)
    g, gld = _grad(out_grad, logits, rows, V, index)
    n = (rows,)
    args = (rows, V, l, code, ld, need(tokens, "tokens", torch.int32, n, index), temperature,
            need_opt(lse, "lse", f32, n, index), need_opt(stats, "stats", f32, (rows, 2), index),
            need(d_logprob, "d_logprob", f32, n, index), need_opt(d_entropy, "d_entropy", f32, n, index),
            need_opt(entropy, "entropy", f32, n, index), g, gld, raw_stream(stream, index))
    call("tail_token_logprobs_grad_ex", args, index)
    return out_grad


def policy_loss(logits, tokens, old_logprob, advantage, *, ref_logprob=None, temperature=1.0, clip_low=0.2,
                clip_high=0.2, kl_coef=0.0, entropy_coef=0.0, weight=None, grad=True, out_loss=None, out_logprob=None,
                out_entropy=None, out_grad=None, stream=None):
    """The clipped policy loss of every row with its KL and entropy terms, and its gradient (tail_policy_loss).

    logits [rows, V] float32, float16 or bfloat16 (rows may be strided), tokens [rows] int32 (outside [0, V): an
    ignored row), old_logprob, advantage, ref_logprob (needed with kl_coef) and weight [rows] float32.  Returns
    (loss, logprob, grad): [rows] float32 twice and the gradient of loss.sum(), [rows, V] of the logits' type; allocated
    when not given, grad None with ``grad=False``.  ``out_entropy`` [rows] float32 receives the entropies."""
    import torch
    f32 = torch.float32
    index = cuda_index(logits, "logits")
    rows = logits.shape[0]
    l, code, V, ld = need_matrix(logits, "logits", rows, index)
    if out_loss is None or out_logprob is None or (grad and out_grad is None):
        with allocating_on(stream, index):
            out_loss = _empty(out_loss, rows, True, logits)
            out_logprob = _empty(out_logprob, rows, True, logits)
            if grad and out_grad is None:
                out_grad = torch.empty((rows, V), dtype=logits.dtype, device=logits.device)
    g, gld = _grad(out_grad, logits, rows, V, index)
    n = (rows,)
    args = (rows, V, l, code, ld, need(tokens, "tokens", torch.int32, n, index), temperature,
            need(old_logprob, "old_logprob", f32, n, index), need(advantage, "advantage", f32, n, index),
            need_opt(ref_logprob, "ref_logprob", f32, n, index), clip_low, clip_high, kl_coef, entropy_coef,
            need_opt(weight, "weight", f32, n, index), need(out_loss, "out_loss", f32, n, index),
            need(out_logprob, "out_logprob", f32, n, index), need_opt(out_entropy, "out_entropy", f32, n, index),
            g, gld, raw_stream(stream, index))
    call("tail_policy_loss", args, index)
    return out_loss, out_logprob, out_grad


@functools.lru_cache(maxsize=64)
def preference_loss_workspace(rows: int) -> int:
    """Bytes of workspace that ``preference_loss`` needs for this many rows."""
    if rows >> 31:
        raise ValueError(f"rows must be 0 to 2^31 - 1, not {rows}")
    n = ctypes.c_int64()
    rc = lib().tail_preference_loss_workspace(rows, ctypes.byref(n))
    if rc != TAIL_OK:
        fail(rc, "tail_preference_loss_workspace")
    return n.value


def preference_loss(logits, tokens, cu_rows, *, ref_logprob=None, beta=0.1, label_smoothing=0.0, margin=0.0,
                    average=False, temperature=1.0, weight=None, grad=True, out_loss=None, out_seq_logprob=None,
                    out_grad=None, workspace=None, stream=None):
    """The paired preference loss over sequences of rows, and its gradient (tail_preference_loss).

    logits [rows, V] float32, float16 or bfloat16 (rows may be strided), tokens [rows] int32 (outside [0, V): a row
    that does not count), cu_rows [nseq + 1] int32 with sequence 2i chosen over 2i + 1, ref_logprob [nseq] and weight
    [nseq / 2] float32.  ``workspace``: a uint8 tensor of at least ``preference_loss_workspace(rows)`` bytes
    that no call which may overlap this one uses; allocated when not given.  Returns (loss [nseq / 2], seq_logprob [nseq],
    grad [rows, V] of the logits' type: the gradient of loss.sum()), allocated when not given, grad None with
    ``grad=False``."""
    import torch
    f32, i32 = torch.float32, torch.int32
    index = cuda_index(logits, "logits")
    rows = logits.shape[0]
    if cu_rows.dim() != 1 or cu_rows.shape[0] < 1 or cu_rows.shape[0] % 2 == 0:
        raise ValueError("cu_rows must be [nseq + 1] with nseq even")
    nseq = cu_rows.shape[0] - 1
    if nseq >> 31:
        raise ValueError("cu_rows has more than 2^31 entries")
    l, code, V, ld = need_matrix(logits, "logits", rows, index)
    if out_loss is None or out_seq_logprob is None or workspace is None or (grad and out_grad is None):
        with allocating_on(stream, index):
            out_loss = _empty(out_loss, nseq // 2, True, logits)
            out_seq_logprob = _empty(out_seq_logprob, nseq, True, logits)
            if workspace is None:
                workspace = torch.empty(preference_loss_workspace(rows), dtype=torch.uint8, device=logits.device)
            if grad and out_grad is None:
                out_grad = torch.empty((rows, V), dtype=logits.dtype, device=logits.device)
    g, gld = _grad(out_grad, logits, rows, V, index)
    size = workspace.numel()
    args = (rows, V, nseq, l, code, ld, need(tokens, "tokens", i32, (rows,), index),
            need(cu_rows, "cu_rows", i32, (nseq + 1,), index), temperature,
            need_opt(ref_logprob, "ref_logprob", f32, (nseq,), index), beta, label_smoothing, margin, int(average),
            need_opt(weight, "weight", f32, (nseq // 2,), index),
            need(workspace, "workspace", torch.uint8, (size,), index), size,
            need(out_loss, "out_loss", f32, (nseq // 2,), index),
            need(out_seq_logprob, "out_seq_logprob", f32, (nseq,), index), g, gld, raw_stream(stream, index))
    call("tail_preference_loss", args, index)
    return out_loss, out_seq_logprob, out_grad


def distill_topk(logits, topk_vals, topk_idx, *, teacher_rest=None, temperature=1.0, weight=None, grad=True,
                 out_loss=None, out_grad=None, stream=None):
    """Distillation of a student's logits from a teacher's top logits, and its gradient (tail_distill_topk).

    logits [rows, V] and topk_vals [rows, k] float32, float16 or bfloat16, topk_idx [rows, k] int32 (outside [0, V): no
    entry; all three may have strided rows), as ``Tail.run`` writes them for the teacher; teacher_rest [rows] float32:
    the log-sum-exp of the teacher's other logits / temperature; weight [rows] float32.  Returns (loss [rows] float32,
    grad [rows, V] of the logits' type: the gradient of loss.sum()), allocated when not given, grad None with
    ``grad=False``.

    The rest comes from the teacher's logits without the listed ones (every id a valid one), whatever the list holds::

        others = teacher_logits.scatter(1, topk_idx.long(), -math.inf)
        rest = token_logprobs(others, topk_idx[:, 0].contiguous(), temperature)[1]

    Where only the teacher's lse (``token_logprobs``) and the list are left, it is known to about 2^-24 |lse| of all
    tokens' weight, and may come out below nothing::

        listed = torch.exp(topk_vals.double() / temperature - lse.double()[:, None]).sum(-1)
        rest = (lse.double() + torch.log(torch.clamp(1 - listed, min=0))).float()
    """
    import torch
    f32 = torch.float32
    index = cuda_index(logits, "logits")
    rows = logits.shape[0]
    l, code, V, ld = need_matrix(logits, "logits", rows, index)
    v, vcode, k, vld = need_matrix(topk_vals, "topk_vals", rows, index)
    if (topk_idx.dtype is not torch.int32 or topk_idx.shape != topk_vals.shape or topk_idx.get_device() != index or
            (k > 1 and topk_idx.stride(1) != 1)):
        raise ValueError(f"topk_idx must be int32 [{rows}, {k}] on cuda:{index} with contiguous rows; got "
                         f"{topk_idx.dtype}, {tuple(topk_idx.shape)}, strides {topk_idx.stride()}, {topk_idx.device}")
    ild = topk_idx.stride(0) if rows > 1 else k
    if out_loss is None or (grad and out_grad is None):
        with allocating_on(stream, index):
            out_loss = _empty(out_loss, rows, True, logits)
            if grad and out_grad is None:
                out_grad = torch.empty((rows, V), dtype=logits.dtype, device=logits.device)
    g, gld = _grad(out_grad, logits, rows, V, index)
    n = (rows,)
    args = (rows, V, k, l, code, ld, v, vcode, vld, topk_idx.data_ptr(), ild, temperature,
            need_opt(teacher_rest, "teacher_rest", f32, n, index), need_opt(weight, "weight", f32, n, index),
            need(out_loss, "out_loss", f32, n, index), g, gld, raw_stream(stream, index))
    call("tail_distill_topk", args, index)
    return out_loss, out_grad
