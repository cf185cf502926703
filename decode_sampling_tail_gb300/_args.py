"""Argument checks of the torch wrappers: a tensor that fits gives its pointer, any other a ValueError."""
from __future__ import annotations

import contextlib

from . import TAIL_BF16, TAIL_ERR_UNSUPPORTED, TAIL_F16, TAIL_F32, TailError, lib


def need(t, what, dtype, shape, index):
    """The pointer of a contiguous tensor of this type and shape on CUDA device `index`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{index}; "
                     f"got {t.dtype}, {tuple(t.shape)}, strides {t.stride()}, {t.device}")


def need_opt(t, what, dtype, shape, index):
    return None if t is None else need(t, what, dtype, shape, index)


def need_matrix(t, what, rows, index):
    """[rows, n >= 1] of a float type with unit stride along the columns: (pointer, type code, n, leading dimension)."""
    import torch
    code = {torch.float32: TAIL_F32, torch.float16: TAIL_F16, torch.bfloat16: TAIL_BF16}.get(t.dtype)
    if code is None:
        raise ValueError(f"{what} must be float32, float16 or bfloat16, not {t.dtype}")
    if t.dim() != 2 or t.shape[0] != rows or t.get_device() != index or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what} must be [{rows}, n] on cuda:{index} with contiguous rows; got {tuple(t.shape)}, "
                         f"strides {t.stride()}, {t.device}")
    n = t.shape[1]
    if n < 1:
        raise ValueError(f"{what} must have at least one column")  # (no columns have no pointer: None to the library)
    ld = t.stride(0) if rows > 1 else n
    if ld < n:
        raise ValueError(f"{what}: rows overlap (strides {t.stride()})")
    return t.data_ptr(), code, n, ld


def cuda_index(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device, not {t.device}")
    return t.get_device()


def raw_stream(stream, index):
    """The cudaStream_t of a torch stream, an integer, or None (the device's current stream)."""
    if stream is None:
        import torch
        return torch.cuda.current_stream(index).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def allocating_on(stream, index):
    """Allocations inside belong to the call's stream."""
    import torch
    if stream is None:
        return torch.cuda.device(index)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    return torch.cuda.stream(stream)


def device_guard(index):
    """Makes the device current for the call (the entry points without a handle run on the current one)."""
    import torch
    return contextlib.nullcontext() if torch.cuda.current_device() == index else torch.cuda.device(index)


def fail(rc, what):
    if rc == TAIL_ERR_UNSUPPORTED:
        raise TailError(rc, what + " [" + lib().tail_last_error().decode() + "]")
    raise TailError(rc, what)
