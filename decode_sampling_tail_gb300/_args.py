"""Argument checks of the torch wrappers: a tensor that fits gives its pointer, any other a ValueError."""
from __future__ import annotations

import contextlib
import sys

from . import TAIL_BF16, TAIL_ERR_UNSUPPORTED, TAIL_F16, TAIL_F32, TAIL_OK, TailError, lib

_HERE = contextlib.nullcontext()


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
    torch = sys.modules["torch"]  # (an import statement a check adds up: 0.2 us each)
    dtype = t.dtype
    code = (TAIL_F32 if dtype is torch.float32 else TAIL_F16 if dtype is torch.float16 else
            TAIL_BF16 if dtype is torch.bfloat16 else None)
    if code is None:
        raise ValueError(f"{what} must be float32, float16 or bfloat16, not {dtype}")
    shape, strides = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != rows or t.get_device() != index or (shape[1] > 1 and strides[1] != 1):
        raise ValueError(f"{what} must be [{rows}, n] on cuda:{index} with contiguous rows; got {tuple(shape)}, "
                         f"strides {strides}, {t.device}")
    n = shape[1]
    if n < 1:
        raise ValueError(f"{what} must have at least one column")  # (no columns have no pointer: None to the library)
    if (rows | n) >> 31:
        raise ValueError(f"{what} has more than 2^31 - 1 rows or columns")  # (the library takes 32 bits)
    ld = strides[0] if rows > 1 else n
    if ld < n:
        raise ValueError(f"{what}: rows overlap (strides {strides})")
    return t.data_ptr(), code, n, ld


def cuda_index(t, what):
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a CUDA device, not {t.device}")
    return t.get_device()


def raw_stream(stream, index):
    """The cudaStream_t of a torch stream, an integer, or None (the device's current stream)."""
    if stream is None:
        torch = sys.modules["torch"]
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the number alone: 0.1 us instead of 1.3
        return raw(index) if raw else torch.cuda.current_stream(index).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def allocating_on(stream, index):
    """Allocations inside belong to the call's stream."""
    if stream is None:
        return device_guard(index)
    import torch
    if not hasattr(stream, "cuda_stream"):
        # (0 and cudaStreamLegacy are the default stream; to ExternalStream the number 0 is any stream of torch's pool)
        stream = (torch.cuda.default_stream(index) if int(stream) in (0, 1) else
                  torch.cuda.ExternalStream(int(stream), device=index))
    return torch.cuda.stream(stream)


def device_guard(index):
    """Makes the device current for the call (the entry points without a handle run on the current one)."""
    cuda = sys.modules["torch"].cuda
    return _HERE if cuda.current_device() == index else cuda.device(index)


def fail(rc, what):
    if rc == TAIL_ERR_UNSUPPORTED:
        raise TailError(rc, what + " [" + lib().tail_last_error().decode() + "]")
    raise TailError(rc, what)


def call(name, args, index):
    """The library's function on the device; a status other than TAIL_OK raises."""
    cuda, fn = sys.modules["torch"].cuda, getattr(lib(), name)
    if cuda.current_device() == index:
        rc = fn(*args)
    else:
        with cuda.device(index):
            rc = fn(*args)
    if rc != TAIL_OK:
        fail(rc, name)
