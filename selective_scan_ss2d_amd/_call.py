"""What the bindings of the sequence operators share: the stream and device that a call
belongs to, and its outputs."""
from __future__ import annotations

import contextlib

from . import _binding as bnd
from ._binding import _torch


def code_of(dtype):
    """The data type's code, None for a type that the operators do not take."""
    torch = _torch()
    if dtype is torch.bfloat16:
        return bnd.SS2D_BF16
    return bnd.SS2D_F32 if dtype is torch.float32 else None


@contextlib.contextmanager
def _switched(device, stream):
    torch = _torch()
    with torch.cuda.device(device), torch.cuda.stream(stream or torch.cuda.current_stream(device)):
        yield


def scope(device, stream, *tensors):
    """The device and stream that a call's outputs and scratch belong to: a context only
    where they are not the current ones already.  tensors: the caller's, None among them."""
    torch = _torch()
    if stream is None and device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    if stream is not None and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    if stream is not None:  # their memory is not to be reused before the call has run
        for t in tensors:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    return _switched(device, stream)


def handle(device, stream):
    """The HIP stream that a call runs on (without making a torch.cuda.Stream, 2 us)."""
    if stream is None:
        return _torch()._C._cuda_getCurrentRawStream(device.index)
    return stream.cuda_stream


def expect(name, t, shape, dtype, device):
    """Checks a contiguous tensor."""
    try:
        fits = (t.shape == shape and t.dtype is dtype and t.device == device
                and t.is_contiguous())
    except AttributeError:
        fits = False
    if not fits:
        bnd._expect(name, t, shape, dtype, device)  # says what is wrong


def ptr(t):
    return None if t is None else t.data_ptr()


def output(name, t, shape, dtype, device):
    if t is None:
        return _torch().empty(shape, dtype=dtype, device=device)
    expect(name, t, shape, dtype, device)
    return t


def scratch(size, device):
    """Scratch of a call on the current stream (size -1: of a call that will be refused).  It goes
    back to torch's allocator when the call returns, which hands it to later work of the same stream
    only; in a captured graph it belongs to the graph."""
    return _torch().empty(max(256, size), dtype=_torch().uint8, device=device)


def rows(name, t, shape, dtype, device):
    """Checks a (batch, token, ...) tensor whose last axis alone has to be contiguous; whether all
    of it is."""
    try:
        fits = t.shape == shape and t.dtype is dtype and t.device == device
        if fits and t.is_contiguous():
            return True
        fits = fits and (t.stride(-1) == 1 or shape[-1] <= 1)
    except AttributeError:
        fits = False
    if not fits:
        bnd._expect(name, t, shape, dtype, device)  # says what is wrong
        raise ValueError(f"{name}'s last axis must be contiguous")
    return False


def packed_sequences(cu_seqlens, B, device):
    """The number of sequences: the rows, or those that the offsets name."""
    if cu_seqlens is None:
        return B
    torch = _torch()
    if not isinstance(cu_seqlens, torch.Tensor):
        raise TypeError("cu_seqlens must be a torch.Tensor")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must hold S + 1 offsets")
    expect("cu_seqlens", cu_seqlens, cu_seqlens.shape, torch.int32, device)
    if B != 1:
        raise ValueError("packed sequences (cu_seqlens) need a batch of 1")
    return cu_seqlens.shape[0] - 1
