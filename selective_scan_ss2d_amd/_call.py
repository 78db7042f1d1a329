"""What the bindings of the sequence operators share: the stream and device that a call
belongs to, and its outputs."""
from __future__ import annotations

import contextlib

import torch

from . import _binding as bnd

CODES = {torch.float32: bnd.SS2D_F32, torch.bfloat16: bnd.SS2D_BF16}


@contextlib.contextmanager
def _switched(device, stream):
    with torch.cuda.device(device), torch.cuda.stream(stream or torch.cuda.current_stream(device)):
        yield


def scope(device, stream, *inputs):
    """The device and stream that a call's outputs and scratch belong to: a context only
    where they are not the current ones already."""
    if stream is None and device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    if stream is not None:  # the inputs' memory is not to be reused before the call has run
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
    return _switched(device, stream)


def ptr(t):
    return None if t is None else t.data_ptr()


def output(name, t, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    bnd._expect(name, t, shape, dtype, device)
    return t
