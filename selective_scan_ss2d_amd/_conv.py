"""Binding of the short causal convolution (``ss1d_conv_*`` of ``include/ss2d.h``).

Argument checks and marshalling only; every step runs in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes

from . import _binding as bnd
from ._binding import _torch
from ._call import (code_of, expect, handle, output, packed_sequences, ptr, rows, scope, scratch)


def _inputs(x, conv_w, conv_b):
    """Checks the convolution's inputs; (B, L, D, KW), the data type's code and the strides (None
    for a contiguous x)."""
    torch = _torch()
    if not (isinstance(x, torch.Tensor) and isinstance(conv_w, torch.Tensor)):
        raise TypeError("x and conv_w must be torch.Tensors")
    if x.dim() != 3 or conv_w.dim() != 2:
        raise ValueError("x must be (B, L, D) and conv_w (D, KW)")
    dev, dtype = x.device, x.dtype
    if dev.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    code = code_of(dtype)
    if code is None:
        raise TypeError(f"x must be float32 or bfloat16, not {dtype}")
    B, L, D = x.shape
    KW = conv_w.shape[1]
    strides = None
    if not rows("x", x, x.shape, dtype, dev):
        strides = (ctypes.c_int64 * 2)(*x.stride()[:2])
    expect("conv_w", conv_w, (D, KW), torch.float32, dev)
    if conv_b is not None:
        expect("conv_b", conv_b, (D,), torch.float32, dev)
    if not 1 <= KW <= 8:
        raise ValueError(f"conv_w has {KW} taps, expected 1 to 8")
    return (B, L, D, KW), code, strides


def ss1d_conv_forward(x, conv_w, conv_b=None, silu=True, cu_seqlens=None, initial_state=None,
                      final_state=False, y=None, stream=None):
    """The short causal convolution of each channel, with its SiLU.

    y_t = act(conv_b + sum_j conv_w_j x_{t - KW + 1 + j}); act is SiLU, or nothing with
    silu=False.  x (B, L, D) float32 or bfloat16, last axis contiguous; conv_w (D, KW), KW <= 8,
    and conv_b (D) float32.

    cu_seqlens: int32 offsets (S + 1) of S sequences packed into the tokens of B = 1 (tokens
    outside of them are left as they are in y).  initial_state (S, KW - 1, D), x's dtype: the
    inputs before the first token, the oldest first (zero without it).  Returns y (B, L, D); with
    final_state True (or a tensor to write, which may be initial_state itself) the pair
    (y, the last KW - 1 inputs (S, KW - 1, D)).
    """
    torch, lib = _torch(), bnd.load_library()
    (B, L, D, KW), code, strides = _inputs(x, conv_w, conv_b)
    dev = x.device
    S = packed_sequences(cu_seqlens, B, dev)
    if initial_state is not None:
        expect("initial_state", initial_state, (S, KW - 1, D), x.dtype, dev)
    given = final_state if isinstance(final_state, torch.Tensor) else None
    with scope(dev, stream, x, conv_w, conv_b, cu_seqlens, initial_state, y, given):
        y = output("y", y, (B, L, D), x.dtype, dev)
        ht = None
        if final_state is not False and final_state is not None:
            ht = output("final_state", given, (S, KW - 1, D), x.dtype, dev)
        bnd._check(lib.ss1d_conv_forward(
            x.data_ptr(), conv_w.data_ptr(), ptr(conv_b), ptr(initial_state), ptr(cu_seqlens),
            y.data_ptr(), ptr(ht), B, L, S, D, KW, strides, 1 if silu else 0, code,
            handle(dev, stream)))
    return y if ht is None else (y, ht)


def ss1d_conv_backward(x, conv_w, dy, conv_b=None, silu=True, cu_seqlens=None, initial_state=None,
                       dstate=None, stream=None):
    """Gradients of sum(dy * y) + sum(dstate * final state) for ss1d_conv_forward's outputs on the
    same inputs: a dict with those of x and conv_w, and of conv_b and initial_state if they are
    given.

    dy: contiguous, y's shape and dtype; dstate: (S, KW - 1, D), x's dtype, or None.  Rows outside
    of every packed sequence are zero.
    """
    torch, lib = _torch(), bnd.load_library()
    (B, L, D, KW), code, strides = _inputs(x, conv_w, conv_b)
    dev = x.device
    S = packed_sequences(cu_seqlens, B, dev)
    packed = cu_seqlens is not None
    expect("dy", dy, (B, L, D), x.dtype, dev)
    for name, t in (("initial_state", initial_state), ("dstate", dstate)):
        if t is not None:
            expect(name, t, (S, KW - 1, D), x.dtype, dev)
    with scope(dev, stream, x, conv_w, conv_b, dy, cu_seqlens, initial_state, dstate):
        d = {"x": (torch.zeros if packed else torch.empty)(x.shape, dtype=x.dtype, device=dev),
             "conv_w": torch.empty_like(conv_w)}
        if conv_b is not None:
            d["conv_b"] = torch.empty_like(conv_b)
        if initial_state is not None:
            d["initial_state"] = torch.empty_like(initial_state)
        ws = scratch(lib.ss1d_conv_scratch_bytes(B, L, S, D, KW, code, packed), dev)
        bnd._check(lib.ss1d_conv_backward(
            x.data_ptr(), conv_w.data_ptr(), ptr(conv_b), ptr(initial_state), ptr(cu_seqlens),
            dy.data_ptr(), ptr(dstate), d["x"].data_ptr(), d["conv_w"].data_ptr(),
            ptr(d.get("conv_b")), ptr(d.get("initial_state")), ws.data_ptr(), ws.numel(), B, L, S, D,
            KW, strides, 1 if silu else 0, code, handle(dev, stream)))
    return d


def ss1d_conv_step(x, conv_w, state, conv_b=None, silu=True, slots=None, y=None, stream=None):
    """The short causal convolution for T (few) tokens of each of B sequences, states in place.

    x (B, T, D), conv_w, conv_b and silu as in ss1d_conv_forward; state (S, KW - 1, D), x's dtype,
    the last inputs of each sequence, the oldest first, updated in place.  slots: as in
    ss1d_scan_step.  Returns y (B, T, D).
    """
    torch, lib = _torch(), bnd.load_library()
    (B, T, D, KW), code, strides = _inputs(x, conv_w, conv_b)
    dev = x.device
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be (S, KW - 1, D)")
    S = state.shape[0]
    expect("state", state, (S, KW - 1, D), x.dtype, dev)
    if slots is not None:
        expect("slots", slots, (B,), torch.int32, dev)
    elif S != B:
        raise ValueError(f"state holds {S} sequences, expected {B} without slots")
    with scope(dev, stream, x, conv_w, conv_b, state, slots, y):
        y = output("y", y, (B, T, D), x.dtype, dev)
        bnd._check(lib.ss1d_conv_step(
            x.data_ptr(), conv_w.data_ptr(), ptr(conv_b), state.data_ptr(), ptr(slots), y.data_ptr(),
            B, T, S, D, KW, strides, 1 if silu else 0, code, handle(dev, stream)))
    return y
