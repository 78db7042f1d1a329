"""Binding of the gated delta rule (``ss1d_delta_*`` of ``include/ss2d.h``).

Argument checks and marshalling only; every step runs in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes

from . import _binding as bnd
from ._binding import _torch
from ._call import (code_of, expect as _expect, handle as _handle, output as _output, ptr as _ptr,
                    scope as _scope, scratch as _scratch)


def _strided(name, t, shape, dtype, device):
    """Checks a tensor whose last axis alone has to be contiguous."""
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.stride(3) != 1 and shape[3] > 1:
        raise ValueError(f"{name}'s last axis must be contiguous")


def _inputs(q, k, v, g, beta):
    """Checks the rule's inputs; (B, L, HK, DK, H, DV), the data type's code and the strides
    (None for contiguous tensors)."""
    torch = _torch()
    tensor = torch.Tensor
    if not (isinstance(q, tensor) and isinstance(k, tensor) and isinstance(v, tensor)):
        raise TypeError("q, k and v must be torch.Tensors")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be (B, L, HK, DK) and v (B, L, H, DV)")
    dev, dtype = q.device, q.dtype
    if dev.type != "cuda":
        raise ValueError("q must be a GPU tensor")
    code = code_of(dtype)
    if code is None:
        raise TypeError(f"q must be float32 or bfloat16, not {dtype}")
    B, L, HK, DK = q.shape
    H, DV = v.shape[2], v.shape[3]
    if HK < 1 or H % HK:
        raise ValueError(f"v has {H} heads, expected a multiple of q's {HK}")
    _strided("q", q, (B, L, HK, DK), dtype, dev)
    _strided("k", k, (B, L, HK, DK), dtype, dev)
    _strided("v", v, (B, L, H, DV), dtype, dev)
    _expect("g", g, (B, L, H), torch.float32, dev)
    _expect("beta", beta, (B, L, H), torch.float32, dev)
    strides = None
    if not (q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        strides = (ctypes.c_int64 * 9)(*q.stride()[:3], *k.stride()[:3], *v.stride()[:3])
    return (B, L, HK, DK, H, DV), code, strides


def _sequences(cu_seqlens, B, device):
    if cu_seqlens is None:
        return B
    if not isinstance(cu_seqlens, _torch().Tensor):
        raise TypeError("cu_seqlens must be a torch.Tensor")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must hold S + 1 offsets")
    _expect("cu_seqlens", cu_seqlens, cu_seqlens.shape, _torch().int32, device)
    if B != 1:
        raise ValueError("packed sequences (cu_seqlens) need a batch of 1")
    return cu_seqlens.shape[0] - 1


def _forward(q, k, v, g, beta, scale, cu_seqlens, initial_state, final_state, o, stream, save):
    torch, lib = _torch(), bnd.load_library()
    (B, L, HK, DK, H, DV), code, strides = _inputs(q, k, v, g, beta)
    dev = q.device
    S = _sequences(cu_seqlens, B, dev)
    if initial_state is not None:
        _expect("initial_state", initial_state, (S, H, DK, DV), torch.float32, dev)
    given = final_state if isinstance(final_state, torch.Tensor) else None
    with _scope(dev, stream, q, k, v, g, beta, cu_seqlens, initial_state, o, given):
        o = _output("o", o, (B, L, H, DV), q.dtype, dev)
        ht = saved = None
        if final_state is not False and final_state is not None:
            ht = _output("final_state", None if final_state is True else final_state,
                         (S, H, DK, DV), torch.float32, dev)
        if save:
            size = lib.ss1d_delta_saved_bytes(B, L, S, H, DK, DV, cu_seqlens is not None)
            saved = torch.empty(max(0, size), dtype=torch.uint8, device=dev)
        ws = _scratch(lib.ss1d_delta_scratch_bytes(0, save, B, L, S, HK, H, DK, DV, code,
                                                   cu_seqlens is not None), dev)
        bnd._check(lib.ss1d_delta_forward_ws(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            _ptr(initial_state), _ptr(cu_seqlens), o.data_ptr(), _ptr(ht), _ptr(saved),
            ws.data_ptr(), ws.numel(), B, L, S, HK, H, DK, DV, strides,
            DK ** -0.5 if scale is None else scale, code, _handle(dev, stream)))
    return o, ht, saved


def ss1d_delta_forward(q, k, v, g, beta, scale=None, cu_seqlens=None, initial_state=None,
                       final_state=False, o=None, stream=None):
    """The gated delta rule over whole sequences.

    Per sequence and value head, from a state S (DK, DV), zero or ``initial_state``:
    S <- exp(g_t) S; u_t = beta_t (v_t - S^T k_t); S <- S + k_t u_t^T; o_t = scale S^T q_t.
    q, k (B, L, HK, DK) and v (B, L, H, DV) float32 or bfloat16, last axis contiguous, H a
    multiple of HK (value head h reads key head h // (H // HK)), DK <= 128; g (log decays)
    and beta (B, L, H) float32.  scale defaults to DK ** -0.5.  k is expected normalised
    (|k_t|^2 beta_t <= 2 keeps the rule stable).

    cu_seqlens: int32 offsets (S + 1) of S sequences packed into the tokens of B = 1 (tokens
    outside of them are left as they are in o).  initial_state (S, H, DK, DV) float32.
    Returns o (B, L, H, DV); with final_state True (or a tensor to write, which may be
    initial_state itself) the pair (o, end states (S, H, DK, DV) float32).
    """
    o, ht, _ = _forward(q, k, v, g, beta, scale, cu_seqlens, initial_state, final_state, o,
                        stream, False)
    return o if ht is None else (o, ht)


def ss1d_delta_forward_save(q, k, v, g, beta, scale=None, cu_seqlens=None, initial_state=None,
                            final_state=False, o=None, stream=None):
    """The training forward: ss1d_delta_forward, and the buffer that ss1d_delta_backward starts
    from.  Returns (o, saved), with final_state (o, end states, saved)."""
    o, ht, saved = _forward(q, k, v, g, beta, scale, cu_seqlens, initial_state, final_state, o,
                            stream, True)
    return (o, saved) if ht is None else (o, ht, saved)


def ss1d_delta_backward(q, k, v, g, beta, do, scale=None, cu_seqlens=None, initial_state=None,
                        dstate=None, saved=None, stream=None):
    """Gradients of sum(do * o) + sum(dstate * end states) for ss1d_delta_forward's outputs on
    the same inputs: a dict with those of q, k, v, g and beta, and of initial_state if it is
    given.

    do: contiguous, the shape and dtype of v's output; dstate: float32 (S, H, DK, DV) or None.
    saved: the buffer of ss1d_delta_forward_save for the same inputs; None computes it again.
    Rows outside of every packed sequence are zero.
    """
    torch, lib = _torch(), bnd.load_library()
    (B, L, HK, DK, H, DV), code, strides = _inputs(q, k, v, g, beta)
    dev = q.device
    S = _sequences(cu_seqlens, B, dev)
    _expect("do", do, (B, L, H, DV), q.dtype, dev)
    for name, t in (("initial_state", initial_state), ("dstate", dstate)):
        if t is not None:
            _expect(name, t, (S, H, DK, DV), torch.float32, dev)
    if saved is not None:
        size = lib.ss1d_delta_saved_bytes(B, L, S, H, DK, DV, cu_seqlens is not None)
        _expect("saved", saved, (max(0, size),), torch.uint8, dev)
    with _scope(dev, stream, q, k, v, g, beta, do, cu_seqlens, initial_state, dstate, saved):
        make = torch.empty if cu_seqlens is None else torch.zeros
        d = {n: make(t.shape, dtype=t.dtype, device=dev)
             for n, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta))}
        if initial_state is not None:
            d["initial_state"] = torch.empty_like(initial_state)
        ws = _scratch(lib.ss1d_delta_scratch_bytes(1, saved is not None, B, L, S, HK, H, DK, DV,
                                                   code, cu_seqlens is not None), dev)
        bnd._check(lib.ss1d_delta_backward_ws(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            _ptr(initial_state), _ptr(cu_seqlens), _ptr(saved), do.data_ptr(), _ptr(dstate),
            d["q"].data_ptr(), d["k"].data_ptr(), d["v"].data_ptr(), d["g"].data_ptr(),
            d["beta"].data_ptr(), _ptr(d.get("initial_state")), ws.data_ptr(), ws.numel(), B, L, S,
            HK, H, DK, DV, strides, DK ** -0.5 if scale is None else scale, code,
            _handle(dev, stream)))
    return d


def ss1d_delta_step(q, k, v, g, beta, state, slots=None, scale=None, o=None, stream=None):
    """The gated delta rule for T (few) tokens of each of B sequences, states in place.

    q, k (B, T, HK, DK), v (B, T, H, DV), g and beta (B, T, H) as in ss1d_delta_forward; state
    (S, H, DK, DV) float32, updated in place.  Row b's state is state[slots[b]] (int32 slots
    (B)), or state[b].  Rows with a slot outside 0 .. S - 1 are padding and their rows of o
    stay as they are; rows that name one slot are successive tokens of one sequence, in row
    order.  Returns o (B, T, H, DV).
    """
    torch, lib = _torch(), bnd.load_library()
    (B, T, HK, DK, H, DV), code, strides = _inputs(q, k, v, g, beta)
    dev = q.device
    if not isinstance(state, torch.Tensor) or state.dim() != 4:
        raise ValueError("state must be (S, H, DK, DV)")
    S = state.shape[0]
    _expect("state", state, (S, H, DK, DV), torch.float32, dev)
    if slots is not None:
        _expect("slots", slots, (B,), torch.int32, dev)
    elif S != B:
        raise ValueError(f"state holds {S} sequences, expected {B} without slots")
    with _scope(dev, stream, q, k, v, g, beta, state, slots, o):
        o = _output("o", o, (B, T, H, DV), q.dtype, dev)
        bnd._check(lib.ss1d_delta_step(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
            state.data_ptr(), _ptr(slots), o.data_ptr(), B, T, S, HK, H, DK, DV, strides,
            DK ** -0.5 if scale is None else scale, code, _handle(dev, stream)))
    return o
