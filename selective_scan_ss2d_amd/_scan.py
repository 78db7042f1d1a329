"""Binding of the token-order selective scan (``ss1d_scan_*`` of ``include/ss2d.h``).

Argument checks and marshalling only; every step runs in the library's HIP kernels.
"""
from __future__ import annotations

import ctypes

from . import _binding as bnd
from ._binding import _torch
from ._call import (code_of, expect, handle, output, packed_sequences, ptr, rows, scope, scratch)


def _inputs(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z):
    """Checks the scan's inputs; (B, L, D, G, N), the data type's code and the strides (None for
    contiguous tensors)."""
    torch = _torch()
    if not (isinstance(u, torch.Tensor) and isinstance(Bs, torch.Tensor)):
        raise TypeError("u and Bs must be torch.Tensors")
    if u.dim() != 3 or Bs.dim() != 4:
        raise ValueError("u must be (B, L, D) and Bs (B, L, G, N)")
    dev, dtype = u.device, u.dtype
    if dev.type != "cuda":
        raise ValueError("u must be a GPU tensor")
    code = code_of(dtype)
    if code is None:
        raise TypeError(f"u must be float32 or bfloat16, not {dtype}")
    shape = u.shape
    B, L, D = shape
    G, N = Bs.shape[2], Bs.shape[3]
    if G < 1 or D % G:
        raise ValueError(f"Bs has {G} groups, expected a divisor of u's {D} channels")
    whole = rows("u", u, shape, dtype, dev) & rows("dt_raw", dt_raw, shape, dtype, dev)
    whole &= rows("Bs", Bs, (B, L, G, N), dtype, dev) & rows("Cs", Cs, (B, L, G, N), dtype, dev)
    if z is not None:
        whole &= rows("z", z, shape, dtype, dev)
    f32 = torch.float32
    expect("A_log", A_log, (D, N), f32, dev)
    expect("Ds", Ds, (D,), f32, dev)
    expect("dt_bias", dt_bias, (D,), f32, dev)
    strides = None
    if not whole:
        strides = (ctypes.c_int64 * 12)(*u.stride()[:2], *dt_raw.stride()[:2],
                                        *(u if z is None else z).stride()[:2], *Bs.stride()[:3],
                                        *Cs.stride()[:3])
    return (B, L, D, G, N), code, strides


def _forward(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z, cu_seqlens, initial_state, final_state, y,
             stream, save):
    torch, lib = _torch(), bnd.load_library()
    (B, L, D, G, N), code, strides = _inputs(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z)
    dev = u.device
    S = packed_sequences(cu_seqlens, B, dev)
    if initial_state is not None:
        expect("initial_state", initial_state, (S, D, N), torch.float32, dev)
    given = final_state if isinstance(final_state, torch.Tensor) else None
    with scope(dev, stream, u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z, cu_seqlens, initial_state, y,
               given):
        y = output("y", y, (B, L, D), u.dtype, dev)
        ht = saved = None
        if final_state is not False and final_state is not None:
            ht = output("final_state", given, (S, D, N), torch.float32, dev)
        packed = cu_seqlens is not None
        if save:
            size = lib.ss1d_scan_saved_bytes(B, L, S, D, N, packed)
            saved = torch.empty(max(0, size), dtype=torch.uint8, device=dev)
        size = lib.ss1d_scan_scratch_bytes(0, save, B, L, S, D, G, N, code, packed)
        ws = scratch(size, dev) if size else None
        bnd._check(lib.ss1d_scan_forward(
            u.data_ptr(), dt_raw.data_ptr(), A_log.data_ptr(), Bs.data_ptr(), Cs.data_ptr(),
            Ds.data_ptr(), dt_bias.data_ptr(), ptr(z), ptr(initial_state), ptr(cu_seqlens),
            y.data_ptr(), ptr(ht), ptr(saved), ptr(ws), 0 if ws is None else ws.numel(), B, L, S, D,
            G, N, strides, code, handle(dev, stream)))
    return y, ht, saved


def ss1d_scan_forward(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z=None, cu_seqlens=None,
                      initial_state=None, final_state=False, y=None, stream=None):
    """The selective scan in token order, over whole sequences.

    Per sequence and channel, from a state h (N), zero or ``initial_state``, per token:
    delta = softplus(dt_raw + dt_bias); h_n <- exp(-exp(A_log_n) delta) h_n + delta B_n u;
    y = (sum_n C_n h_n + Ds u) * SiLU(z) (without z: no gate).
    u, dt_raw, z (B, L, D) and Bs, Cs (B, L, G, N) float32 or bfloat16, last axis contiguous; D a
    multiple of G (channel d reads group d // (D // G)), N <= 32; A_log (D, N), Ds and dt_bias (D)
    float32.

    cu_seqlens: int32 offsets (S + 1) of S sequences packed into the tokens of B = 1 (tokens
    outside of them are left as they are in y).  initial_state (S, D, N) float32.  Returns y
    (B, L, D); with final_state True (or a tensor to write, which may be initial_state itself)
    the pair (y, end states (S, D, N) float32).
    """
    y, ht, _ = _forward(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z, cu_seqlens, initial_state,
                        final_state, y, stream, False)
    return y if ht is None else (y, ht)


def ss1d_scan_forward_save(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z=None, cu_seqlens=None,
                           initial_state=None, final_state=False, y=None, stream=None):
    """The training forward: ss1d_scan_forward, and the buffer that ss1d_scan_backward starts
    from.  Returns (y, saved), with final_state (y, end states, saved)."""
    y, ht, saved = _forward(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z, cu_seqlens, initial_state,
                            final_state, y, stream, True)
    return (y, saved) if ht is None else (y, ht, saved)


def ss1d_scan_backward(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, dy, z=None, cu_seqlens=None,
                       initial_state=None, dstate=None, saved=None, stream=None):
    """Gradients of sum(dy * y) + sum(dstate * end states) for ss1d_scan_forward's outputs on the
    same inputs: a dict with those of u, dt_raw, A_log, Bs, Cs, Ds and dt_bias, and of z and
    initial_state if they are given, contiguous, each with its input's shape and dtype.

    dy: contiguous, y's shape and dtype; dstate: float32 (S, D, N) or None.  saved: the buffer of
    ss1d_scan_forward_save for the same inputs; None computes it again.  Rows outside of every
    packed sequence are zero.
    """
    torch, lib = _torch(), bnd.load_library()
    (B, L, D, G, N), code, strides = _inputs(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z)
    dev = u.device
    S = packed_sequences(cu_seqlens, B, dev)
    packed = cu_seqlens is not None
    expect("dy", dy, (B, L, D), u.dtype, dev)
    for name, t in (("initial_state", initial_state), ("dstate", dstate)):
        if t is not None:
            expect(name, t, (S, D, N), torch.float32, dev)
    if saved is not None:
        size = lib.ss1d_scan_saved_bytes(B, L, S, D, N, packed)
        expect("saved", saved, (max(0, size),), torch.uint8, dev)
    with scope(dev, stream, u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z, dy, cu_seqlens, initial_state,
               dstate, saved):
        make = torch.zeros if packed else torch.empty  # rows outside of every sequence are not written
        d = {n: (torch.empty if n in ("A_log", "Ds", "dt_bias") else make)(t.shape, dtype=t.dtype, device=dev)
             for n, t in (("u", u), ("dt_raw", dt_raw), ("A_log", A_log), ("Bs", Bs), ("Cs", Cs),
                          ("Ds", Ds), ("dt_bias", dt_bias))}
        if z is not None:
            d["z"] = make(z.shape, dtype=z.dtype, device=dev)
        if initial_state is not None:
            d["initial_state"] = torch.empty_like(initial_state)
        ws = scratch(lib.ss1d_scan_scratch_bytes(1, saved is not None, B, L, S, D, G, N, code,
                                                 packed), dev)
        bnd._check(lib.ss1d_scan_backward(
            u.data_ptr(), dt_raw.data_ptr(), A_log.data_ptr(), Bs.data_ptr(), Cs.data_ptr(),
            Ds.data_ptr(), dt_bias.data_ptr(), ptr(z), ptr(initial_state), ptr(cu_seqlens),
            ptr(saved), dy.data_ptr(), ptr(dstate), d["u"].data_ptr(), d["dt_raw"].data_ptr(),
            d["A_log"].data_ptr(), d["Bs"].data_ptr(), d["Cs"].data_ptr(), d["Ds"].data_ptr(),
            d["dt_bias"].data_ptr(), ptr(d.get("z")), ptr(d.get("initial_state")), ws.data_ptr(),
            ws.numel(), B, L, S, D, G, N, strides, code, handle(dev, stream)))
    return d


def ss1d_scan_step(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, state, z=None, slots=None, y=None,
                   stream=None):
    """The selective scan for T (few) tokens of each of B sequences, states in place.

    u, dt_raw, z (B, T, D), Bs, Cs (B, T, G, N) and the parameters as in ss1d_scan_forward; state
    (S, D, N) float32, updated in place.  Row b's state is state[slots[b]] (int32 slots (B)), or
    state[b].  Rows with a slot outside 0 .. S - 1 are padding and their rows of y stay as they
    are; rows that name one slot are successive tokens of one sequence, in row order.  Returns y
    (B, T, D).
    """
    torch, lib = _torch(), bnd.load_library()
    (B, T, D, G, N), code, strides = _inputs(u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, z)
    dev = u.device
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be (S, D, N)")
    S = state.shape[0]
    expect("state", state, (S, D, N), torch.float32, dev)
    if slots is not None:
        expect("slots", slots, (B,), torch.int32, dev)
    elif S != B:
        raise ValueError(f"state holds {S} sequences, expected {B} without slots")
    with scope(dev, stream, u, dt_raw, A_log, Bs, Cs, Ds, dt_bias, state, z, slots, y):
        y = output("y", y, (B, T, D), u.dtype, dev)
        bnd._check(lib.ss1d_scan_step(
            u.data_ptr(), dt_raw.data_ptr(), A_log.data_ptr(), Bs.data_ptr(), Cs.data_ptr(),
            Ds.data_ptr(), dt_bias.data_ptr(), ptr(z), state.data_ptr(), ptr(slots), y.data_ptr(), B,
            T, S, D, G, N, strides, code, handle(dev, stream)))
    return y
