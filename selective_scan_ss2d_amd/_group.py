"""Binding of the group norm (``ss2d_group_norm_*`` of ``include/ss2d.h``).

Argument checks and marshalling only; every step runs in the library's HIP kernels.
"""
from __future__ import annotations

from . import _binding as bnd
from ._binding import _torch
from ._call import code_of, expect, handle, output, ptr, scope, scratch


def _shape(x, groups, weight, bias):
    """(B, L, C) of x and the data type's code."""
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.device.type != "cuda":
        raise ValueError("x must be a GPU tensor")
    code = code_of(x.dtype)
    if code is None:
        raise TypeError(f"x must be float32 or bfloat16, not {x.dtype}")
    if x.dim() < 2:
        raise ValueError("x must be (B, ..., C)")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    B, C = x.shape[0], x.shape[-1]
    if groups < 1 or C < 1 or C % groups:
        raise ValueError(f"groups is {groups}, expected a divisor of x's {C} channels")
    for name, w in (("weight", weight), ("bias", bias)):
        if w is not None:
            expect(name, w, (C,), torch.float32, x.device)
    return (B, x.shape[1:-1].numel(), C), code


def ss2d_group_norm_forward(x, groups, weight=None, bias=None, silu=True, eps=1e-5, stats=False,
                            y=None, stream=None):
    """The group norm with its activation, channels last.

    y = act((x - mean) / sqrt(var + eps) * weight + bias) with mean and var over the positions and
    the C / groups channels of a group of each of the B images; act is SiLU, or nothing with
    silu=False.  x (B, ..., C) float32 or bfloat16, contiguous; weight and bias (C) float32.
    Returns y, or with stats=True the pair (y, stats (B, groups, 2) float32), the groups' mean and
    1 / sqrt(var + eps) (0 and 1 / sqrt(eps) without positions), which the backward takes.
    """
    torch, lib = _torch(), bnd.load_library()
    (B, L, C), code = _shape(x, groups, weight, bias)
    dev = x.device
    with scope(dev, stream, x, weight, bias, y):
        y = output("y", y, x.shape, x.dtype, dev)
        kept = torch.empty((B, groups, 2), dtype=torch.float32, device=dev) if stats else None
        size = lib.ss2d_group_norm_scratch_bytes(0, kept is not None, B, L, C, groups, code)
        ws = scratch(size, dev) if size else None
        bnd._check(lib.ss2d_group_norm_forward(
            x.data_ptr(), ptr(weight), ptr(bias), y.data_ptr(), ptr(kept), ptr(ws),
            0 if ws is None else ws.numel(), B, L, C, groups, 1 if silu else 0, eps, code,
            handle(dev, stream)))
    return (y, kept) if stats else y


def ss2d_group_norm_backward(x, dy, groups, weight=None, bias=None, silu=True, eps=1e-5, stats=None,
                             stream=None):
    """Gradients of sum(dy * y) for ss2d_group_norm_forward's y on the same inputs: a dict with
    those of x, and of weight and bias if they are given.

    dy: contiguous, x's shape and dtype.  stats: the forward's for the same x; None computes them
    again.
    """
    torch, lib = _torch(), bnd.load_library()
    (B, L, C), code = _shape(x, groups, weight, bias)
    dev = x.device
    expect("dy", dy, x.shape, x.dtype, dev)
    if stats is not None:
        expect("stats", stats, (B, groups, 2), torch.float32, dev)
    with scope(dev, stream, x, dy, weight, bias, stats):
        d = {"x": torch.empty_like(x)}
        for name, w in (("weight", weight), ("bias", bias)):
            if w is not None:
                d[name] = torch.empty_like(w)
        ws = scratch(lib.ss2d_group_norm_scratch_bytes(1, stats is not None, B, L, C, groups, code),
                     dev)
        bnd._check(lib.ss2d_group_norm_backward(
            x.data_ptr(), ptr(weight), ptr(bias), ptr(stats), dy.data_ptr(), d["x"].data_ptr(),
            ptr(d.get("weight")), ptr(d.get("bias")), ws.data_ptr(), ws.numel(), B, L, C, groups,
            1 if silu else 0, eps, code, handle(dev, stream)))
    return d
