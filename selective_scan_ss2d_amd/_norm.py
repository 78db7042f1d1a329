"""Binding of the block norm (``ss2d_norm_*`` of ``include/ss2d.h``).

Argument checks and marshalling only; every step runs in the library's HIP kernels.
"""
from __future__ import annotations

from . import _binding as bnd
from ._binding import _torch
from ._call import code_of, expect, handle, output, ptr, scope, scratch


def _shape(h, channels_first):
    """(B, L, D) of h and the data type's code."""
    if not isinstance(h, _torch().Tensor):
        raise TypeError("h must be a torch.Tensor")
    if h.device.type != "cuda":
        raise ValueError("h must be a GPU tensor")
    code = code_of(h.dtype)
    if code is None:
        raise TypeError(f"h must be float32 or bfloat16, not {h.dtype}")
    if h.dim() < (3 if channels_first else 1):
        raise ValueError("h must be (B, D, ...) with channels first, else (..., D)")
    if not h.is_contiguous():
        raise ValueError("h must be contiguous")
    if channels_first:
        B, D = h.shape[0], h.shape[1]
        return (B, h.shape[2:].numel(), D), code
    D = h.shape[-1]
    return (h.shape[:-1].numel(), 1, D), code


def _vectors(D, dev, rows, res_scale, **vectors):
    for name, w in vectors.items():
        if w is not None:
            expect(name, w, (D,), _torch().float32, dev)
    for norm in ("post", "pre"):
        if vectors.get("b_" + norm) is not None and vectors["w_" + norm] is None:
            raise ValueError(f"b_{norm} needs w_{norm}")
    if res_scale is None:
        return 0
    G = res_scale.shape[0] if res_scale.dim() == 2 else 1
    if res_scale.dim() == 1:
        res_scale = res_scale[None]
    expect("res_scale", res_scale, (G, D), _torch().float32, dev)
    if G < 1 or rows % G:
        raise ValueError(f"res_scale has {G} rows, expected a divisor of {rows}")
    return G


def ss2d_norm_forward(h, residual=None, w_post=None, b_post=None, z=None, res_scale=None,
                      w_pre=None, b_pre=None, layer=False, eps=1e-6, channels_first=False,
                      y=None, n=None, stream=None):
    """The norms around a block, its gate, residual scale and residual in one pass.

    p = Norm(h; w_post, b_post) (h without w_post); p <- p * SiLU(z) (with z);
    y = residual + res_scale * p; n = Norm(y; w_pre, b_pre).  Norm is the root-mean-square
    norm, or with layer=True the layer norm, over the last axis of h, or with
    channels_first=True over axis 1 of (B, D, ...).

    h and z: float32 or bfloat16; residual: h's dtype or float32, which is then y's; w_*, b_*
    (D) float32; res_scale (D) or (G, D) float32, row g for the g-th of G equal runs of rows
    (channels first: of images).  Returns (y, n), n None without w_pre; y is h itself if
    nothing but the second norm is asked for.  y may be given as the residual (in place).
    """
    torch, lib = _torch(), bnd.load_library()
    (B, L, D), code = _shape(h, channels_first)
    dev = h.device
    G = _vectors(D, dev, B if channels_first else B * L, res_scale, w_post=w_post, b_post=b_post,
                 w_pre=w_pre, b_pre=b_pre)
    if z is not None:
        expect("z", z, h.shape, h.dtype, dev)
    ytype = h.dtype
    if residual is not None:
        if residual.dtype not in (h.dtype, torch.float32):
            raise TypeError(f"residual has dtype {residual.dtype}, expected {h.dtype} or float32")
        ytype = residual.dtype
        expect("residual", residual, h.shape, ytype, dev)
    if n is not None and w_pre is None:
        raise ValueError("n needs w_pre")
    alone = w_post is None and z is None and residual is None and res_scale is None
    if alone and w_pre is None:
        raise ValueError("nothing to compute: give w_post, z, residual, res_scale or w_pre")
    with scope(dev, stream, h, z, residual, res_scale, w_post, b_post, w_pre, b_pre, y, n):
        if alone and y is None:
            kept = None
        else:
            y = kept = output("y", y, h.shape, ytype, dev)
        n = output("n", n, h.shape, h.dtype, dev) if w_pre is not None else None
        bnd._check(lib.ss2d_norm_forward(
            h.data_ptr(), ptr(z), ptr(residual), ptr(res_scale), ptr(w_post), ptr(b_post),
            ptr(w_pre), ptr(b_pre), ptr(kept), ptr(n), B, L, D, G, 1 if channels_first else 0,
            1 if layer else 0, eps, code, code_of(ytype), handle(dev, stream)))
    return (h if kept is None else y), n


def ss2d_norm_backward(h, y=None, dy=None, dn=None, residual=True, w_post=None, b_post=None, z=None,
                       res_scale=None, w_pre=None, b_pre=None, layer=False, eps=1e-6,
                       channels_first=False, stream=None):
    """Gradients of sum(dy * y) + sum(dn * n) for ss2d_norm_forward's outputs on the same inputs.

    y: the forward's, as stored (needed with w_pre); dy: y's dtype, None for no gradient at y;
    dn: with w_pre.  residual: whether there was one, of y's dtype.  Returns a dict with the
    gradients of h and of what was given of residual, z, res_scale, w_post, b_post, w_pre and
    b_pre, each with its input's shape.
    """
    torch, lib = _torch(), bnd.load_library()
    (B, L, D), code = _shape(h, channels_first)
    dev = h.device
    G = _vectors(D, dev, B if channels_first else B * L, res_scale, w_post=w_post, b_post=b_post,
                 w_pre=w_pre, b_pre=b_pre)
    if (dn is None) != (w_pre is None):
        raise ValueError("dn and w_pre go together")
    if w_pre is not None and y is None:
        raise ValueError("the second norm's backward needs y")
    if dy is None and dn is None:
        raise ValueError("give dy, dn or both")
    ytype = (y if y is not None else dy).dtype
    if ytype not in (h.dtype, torch.float32):
        raise TypeError(f"y has dtype {ytype}, expected {h.dtype} or float32")
    for name, t, dtype in (("z", z, h.dtype), ("dn", dn, h.dtype), ("y", y, ytype),
                           ("dy", dy, ytype)):
        if t is not None:
            expect(name, t, h.shape, dtype, dev)
    with scope(dev, stream, h, y, dy, dn, z, res_scale, w_post, b_post, w_pre):
        d = {"h": torch.empty_like(h)}
        if residual:
            d["residual"] = torch.empty(h.shape, dtype=ytype, device=dev)
        for name, t in (("z", z), ("res_scale", res_scale), ("w_post", w_post),
                        ("b_post", b_post), ("w_pre", w_pre), ("b_pre", b_pre)):
            if t is not None:
                d[name] = torch.empty_like(t)
        ws = scratch(lib.ss2d_norm_scratch_bytes(B, L, D, G, 1 if channels_first else 0), dev)
        bnd._check(lib.ss2d_norm_backward_ws(
            h.data_ptr(), ptr(z), ptr(res_scale), ptr(w_post), ptr(b_post), ptr(w_pre), ptr(y),
            ptr(dy), ptr(dn), d["h"].data_ptr(), *[ptr(d.get(k)) for k in
                                                   ("z", "residual", "res_scale", "w_post",
                                                    "b_post", "w_pre", "b_pre")],
            ws.data_ptr(), ws.numel(), B, L, D, G, 1 if channels_first else 0, 1 if layer else 0,
            eps, code, code_of(ytype), handle(dev, stream)))
    return d
