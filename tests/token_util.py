"""Bounds by norms for the token-order scan and the group norm: the error of a whole gradient against the
norm of the magnitudes that went into it, which stays far below the gradient itself.

A value of fp32 carries some tens of half steps of 2^-24: a state and its adjoint 8 per token over the 20
or so tokens that a state remembers, in quadrature 36 each; 20 for the products, 6 for a sum over 32 states
and 24 for one over 560 tokens.  In quadrature that is 60; 128 are allowed, of the sum of the terms'
magnitudes.  An output of bfloat16 is off by half a step of the value more."""
from __future__ import annotations

import torch

from tests import scan_util as su

STEPS = 128 * su.F32_HALF


def magnitudes(t, cu=None):
    """The sums of the absolute values of what each output and gradient of the scan adds up, in float64:
    y, the end states ("ht"), and the gradients by the names of su.adjoint."""
    c = su._doubles(t)
    A, D = c["A"], c["u"].shape[2]
    G, N = c["Bs"].shape[2:]
    rep = D // G
    a = {n: c[n].abs() for n in ("u", "Bs", "Cs", "Ds", "dy")}
    m = {n: torch.zeros_like(c[n]) for n in su.NAMES}
    m["y"] = torch.zeros_like(c["u"])
    rows = su.sequences(t, cu)
    m["h0"], m["ht"] = torch.zeros(len(rows), D, N).double(), torch.zeros(len(rows), D, N).double()
    gate, g = 1.0, a["dy"]
    if c["z"] is not None:
        gate = (c["z"] * torch.sigmoid(c["z"])).abs()
        g = g * gate
        m["z"] = torch.zeros_like(c["z"])
    for i, (b, s, e) in enumerate(rows):
        h = c["h0"][i].abs() if c["h0"] is not None else torch.zeros_like(A)
        states = [h]
        for j in range(s, e):
            decay = (c["delta"][b, j][:, None] * A).exp()
            Bt = a["Bs"][b, j].repeat_interleave(rep, 0)
            h = decay * h + (c["delta"][b, j] * a["u"][b, j])[:, None] * Bt
            states.append(h)
        m["ht"][i] = h
        lam = c["dht"][i].abs() if c["dht"] is not None else torch.zeros_like(A)
        for j in range(e - 1, s - 1, -1):
            at, h = (b, j), states[j - s + 1]
            Bt, Ct = (a[n][at].repeat_interleave(rep, 0) for n in ("Bs", "Cs"))
            delta = c["delta"][at]
            lam = lam + g[at][:, None] * Ct
            plain = (h * Ct).sum(1) + a["Ds"] * a["u"][at]
            if c["z"] is not None:
                m["z"][at] = a["dy"][at] * 1.1 * plain  # the slope of SiLU is at most 1.1
            m["Cs"][at] = (g[at][:, None] * h).view(G, -1, N).sum(1)
            m["Bs"][at] = (lam * (delta * a["u"][at])[:, None]).view(G, -1, N).sum(1)
            decay = (delta[:, None] * A).exp()
            w, q = lam * decay * states[j - s], (lam * Bt).sum(1)
            m["A_log"] += w * delta[:, None] * A.abs()
            m["dt_raw"][at] = ((w * A.abs()).sum(1) + q * a["u"][at]) * c["slope"][at]
            m["u"][at] = delta * q + a["Ds"] * g[at]
            m["Ds"] += g[at] * a["u"][at]
            m["y"][at] = plain * (gate[at] if c["z"] is not None else 1.0)
            lam = lam * decay
        m["h0"][i] = lam
    m["dt_bias"] = m["dt_raw"].sum((0, 1))
    return m


def allowed(ref, mag, dtype):
    """The norm of the error that is allowed; far below the result's, or the check would say nothing."""
    bound = STEPS * float(mag.norm()) + su.half(dtype) * float(ref.norm())
    assert bound <= 0.02 * float(ref.norm()), "the bound says nothing"
    return bound


def check_norm(got, ref, mag, what, dtype=torch.float32):
    got, ref = got.double().cpu(), ref.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{what}: not finite"
    if not float(ref.abs().sum()):
        assert not got.any(), what
        return
    err, bound = float((got - ref).norm()), allowed(ref, mag.double().cpu(), dtype)
    assert err <= bound, f"{what}: off by {err:.3e} against {bound:.3e}"


def check_scan(t, y, ht, got, cu=None):
    """y, the end states and the gradients (each may be None) against 64 bits."""
    mag = magnitudes(t, cu)
    dtype = t["u"].dtype
    if y is not None:
        y64, h64, _ = su.reference(t, cu)
        check_norm(y, y64, mag["y"], "y", dtype)
        check_norm(ht, h64, mag["ht"], "end states")
    if got is None:
        return
    ref, _ = su.adjoint(t, cu)
    for n in list(su.NAMES) + (["z"] if t["z"] is not None else []):
        check_norm(got[n], ref[n], mag[n], "d" + n, got[n].dtype)
    if t["h0"] is not None:
        check_norm(got["initial_state"], ref["h0"], mag["h0"], "dh0")
