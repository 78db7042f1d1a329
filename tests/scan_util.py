"""Inputs, the definition in 64 bits (token by token, with its adjoint) and the error bounds shared
by the tests of the token-order scan and its convolution."""
from __future__ import annotations

import math

import torch

NAMES = ("u", "dt_raw", "A_log", "Bs", "Cs", "Ds", "dt_bias")
BF16_HALF = 2.0 ** -8   # half a step of bfloat16 relative to the value (eps / 2)
F32_HALF = 2.0 ** -24


def half(dtype):
    return BF16_HALF if dtype == torch.bfloat16 else 0.0


def make_inputs(B, L, D, G, N, dtype, seed=0, gate=True, h0=0, views=False, device="cpu"):
    """Seeded inputs; delta about 0.05 to 0.7; h0 > 0 adds that many initial states; views: u and z,
    B and C lie side by side in wider tensors."""
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    def pair(*shape):
        if not views:
            return normal(*shape).to(dtype).to(device), normal(*shape).to(dtype).to(device)
        wide = normal(*shape[:2], 3 + 2 * math.prod(shape[2:])).to(dtype).to(device)
        w = math.prod(shape[2:])
        return tuple(wide[..., 3 + i * w:3 + (i + 1) * w].unflatten(-1, shape[2:]) for i in range(2))

    u, z = pair(B, L, D)
    Bs, Cs = pair(B, L, G, N)
    t = dict(u=u, dt_raw=normal(B, L, D).to(dtype).to(device),
             A_log=(torch.arange(1, N + 1).float().log() + 0.2 * normal(D, N)).to(device), Bs=Bs, Cs=Cs,
             Ds=(1 + 0.2 * normal(D)).to(device), dt_bias=(0.3 * normal(D) - 1.5).to(device))
    t["z"] = z if gate else None
    t["h0"] = (0.3 * normal(h0, D, N)).to(device) if h0 else None
    t["dy"] = normal(B, L, D).to(dtype).to(device)
    t["dht"] = (0.5 * normal(h0, D, N)).to(device) if h0 else None
    return t


def sequences(t, cu=None):
    """(row, first token, end) of every sequence."""
    if cu is None:
        return [(b, 0, t["u"].shape[1]) for b in range(t["u"].shape[0])]
    return [(0, int(a), int(e)) for a, e in zip(cu[:-1], cu[1:])]


def scan(u, delta, A, Bs, Cs, Ds, h):
    """One sequence in float64: u, delta (L, D), A (D, N), Bs, Cs (L, G, N), h (D, N).  Returns the
    ungated y, the states before every token and at the end."""
    rep = A.shape[0] // Bs.shape[1]
    ys, states = [], [h]
    for i in range(u.shape[0]):
        Bt, Ct = (x[i].repeat_interleave(rep, 0) for x in (Bs, Cs))
        h = (delta[i][:, None] * A).exp() * h + (delta[i] * u[i])[:, None] * Bt
        states.append(h)
        ys.append((h * Ct).sum(1) + Ds * u[i])
    return (torch.stack(ys) if ys else torch.zeros_like(u)), states


def _doubles(t):
    c = {n: t[n].detach().double().cpu() for n in NAMES}
    c["A"] = -c["A_log"].exp()
    v = c["dt_raw"] + c["dt_bias"]
    c["delta"] = torch.nn.functional.softplus(v, threshold=1e3)
    c["slope"] = torch.sigmoid(v)
    for n in ("z", "h0", "dy", "dht"):
        c[n] = t[n].double().cpu() if t.get(n) is not None else None
    return c


def reference(t, cu=None):
    """y, the end states in float64, and the largest |h| and |delta u B| on the way."""
    c = _doubles(t)
    y, ends, hm = torch.zeros_like(c["u"]), [], 1e-6
    for i, (b, s, e) in enumerate(sequences(t, cu)):
        h = c["h0"][i] if c["h0"] is not None else torch.zeros_like(c["A"])
        y[b, s:e], states = scan(*(c[n][b, s:e] for n in ("u", "delta")), c["A"],
                                 *(c[n][b, s:e] for n in ("Bs", "Cs")), c["Ds"], h)
        ends.append(states[-1])
        hm = max([hm] + [float(x.abs().max()) for x in states if x.numel()])
    if c["z"] is not None:
        y = y * c["z"] * torch.sigmoid(c["z"])
    return y, torch.stack(ends), hm


def top(x):
    return float(x.abs().max()) if x is not None and x.numel() else 0.0


def longest(t, cu=None):
    return max(e - s for _, s, e in sequences(t, cu))


def state_bound(t, hm, cu=None):
    """The absolute error allowed of a state in fp32.  A token rounds it at most 8 times: its decay
    is off by 6 half steps at most (delta 3, A 2 and the exponential 1, and x exp(-x) < 0.4), the
    sum and product round once each; and delta u B, off by 6 of its own.  Decays are below 1, so
    that the errors of L tokens at most add."""
    c = _doubles(t)
    wm = top(c["delta"]) * top(c["u"]) * top(c["Bs"])
    return F32_HALF * (longest(t, cu) + 1) * (8 * hm + 6 * wm)


def y_bounds(t, hm, cu=None):
    """(absolute, relative) bounds of y: N states' errors times C, the sum's N roundings, the gate's
    6 half steps, and the rounding to the data type."""
    c = _doubles(t)
    N, cm = c["A"].shape[1], top(c["Cs"])
    gate = max(1.0, top(c["z"])) if c["z"] is not None else 1.0
    err = N * cm * state_bound(t, hm, cu) + F32_HALF * (N + 8) * (N * cm * hm + 2 * top(c["u"]) * top(c["Ds"]))
    return gate * err, half(t["u"].dtype)


def check(got, ref, what, abs_tol, rel=0.0):
    got = got.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    if not got.numel():
        return
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got - ref).abs()
    worst = float((err - rel * ref.abs()).max())
    assert worst <= abs_tol, f"{what}: off by {float(err.max()):.3e}, {worst:.3e} against {abs_tol:.3e}"


def adjoint(t, cu=None):
    """The gradients of sum(dy * y) + sum(dht * end states) in float64 token by token, and a bound of
    the absolute error of each in fp32."""
    c = _doubles(t)
    A, D = c["A"], c["u"].shape[2]
    G, N = c["Bs"].shape[2:]
    d = {n: torch.zeros_like(c[n]) for n in NAMES}
    d["h0"] = torch.zeros(len(sequences(t, cu)), D, N).double()
    z, g = c["z"], c["dy"]
    if z is not None:
        sg = torch.sigmoid(z)
        d["z"], g = torch.zeros_like(z), g * z * sg
    hm = lm = 1e-6
    for i, (b, s, e) in enumerate(sequences(t, cu)):
        h = c["h0"][i] if c["h0"] is not None else torch.zeros_like(A)
        part = [c[n][b, s:e] for n in ("u", "delta")] + [A] + [c[n][b, s:e] for n in ("Bs", "Cs")]
        y, states = scan(*part, c["Ds"], h)
        if z is not None:
            d["z"][b, s:e] = c["dy"][b, s:e] * y * (sg * (1 + z * (1 - sg)))[b, s:e]
        carry = c["dht"][i] if c["dht"] is not None else torch.zeros_like(A)
        hm = max([hm] + [top(x) for x in states])
        for j in range(e - s - 1, -1, -1):
            at = (b, s + j)
            Bt, Ct = (c[n][at].repeat_interleave(D // G, 0) for n in ("Bs", "Cs"))
            lam = g[at][:, None] * Ct + carry
            lm = max(lm, top(lam))
            a = (c["delta"][at][:, None] * A).exp()
            d["Cs"][at] = (g[at][:, None] * states[j + 1]).view(G, -1, N).sum(1)
            d["Bs"][at] = (lam * (c["delta"][at] * c["u"][at])[:, None]).view(G, -1, N).sum(1)
            q = (lam * Bt).sum(1)
            w = lam * a * states[j]
            d["A_log"] += w * c["delta"][at][:, None] * A
            d["dt_raw"][at] = ((w * A).sum(1) + q * c["u"][at]) * c["slope"][at]
            d["u"][at] = c["delta"][at] * q + c["Ds"] * g[at]
            d["Ds"] += g[at] * c["u"][at]
            carry = lam * a
        d["h0"][i] = carry
    d["dt_bias"] = d["dt_raw"].sum((0, 1))
    # bounds: a gradient's products carry the errors of its factors, eh of h, el of lambda (as the
    # state's: gates and C in place of delta u and B), and round once or twice each
    um, dm, bm, cm, am = (top(c[n]) for n in ("u", "delta", "Bs", "Cs", "A"))
    gm, T = top(g), c["u"].shape[0] * c["u"].shape[1]
    eh = state_bound(t, hm, cu)
    el = F32_HALF * (longest(t, cu) + 1) * (8 * lm + 8 * gm * cm)
    r = 16 * F32_HALF
    wide = am * (lm * eh + hm * el + (r + N * F32_HALF) * lm * hm)  # one term of sum A w
    back = bm * (el + (r + N * F32_HALF) * lm)                      # one term of sum lambda B
    eraw = N * (wide + um * back)
    bounds = dict(u=N * dm * back + r * (N * dm * bm * lm + top(c["Ds"]) * gm), dt_raw=eraw,
                  Bs=(D // G) * um * dm * (el + (r + D * F32_HALF) * lm),
                  Cs=(D // G) * (gm * eh + (r + D * F32_HALF) * gm * hm),
                  A_log=T * dm * wide + T * F32_HALF * T * dm * am * lm * hm, Ds=T * (r + T * F32_HALF) * gm * um,
                  dt_bias=T * eraw + T * F32_HALF * top(d["dt_raw"]) * T, h0=el + r * lm)
    if z is not None:
        ym = N * cm * hm + top(c["Ds"]) * um
        bounds["z"] = top(c["dy"]) * 1.1 * (N * cm * eh + (r + N * F32_HALF) * ym)
    return d, bounds


class plan:
    """Forces the scan's segment length (tokens; 0: whole sequences) and the lanes of a channel in the
    forward (0: the rule's) for this thread's calls inside the block."""

    def __init__(self, tokens=-1, lanes=0):
        self.tokens, self.lanes = tokens, lanes

    def __enter__(self):
        from selective_scan_ss2d_amd import _binding as bnd
        assert bnd.load_library().ss1d_scan_set_plan(self.lanes, self.tokens) == 0

    def __exit__(self, *exc):
        from selective_scan_ss2d_amd import _binding as bnd
        bnd.load_library().ss1d_scan_set_plan(0, -1)


# ---- the convolution -------------------------------------------------------------------------
def conv_inputs(B, L, D, KW, dtype, seed=0, bias=True, h0=0, views=False, device="cpu"):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(B, L, 2 * D + 5 if views else D, generator=gen).to(dtype).to(device)
    t = dict(x=x[..., 5:5 + D] if views else x, conv_w=torch.randn(D, KW, generator=gen).to(device))
    t["conv_b"] = torch.randn(D, generator=gen).to(device) if bias else None
    for n in ("h0", "dht"):
        t[n] = torch.randn(h0, KW - 1, D, generator=gen).to(dtype).to(device) if h0 else None
    t["dy"] = torch.randn(B, L, D, generator=gen).to(dtype).to(device)
    return t


def conv_reference(t, silu=True, cu=None, grads=False):
    """y and the final states in float64; with grads, the gradients of sum(dy * y) +
    sum(dht * final states)."""
    x, w = (t[n].detach().double().cpu().requires_grad_(grads) for n in ("x", "conv_w"))
    b, h0 = (t[n].detach().double().cpu().requires_grad_(grads) if t[n] is not None else None
             for n in ("conv_b", "h0"))
    KW, L = w.shape[1], x.shape[1]
    rows = [(i, 0, L) for i in range(x.shape[0])] if cu is None else \
        [(0, int(a), int(e)) for a, e in zip(cu[:-1], cu[1:])]
    loss, y, ends = 0.0, torch.zeros_like(x), []
    for i, (r, s, e) in enumerate(rows):
        before = h0[i] if h0 is not None else torch.zeros(KW - 1, x.shape[2]).double()
        whole = torch.cat([before, x[r, s:e]])
        v = sum(whole[j:j + e - s] * w[:, j] for j in range(KW))
        v = v if b is None else v + b
        v = v * torch.sigmoid(v) if silu else v
        y[r, s:e] = v.detach() if grads else v
        ends.append(whole[e - s:])
        if grads:
            loss = loss + (v * t["dy"][r, s:e].double().cpu()).sum()
            if t["dht"] is not None:
                loss = loss + (ends[-1] * t["dht"][i].double().cpu()).sum()
    ends = torch.stack([x.detach() for x in ends])
    if not grads:
        return y.detach(), ends
    names = [n for n, p in (("x", x), ("conv_w", w), ("conv_b", b), ("h0", h0)) if p is not None]
    leaves = [p for p in (x, w, b, h0) if p is not None]
    g = torch.autograd.grad(loss, leaves, allow_unused=True)
    return {n: torch.zeros_like(p) if v is None else v for n, p, v in zip(names, leaves, g)}
