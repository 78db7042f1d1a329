"""Inputs, the definition in 64 bits (token by token, with its adjoint) and the error bounds
shared by the tests of the gated delta rule."""
from __future__ import annotations

import torch

NAMES = ("q", "k", "v", "g", "beta")
BF16_HALF = 2.0 ** -8   # half a step of bfloat16 relative to the value (eps / 2)
F32_HALF = 2.0 ** -24


def make_inputs(B, L, HK, H, DK, DV, dtype, seed=0, decay=0.1, h0=0):
    """Seeded inputs on the CPU in the data type: normalised keys and queries, log decays in
    (-2 decay, 0], beta in (0, 1); h0 > 0 adds that many initial states."""
    gen = torch.Generator().manual_seed(seed)

    def unit(*shape):
        x = torch.randn(shape, generator=gen)
        return (x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)).to(dtype)

    t = dict(q=unit(B, L, HK, DK), k=unit(B, L, HK, DK),
             v=torch.randn(B, L, H, DV, generator=gen).to(dtype),
             g=-2 * decay * torch.rand(B, L, H, generator=gen),
             beta=torch.sigmoid(torch.randn(B, L, H, generator=gen)))
    t["h0"] = 0.3 * torch.randn(h0, H, DK, DV, generator=gen) if h0 else None
    t["do"] = torch.randn(B, L, H, DV, generator=gen).to(dtype)
    return t


def to_gpu(t):
    return {n: x.cuda() if x is not None else None for n, x in t.items()}


def rule(q, k, v, g, beta, scale, S):
    """One sequence: q, k (L, HK, DK), v (L, H, DV), g, beta (L, H), S (H, DK, DV), float64.
    Returns o, the end state and the states before every token."""
    rep = v.shape[1] // q.shape[1]
    out, states = [], []
    for t in range(v.shape[0]):
        states.append(S)
        S = S * g[t].exp()[:, None, None]
        kt = k[t].repeat_interleave(rep, 0)
        u = beta[t][:, None] * (v[t] - (kt[:, :, None] * S).sum(1))
        S = S + kt[:, :, None] * u[:, None, :]
        out.append(scale * (q[t].repeat_interleave(rep, 0)[:, :, None] * S).sum(1))
    o = torch.stack(out) if out else torch.zeros_like(v)
    return o, S, states


def reference(t, scale, cu=None):
    """o and the end states in float64 for the dense rows, or the packed sequences of cu (rows
    outside of them zero)."""
    q, k, v, g, beta = (t[n].double() for n in NAMES)
    H, DK, DV = v.shape[2], q.shape[3], v.shape[3]
    parts = [(b, 0, v.shape[1]) for b in range(v.shape[0])] if cu is None else \
        [(0, int(a), int(e)) for a, e in zip(cu[:-1], cu[1:])]
    o, ends = torch.zeros_like(v), []
    for i, (b, s, e) in enumerate(parts):
        S = t["h0"][i].double() if t["h0"] is not None else torch.zeros(H, DK, DV).double()
        o[b, s:e], S, _ = rule(*[x[b, s:e] for x in (q, k, v, g, beta)], scale, S)
        ends.append(S)
    return o, torch.stack(ends)


def f32_bound(DK, ref, chunks=1):
    """The absolute error allowed of fp32 results: each is a chain of sums of DK + 5 * 32
    products (S^T k, the solve's two passes, P u, the update, and the gates), every term
    bounded by the results' own magnitude (the rule contracts), each addition rounding by
    half a step."""
    return F32_HALF * (DK + 5 * 32) * max(float(ref.abs().max()), 1e-6)


def check(got, ref, what, abs_tol, rel=0.0):
    err = (got.double().cpu() - ref).abs()
    over = err - rel * ref.abs() - abs_tol
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = float(over.max()) if over.numel() else -1.0
    assert worst <= 0, f"{what}: off by {float(err.max()):.3e}, {worst:.3e} over the bound"


def o_bounds(DK, ref, dtype):
    """(absolute, relative) bounds of o.  bfloat16: the rounding, and operands held in two
    bfloat16 terms (each off by at most 2^-17 of its value, DK and 32 products of the state's
    and the solution's magnitude: their sum in quadrature is below 16 of them)."""
    if dtype == torch.float32:
        return f32_bound(DK, ref), 0.0
    return f32_bound(DK, ref) + 16 * 2.0 ** -17 * float(ref.abs().max()), BF16_HALF


def adjoint(t, scale, cu=None, dstate=None):
    """The gradients of sum(do * o) + sum(dstate * end states) in float64, token by token."""
    q, k, v, g, beta = (t[n].double() for n in NAMES)
    H, DK, DV = v.shape[2], q.shape[3], v.shape[3]
    rep = H // q.shape[2]
    parts = [(b, 0, v.shape[1]) for b in range(v.shape[0])] if cu is None else \
        [(0, int(a), int(e)) for a, e in zip(cu[:-1], cu[1:])]
    d = {n: torch.zeros_like(x) for n, x in zip(NAMES, (q, k, v, g, beta))}
    first = []
    for i, (b, s, e) in enumerate(parts):
        S = t["h0"][i].double() if t["h0"] is not None else torch.zeros(H, DK, DV).double()
        _, _, states = rule(*[x[b, s:e] for x in (q, k, v, g, beta)], scale, S)
        dS = dstate[i].double() if dstate is not None else torch.zeros(H, DK, DV).double()
        for j in range(e - s - 1, -1, -1):
            at = (b, s + j)
            qt, kt = (x[at].repeat_interleave(rep, 0)[:, :, None] for x in (q, k))
            before = states[j] * g[at].exp()[:, None, None]
            r = v[at] - (kt * before).sum(1)
            u = beta[at][:, None] * r
            do = scale * t["do"][at].double()[:, None, :]
            d["q"][at] = ((before + kt * u[:, None, :]) * do).sum(2).view(-1, rep, DK).sum(1)
            dS = dS + qt * do
            du = (dS * kt).sum(1)
            d["beta"][at] = (du * r).sum(1)
            dr = beta[at][:, None] * du
            d["v"][at] = dr
            dk = (dS * u[:, None, :]).sum(2) - (before * dr[:, None, :]).sum(2)
            d["k"][at] = dk.view(-1, rep, DK).sum(1)
            dS = dS - kt * dr[:, None, :]
            d["g"][at] = (dS * before).sum((1, 2))
            dS = dS * g[at].exp()[:, None, None]
        first.append(dS)
    return d, torch.stack(first)


class segments:
    """Forces the forward's and backward's segment length (chunks of 32 tokens, even; 0: whole
    sequences) for this thread's calls inside the block."""

    def __init__(self, chunks):
        self.chunks = chunks

    def __enter__(self):
        from selective_scan_ss2d_amd import _binding as bnd
        assert bnd.load_library().ss1d_delta_set_segment(self.chunks) == 0

    def __exit__(self, *exc):
        from selective_scan_ss2d_amd import _binding as bnd
        bnd.load_library().ss1d_delta_set_segment(-1)
