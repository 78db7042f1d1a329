"""What bits the gated delta rule's gradients of q and k keep: correlated keys, slow decays, wide
values, against the adjoint in 64 bits.

Bounds.  dq and dk of a block of 64 tokens are sums of products of the state before it, the state's
gradient after it, the solution u and the gradients of o and v.  For bfloat16 data the products'
operands hold two bfloat16 terms, each operand off by at most 2^-16 of its value; a product drops
one pair of terms (2^-16), and the tokens' pairs are rounded to two terms once more: 4 * 2^-16 of
the products' magnitudes, summed.  The operands themselves are fp32 results, whose sums round by
half a step of the largest.  The results are rounded once.
"""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import delta_util as du

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]
BLOCK = 64


def magnitudes(t, scale, dstate=None):
    """The summed magnitudes of the products in dq and dk, float64, of their shapes."""
    q, k, v, g, beta = (t[n].double() for n in du.NAMES)
    B, L, H, DV = v.shape
    HK, DK = q.shape[2:]
    rep = H // HK
    mq, mk = torch.zeros(B, L, H, DK).double(), torch.zeros(B, L, H, DK).double()
    for b in range(B):
        S = t["h0"][b].double() if t["h0"] is not None else torch.zeros(H, DK, DV).double()
        _, _, states = du.rule(q[b], k[b], v[b], g[b], beta[b], scale, S)
        kb, qb = k[b].repeat_interleave(rep, 1), q[b].repeat_interleave(rep, 1)
        do = t["do"][b].double()
        u, dv = torch.zeros_like(v[b]), torch.zeros_like(v[b])
        after = {}  # the gradient of the state after a block's last token
        dS = dstate[b].double() if dstate is not None else torch.zeros(H, DK, DV).double()
        for j in range(L - 1, -1, -1):
            if j == L - 1 or (j + 1) % BLOCK == 0:
                after[j // BLOCK] = dS.abs()
            before = states[j] * g[b, j].exp()[:, None, None]
            u[j] = beta[b, j][:, None] * (v[b, j] - (kb[j][:, :, None] * before).sum(1))
            dS = dS + scale * qb[j][:, :, None] * do[j][:, None, :]
            dv[j] = beta[b, j][:, None] * (dS * kb[j][:, :, None]).sum(1)
            dS = (dS - kb[j][:, :, None] * dv[j][:, None, :]) * g[b, j].exp()[:, None, None]
        for i in range((L + BLOCK - 1) // BLOCK):
            s, e = i * BLOCK, min(L, (i + 1) * BLOCK)
            G = g[b, s:e].cumsum(0)
            later = torch.ones(e - s, e - s).triu(1).bool()[..., None]
            f = (G[:, None] - G[None]).masked_fill(later, -float("inf")).exp().permute(2, 0, 1)
            S0 = states[s].abs()
            qa, ka, ua, va, da = (x[s:e].abs().transpose(0, 1) for x in (qb, kb, u, dv, do))
            into, out = G.exp().T[..., None], (G[-1] - G).exp().T[..., None]
            P, N = f * (da @ ua.transpose(1, 2)), f * (va @ ua.transpose(1, 2))
            mq[b, s:e] = (scale * (into * (da @ S0.transpose(1, 2)) + P @ ka)).transpose(0, 1)
            mk[b, s:e] = (out * (ua @ after[i].transpose(1, 2)) + into * (va @ S0.transpose(1, 2))
                          + scale * P.transpose(1, 2) @ qa + N @ ka
                          + N.transpose(1, 2) @ ka).transpose(0, 1)
    return [m.unflatten(2, (HK, rep)).sum(3) for m in (mq, mk)]


CASES = [  # B, L, HK, H, DK, DV, how much of the first key every key holds, decay
    (1, 200, 2, 2, 64, 64, 0.0, 0.02), (1, 200, 1, 2, 64, 48, 0.9, 0.02),
    (1, 200, 1, 1, 64, 64, 1.0, 0.0), (1, 130, 1, 2, 128, 192, 0.5, 0.1),
    (2, 97, 1, 1, 32, 160, 0.9, 0.0), (1, 129, 1, 3, 100, 96, 0.7, 0.05),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("chunks", [0, 2])
@pytest.mark.parametrize("case", CASES)
def test_dq_and_dk(case, chunks, dtype):
    B, L, HK, H, DK, DV, common, decay = case
    t = du.make_inputs(B, L, HK, H, DK, DV, dtype, seed=L + DV, decay=decay, h0=B if L % 2 else 0)
    k = (1 - common) * t["k"].float() + common * t["k"][:, :1].float()
    t["k"] = (k / k.norm(dim=-1, keepdim=True)).to(dtype)
    scale = DK ** -0.5
    d = du.to_gpu(t)
    args = [d[n] for n in du.NAMES]
    with du.segments(chunks):
        _, saved = ss.ss1d_delta_forward_save(*args, initial_state=d["h0"])
        got = ss.ss1d_delta_backward(*args, d["do"], initial_state=d["h0"], saved=saved)
    ref, _ = du.adjoint(t, scale)
    low = 4 * 2.0 ** -16 if dtype == torch.bfloat16 else 0.0
    for n, m in zip("qk", magnitudes(t, scale)):
        tol = low * m + du.F32_HALF * (DK + DV + 5 * BLOCK) * m.max()
        err = (got[n].double().cpu() - ref[n]).abs()
        over = err - tol - (du.BF16_HALF * ref[n].abs() if dtype == torch.bfloat16 else 0.0)
        assert float(over.max()) <= 0, f"d{n}: over by {float(over.max()):.2e} (error {float(err.max()):.2e})"


def gate_magnitudes(t, scale):
    """The summed magnitudes of what dg of every token is the difference of: do.o and dv.v of the
    tokens from it to its block's end, and <dS, S> behind the block (float64)."""
    q, k, v, g, beta = (t[n].double() for n in du.NAMES)
    B, L, H, DV = v.shape
    rep = H // q.shape[2]
    out = torch.zeros(B, L, H).double()
    for b in range(B):
        S = t["h0"][b].double() if t["h0"] is not None else torch.zeros(H, q.shape[3], DV).double()
        o, end, states = du.rule(q[b], k[b], v[b], g[b], beta[b], scale, S)
        kb, qb = k[b].repeat_interleave(rep, 1), q[b].repeat_interleave(rep, 1)
        do = t["do"][b].double()
        dS, total = torch.zeros_like(S), torch.zeros(H).double()
        for j in range(L - 1, -1, -1):
            if j == L - 1 or (j + 1) % BLOCK == 0:
                total = (dS.abs() * (states[j + 1] if j + 1 < L else end).abs()).sum((1, 2))
            dS = dS + scale * qb[j][:, :, None] * do[j][:, None, :]
            dv = beta[b, j][:, None] * (dS * kb[j][:, :, None]).sum(1)
            dS = (dS - kb[j][:, :, None] * dv[:, None, :]) * g[b, j].exp()[:, None, None]
            total = total + (do[j].abs() * o[j].abs()).sum(1) + (dv.abs() * v[b, j].abs()).sum(1)
            out[b, j] = total
    return out


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("least, most", [(0.0, 0.2), (0.0, 10.0), (0.0, 80.0), (5.0, 20.0), (40.0, 80.0)])
def test_dg_of_decays_from_weak_to_strong(least, most, dtype):
    """dg keeps an absolute accuracy, also where strong decays leave almost nothing of it: fp32
    roundings of what it is the difference of, each the end of sums over DK, DV and a chunk."""
    t = du.make_inputs(1, 200, 1, 2, 64, 48, dtype, seed=int(most), h0=1)
    t["g"] = -(least + (most - least) * torch.rand(t["g"].shape, generator=torch.Generator().manual_seed(1)))
    d = du.to_gpu(t)
    args = [d[n] for n in du.NAMES]
    got = ss.ss1d_delta_backward(*args, d["do"], scale=0.3, initial_state=d["h0"])
    ref, _ = du.adjoint(t, 0.3)
    tol = du.F32_HALF * (64 + 48 + 5 * BLOCK) * gate_magnitudes(t, 0.3)
    over = (got["g"].double().cpu() - ref["g"]).abs() - tol
    assert float(over.max()) <= 0, f"over by {float(over.max()):.2e}"
