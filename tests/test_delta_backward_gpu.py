"""The gated delta rule's backward against the adjoint in 64 bits, and against differences."""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import delta_util as du

pytestmark = pytest.mark.gpu

SHAPES = [  # B, L, HK, H, DK, DV
    (1, 1, 1, 1, 1, 1), (2, 31, 1, 2, 32, 32), (1, 33, 2, 2, 16, 40), (2, 64, 1, 3, 64, 31),
    (1, 65, 2, 4, 128, 96), (2, 100, 3, 3, 64, 64), (1, 130, 1, 2, 80, 100),
    (1, 197, 1, 1, 127, 33), (1, 290, 1, 2, 128, 128),
]
TYPES = [torch.float32, torch.bfloat16]


def check_grads(t, d, dtype, scale, cu=None, dstate=None):
    """Each gradient sums, per token, products of states and gradients over DK or DV and 64
    tokens, of terms no larger than M = (largest |v|, h0) x (largest |do|, dstate) x
    |key| = 1 times the sums' length in quadrature; fp32 rounds each addition by half a step.
    In bfloat16 each product of dq and dk carries one operand rounding (half a step), dk has
    six products, and the results are rounded once."""
    ref, ref0 = du.adjoint(t, scale, cu, dstate)
    DK, DV = t["q"].shape[3], t["v"].shape[3]
    L = t["v"].shape[1]
    for n in du.NAMES:
        big = float(ref[n].abs().max())
        tol = du.F32_HALF * (DK + DV + 5 * 64) * max(big, 1e-6)
        rel = 0.0
        if n == "g":  # sums of up to 64 terms do.o - dv.v that cancel, and <dS, S>
            terms = float((t["do"].double().abs().max() * t["v"].double().abs().max()))
            tol += du.F32_HALF * 64 * max(terms, big)
        if dtype == torch.bfloat16 and n in "qkv":
            rel = du.BF16_HALF
            if n != "v":  # 6 products of root-mean-square 2^-8 / sqrt(3) of their terms, x 5
                tol += 5 * 6 ** 0.5 * du.BF16_HALF / 3 ** 0.5 * float(ref[n].square().mean().sqrt())
        du.check(d[n], ref[n], "d" + n, tol, rel)
    if "initial_state" in d:
        du.check(d["initial_state"], ref0, "dh0",
                 du.F32_HALF * (DV + 5 * 32) * max(float(ref0.abs().max()), 1e-6))
    assert L


def run(t, scale, keep, **kw):
    d = du.to_gpu(t)
    args = [d[n] for n in du.NAMES]
    saved = None
    if keep:
        o, saved = ss.ss1d_delta_forward_save(*args, scale=scale, initial_state=d["h0"],
                                              cu_seqlens=kw.get("cu_seqlens"))
    return ss.ss1d_delta_backward(*args, d["do"], scale=scale, initial_state=d["h0"], saved=saved,
                                  **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, dtype):
    B, L, HK, H, DK, DV = shape
    t = du.make_inputs(*shape, dtype, seed=L, h0=B if L % 2 else 0)
    scale = DK ** -0.5
    dstate = 0.1 * torch.randn(B, H, DK, DV, generator=torch.Generator().manual_seed(1)) \
        if L % 3 else None
    gs = dstate.cuda() if dstate is not None else None
    d = run(t, scale, True, dstate=gs)
    check_grads(t, d, dtype, scale, dstate=dstate)
    again = run(t, scale, False, dstate=gs)  # computing the kept state again: the same bits
    for n in d:
        assert torch.equal(d[n], again[n]), n


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("decay", [0.0, 1.0])
def test_decays(dtype, decay):
    t = du.make_inputs(1, 150, 2, 2, 64, 48, dtype, seed=5, decay=decay, h0=1)
    check_grads(t, run(t, 0.3, True), dtype, 0.3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 8, 8), (2, 130, 1, 2, 64, 48), (1, 257, 2, 2, 127, 33),
                                   (1, 320, 1, 2, 128, 64), (1, 129, 1, 1, 30, 100)])
def test_segments(shape, dtype):
    """Sequences cut into segments of 2 chunks, kept and recomputed."""
    B, L, HK, H, DK, DV = shape
    t = du.make_inputs(*shape, dtype, seed=L, h0=B if L % 2 else 0)
    dstate = 0.1 * torch.randn(B, H, DK, DV, generator=torch.Generator().manual_seed(1))
    with du.segments(2):
        d = run(t, DK ** -0.5, True, dstate=dstate.cuda())
        again = run(t, DK ** -0.5, False, dstate=dstate.cuda())
    check_grads(t, d, dtype, DK ** -0.5, dstate=dstate)
    for n in d:
        assert torch.equal(d[n], again[n]), n


@pytest.mark.parametrize("dtype", TYPES)
def test_segments_of_packed_sequences(dtype):
    lens = [0, 1, 31, 200, 0, 65, 128]
    cu = torch.tensor([3] + [0] * len(lens), dtype=torch.int32)
    for i, n in enumerate(lens):
        cu[i + 1] = cu[i] + n
    t = du.make_inputs(1, int(cu[-1]) + 5, 1, 2, 64, 48, dtype, seed=8, h0=len(lens))
    with du.segments(2):
        d = run(t, 0.5, True, cu_seqlens=cu.cuda())
    check_grads(t, d, dtype, 0.5, cu)


def test_training_forward_is_the_forward():
    """o of the training forward differs from the forward's by its operands' terms only."""
    t = du.make_inputs(2, 100, 1, 2, 64, 64, torch.float32, seed=6)
    d = du.to_gpu(t)
    args = [d[n] for n in du.NAMES]
    o, ht, saved = ss.ss1d_delta_forward_save(*args, final_state=True)
    p, pht = ss.ss1d_delta_forward(*args, final_state=True)
    assert torch.equal(o, p) and torch.equal(ht, pht) and saved.dtype == torch.uint8


@pytest.mark.parametrize("dtype", TYPES)
def test_packed(dtype):
    lens = [0, 1, 31, 64, 0, 33, 65, 100]
    cu = torch.tensor([3] + [0] * len(lens), dtype=torch.int32)
    for i, n in enumerate(lens):
        cu[i + 1] = cu[i] + n
    L = int(cu[-1]) + 5
    t = du.make_inputs(1, L, 1, 2, 64, 48, dtype, seed=8, h0=len(lens))
    d = run(t, 0.5, True, cu_seqlens=cu.cuda())
    for n in du.NAMES:
        assert (d[n][0, :3] == 0).all() and (d[n][0, L - 5:] == 0).all()
    assert (d["initial_state"][0] == 0).all()
    check_grads(t, d, dtype, 0.5, cu)


def test_forgotten_tokens_and_zero_beta():
    t = du.make_inputs(1, 100, 1, 2, 64, 64, torch.float32, seed=9, h0=1)
    t["g"][0, 40, 0] = -float("inf")
    t["beta"][0, 10:20, 1] = 0.0
    d = run(t, 1.0, True)
    assert d["g"][0, 40, 0] == 0
    check_grads(t, d, torch.float32, 1.0)


def test_against_differences():
    """Directional derivatives of the forward itself, central differences: error of the
    difference h^2 / 6 times the third derivative plus 2 half steps of the sum over h."""
    t = du.make_inputs(1, 70, 1, 2, 32, 32, torch.float32, seed=10, h0=1)
    t["do"] = torch.randn_like(t["do"])
    d = run(t, 1.0, True)
    gen = torch.Generator().manual_seed(2)
    for n in du.NAMES + ("h0",):
        step = torch.randn(t[n].shape, generator=gen)
        step /= step.norm()
        h = 2e-2 if n != "g" else 1e-2
        val = []
        for sign in (1, -1):
            m = dict(t)
            m[n] = t[n] + sign * h * step
            g = du.to_gpu(m)
            o = ss.ss1d_delta_forward(*[g[x] for x in du.NAMES], scale=1.0, initial_state=g["h0"])
            val.append((o.double().cpu() * t["do"].double()).sum())
        want = float((val[0] - val[1]) / (2 * h))
        got = float((d["initial_state" if n == "h0" else n].double().cpu() * step.double()).sum())
        norm = float(d["initial_state" if n == "h0" else n].double().norm())
        # along a random unit direction a gradient of norm G has derivative ~ G / sqrt(size)
        assert abs(got - want) <= 1e-3 * norm / step.numel() ** 0.5 + 5e-3 * abs(want), n


def test_shared_and_strided_inputs():
    """Key heads shared by three value heads, inputs as views of one projection."""
    t = du.make_inputs(2, 70, 1, 3, 64, 64, torch.bfloat16, seed=11)
    d = du.to_gpu(t)
    whole = run(t, 0.2, True)
    fused = torch.zeros(2, 70, 64 * 5 + 3, dtype=torch.bfloat16, device="cuda")
    parts, at = [], 1
    for n in ("q", "k", "v"):
        w = d[n].shape[2] * 64
        fused[:, :, at:at + w] = d[n].reshape(2, 70, w)
        parts.append(fused[:, :, at:at + w].unflatten(2, (-1, 64)))
        at += w
    got = ss.ss1d_delta_backward(*parts, d["g"], d["beta"], d["do"], scale=0.2)
    for n in whole:
        assert torch.equal(got[n], whole[n]), n


def test_graph_of_a_training_step():
    t = du.to_gpu(du.make_inputs(2, 90, 1, 2, 64, 64, torch.bfloat16, seed=13))
    args = [t[n] for n in du.NAMES]

    def work():
        o, saved = ss.ss1d_delta_forward_save(*args)
        return o, ss.ss1d_delta_backward(*args, t["do"], saved=saved)

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = work()
    for i in range(3):
        t["v"].copy_(torch.randn_like(t["v"]))
        t["do"].copy_(torch.randn_like(t["do"]))
        graph.replay()
        torch.cuda.synchronize()
        got = [out[0].clone()] + [out[1][n].clone() for n in du.NAMES]
        o, d = work()
        for x, y in zip(got, [o] + [d[n] for n in du.NAMES]):
            assert torch.equal(x, y), i
        torch.cuda.synchronize()
