"""How far the scan, the convolution and the group norm are from 64 bits as a whole: the norm of the
error against the norm of the result.

A value of fp32 is rounded some tens of times on its way; half steps of 2^-24 that add in quadrature
over the 100 or so tokens that a state remembers stay below 128 of them.  bfloat16 data add one
rounding of an output, uniform in a step, whose mean square is (2 * 2^-8)^2 / 12 of the value at most."""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import scan_util as su
from tests.test_scan_gpu import args, gpu

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def bound(dtype):
    return 128 * 2.0 ** -24 + (2 * 2.0 ** -8 / 12 ** 0.5 if dtype == BF16 else 0.0)


def check(got, ref, what, dtype=F32):
    err = float((got.double().cpu() - ref).norm() / ref.norm())
    assert err <= bound(dtype), f"{what}: {err:.2e}"


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B, L, D, G, N, seg", [(2, 300, 100, 1, 16, 0), (1, 300, 100, 2, 16, 64), (1, 200, 40, 1, 32, 40),
                                                (2, 150, 70, 1, 8, 32)])
def test_scan(B, L, D, G, N, seg, dtype):
    t = su.make_inputs(B, L, D, G, N, dtype, seed=1, h0=B)
    y64, h64, _ = su.reference(t)
    g64, _ = su.adjoint(t)
    d = gpu(t)
    kw = dict(z=d["z"], initial_state=d["h0"])
    with su.plan(seg):
        y, h, saved = ss.ss1d_scan_forward_save(*args(d), final_state=True, **kw)
        g = ss.ss1d_scan_backward(*args(d), d["dy"], dstate=d["dht"], saved=saved, **kw)
    check(y, y64, "y", dtype)
    check(h, h64, "h")
    for n in su.NAMES + ("z",):
        check(g[n], g64[n], "d" + n, d[n].dtype)
    check(g["initial_state"], g64["h0"], "dh0")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_conv(dtype):
    t = su.conv_inputs(2, 300, 136, 4, dtype, seed=1, h0=2)
    y64, _ = su.conv_reference(t)
    g64 = su.conv_reference(t, grads=True)
    x, w, b, h0, dy, dht = (t[n].cuda() for n in ("x", "conv_w", "conv_b", "h0", "dy", "dht"))
    check(ss.ss1d_conv_forward(x, w, b, initial_state=h0), y64, "y", dtype)
    g = ss.ss1d_conv_backward(x, w, dy, b, initial_state=h0, dstate=dht)
    for n, m in (("x", "x"), ("conv_w", "conv_w"), ("conv_b", "conv_b"), ("h0", "initial_state")):
        check(g[m], g64[n], "d" + n, g[m].dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape, G", [((2, 30, 30, 96), 16), ((1, 9000, 64), 2)])
def test_group_norm(shape, G, dtype):
    from tests.test_group_norm_gpu import make, reference
    x, dy, w, b = make(shape, dtype, True, seed=2)
    y64, _, g64 = reference(x, dy, G, w, b, True, 1e-5)
    kw = dict(weight=w.cuda(), bias=b.cuda())
    check(ss.ss2d_group_norm_forward(x.cuda(), G, **kw), y64, "y", dtype)
    d = ss.ss2d_group_norm_backward(x.cuda(), dy.cuda(), G, **kw)
    for n, ref in zip(("x", "weight", "bias"), g64):
        check(d[n], ref, "d" + n, d[n].dtype)
