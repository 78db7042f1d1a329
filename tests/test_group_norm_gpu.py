"""The group norm on the GPU against its definition in 64 bits, both directions."""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from selective_scan_ss2d_amd import _binding as bnd
from tests import scan_util as su

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# shape (B, ..., C), groups, type, SiLU, weight and bias
CASES = [
    ((1, 1, 1), 1, F32, False, True), ((2, 1, 8), 8, BF16, True, True), ((2, 3, 5, 6), 3, F32, True, True),
    ((1, 16, 16, 32), 4, BF16, True, True), ((3, 7, 40), 5, BF16, True, False), ((2, 9, 9, 33), 3, F32, True, True),
    ((2, 14, 14, 192), 32, BF16, True, True), ((2, 28, 28, 48), 8, F32, True, True),
    ((1, 56, 56, 96), 16, BF16, True, True), ((2, 300, 7), 1, BF16, False, True),
    ((1, 5000, 16), 2, F32, True, True), ((1, 20000, 8), 1, BF16, True, True), ((1, 2100, 63), 1, F32, True, True),
    ((2, 33, 1032), 3, BF16, True, True), ((70, 4, 64), 2, F32, True, True), ((1, 4, 4, 9000), 1, F32, True, True),
    ((1, 8500, 264), 33, BF16, True, True),
    # by chunks: rows of 8 and 16 threads, of single values, and joins of 64 to 1024 threads
    ((2, 90000, 24), 3, BF16, True, True), ((1, 60000, 72), 1, F32, True, True), ((3, 9000, 5), 1, BF16, True, True),
    ((1, 66000, 64), 8, BF16, True, True), ((5, 5000, 33), 1, F32, False, True),
]


def make(shape, dtype, affine, seed=0, mean=0.5):
    gen = torch.Generator().manual_seed(seed)
    C = shape[-1]
    x = (1.5 * torch.randn(shape, generator=gen) + mean * torch.randn(C, generator=gen)).to(dtype)
    dy = torch.randn(shape, generator=gen).to(dtype)
    w = 1 + 0.2 * torch.randn(C, generator=gen) if affine else None
    b = 0.2 * torch.randn(C, generator=gen) if affine else None
    return x, dy, w, b


def reference(x, dy, G, w, b, silu, eps):
    """y, mean and 1 / sqrt(var + eps), and the gradients, in float64."""
    x64 = x.double().requires_grad_()
    wb = [v.double().requires_grad_() for v in (w, b) if v is not None]
    B, C = x.shape[0], x.shape[-1]
    v = x64.reshape(B, -1, G, C // G)
    mean = v.mean((1, 3), keepdim=True)
    r = ((v - mean).square().mean((1, 3), keepdim=True) + eps).rsqrt()
    n = ((v - mean) * r).reshape(x.shape)
    if wb:
        n = n * wb[0] + wb[1]
    y = n * torch.sigmoid(n) if silu else n
    g = torch.autograd.grad(y, [x64] + wb, dy.double())
    return y.detach(), torch.stack([mean, r], -1).reshape(B, G, 2).detach(), g


def summed(n):
    """Roundings of a sum of n values over a block: a thread's up to 16 or so at a time, then trees,
    at most 64 + n / 256 in a row."""
    return 64 + n / 256


@pytest.mark.parametrize("mean", [0.5, 30.0])
@pytest.mark.parametrize("case", CASES)
def test_both_directions(case, mean):
    shape, G, dtype, silu, affine = case
    eps = 1e-5
    x, dy, w, b = make(shape, dtype, affine, seed=len(shape) + shape[-1], mean=mean)
    y64, stats64, g64 = reference(x, dy, G, w, b, silu, eps)
    xc, dc, wc, bc = (v.cuda() if v is not None else None for v in (x, dy, w, b))
    kw = dict(weight=wc, bias=bc, silu=silu, eps=eps)
    y, stats = ss.ss2d_group_norm_forward(xc, G, stats=True, **kw)
    assert torch.equal(y, ss.ss2d_group_norm_forward(xc, G, **kw))
    half, rel = su.F32_HALF, su.half(dtype)
    count = x.numel() // shape[0] // G
    rm, xm = su.top(stats64[..., 1]), su.top(x.double())
    n64 = (x.double().reshape(shape[0], -1, G, shape[-1] // G) - stats64[:, None, :, None, 0]) * stats64[:, None, :, None, 1]
    um = su.top(n64)
    # the mean: a sum of values up to xm; r: half the relative error of the sum of squares, which the
    # mean's error changes by its square only
    emean = half * (summed(count) + 4) * xm
    er = 0.5 * half * (summed(count) + 8) + (emean * rm) ** 2
    su.check(stats[..., 0], stats64[..., 0], "mean", emean)
    su.check(stats[..., 1], stats64[..., 1], "r", er * rm)
    wm = su.top(w) if affine else 1.0
    eunit = emean * rm + half * xm * rm + (er + 4 * half) * um  # of a unit value
    su.check(y, y64, "y", 1.1 * wm * eunit + 8 * half * (wm * um + 1), rel)
    for given in (stats, None):
        d = ss.ss2d_group_norm_backward(xc, dc, G, stats=given, **kw)
        # d = dy act': off by the unit value's error times act''s slope (at most 0.5) and 12 half steps
        gm = su.top(dy.double())
        e = 1.1 * gm * ((0.5 * wm * eunit if silu else 0.0) + 12 * half)
        total = x.numel() // shape[-1]
        if affine:
            s = total * (e + half * summed(total) * 1.1 * gm)
            su.check(d["bias"], g64[2], "db", s)
            su.check(d["weight"], g64[1], "dw", um * s + total * 1.1 * gm * eunit)
        # the means of e and e n round as sums do, and carry e's and the unit values' errors
        es = wm * (e + half * (summed(count) + 4) * 1.1 * gm)
        ex = wm * e + es + um * (um * es + wm * 1.1 * gm * eunit) + eunit * wm * 1.1 * gm * um
        ex = rm * (ex + (er + 6 * half) * wm * 1.1 * gm * (2 + um * um))
        su.check(d["x"], g64[0], "dx", ex, rel)


def test_far_mean():
    """A mean of 1000 deviations: the squares are summed about the mean."""
    gen = torch.Generator().manual_seed(1)
    x = 1000 + torch.randn(2, 4000, 16, generator=gen)
    y64, stats64, _ = reference(x, torch.ones_like(x), 2, None, None, False, 1e-5)
    y, stats = ss.ss2d_group_norm_forward(x.cuda(), 2, silu=False, stats=True)
    # unit values: the mean's rounding of 1000 (a sum of 32000 values) over a deviation of 1
    e = su.F32_HALF * (summed(32000) + 4) * 1005
    su.check(y, y64, "y", e + 8 * e * e + 32 * su.F32_HALF * su.top(y64))


def test_unaligned():
    """Rows that start off 16 bytes take the path of single values."""
    x, dy, w, b = make((2, 50, 64), BF16, True)
    flat = torch.zeros(x.numel() + 1, dtype=BF16, device="cuda")
    off = flat[1:].view(x.shape)
    off.copy_(x)
    kw = dict(weight=w.cuda(), bias=b.cuda())
    y = ss.ss2d_group_norm_forward(off, 8, **kw)
    y64, _, g64 = reference(x, dy, 8, w, b, True, 1e-5)
    e = 64 * su.F32_HALF * 10
    su.check(y, y64, "y", e, su.BF16_HALF)
    d = ss.ss2d_group_norm_backward(off, dy.cuda(), 8, **kw)
    su.check(d["x"], g64[0], "dx", 8 * e, su.BF16_HALF)


def test_constant_groups():
    """No variance: r is 1 / sqrt(eps) and y the bias."""
    x = torch.full((2, 30, 16), 3.0, device="cuda")
    b = torch.arange(16.0, device="cuda")
    y, stats = ss.ss2d_group_norm_forward(x, 4, bias=b, silu=False, stats=True)
    assert torch.equal(y, b.expand_as(y)) and torch.allclose(stats[..., 1], torch.tensor(1e-5).rsqrt().cuda())


def test_nan_stays_in_its_group():
    x, *_ = make((2, 60, 32), F32, False)
    x = x.cuda()
    clean = ss.ss2d_group_norm_forward(x, 4)
    x[1, 7, 9] = float("nan")
    y = ss.ss2d_group_norm_forward(x, 4)
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[1, :, 8:16] = True
    assert y[hit].isnan().all() and torch.equal(y[~hit], clean[~hit])


@pytest.mark.parametrize("shape", [(0, 5, 8), (2, 0, 8)])
def test_nothing_to_do(shape):
    x = torch.zeros(shape, device="cuda")
    w = torch.ones(8, device="cuda")
    assert ss.ss2d_group_norm_forward(x, 2, weight=w, bias=w).shape == shape
    d = ss.ss2d_group_norm_backward(x, x, 2, weight=w, bias=w)
    assert d["x"].shape == shape and not d["weight"].any() and not d["bias"].any()


def test_refusals():
    x = torch.zeros(2, 4, 8, device="cuda")
    with pytest.raises(ValueError, match="divisor"):
        ss.ss2d_group_norm_forward(x, 3)
    with pytest.raises(ValueError, match="contiguous"):
        ss.ss2d_group_norm_forward(x.transpose(1, 2), 2)
    with pytest.raises(TypeError):
        ss.ss2d_group_norm_forward(x.half(), 2)
    with pytest.raises(ValueError):
        ss.ss2d_group_norm_forward(x, 2, weight=torch.ones(7, device="cuda"))
    with pytest.raises(bnd.SS2DError):
        ss.ss2d_group_norm_forward(x, 2, eps=-1.0)
    with pytest.raises(bnd.SS2DError):
        ss.ss2d_group_norm_forward(x, 2, y=x)
