"""The block norm's forward and backward against the definition in 64 bits.

Bounds.  A result is a chain of at most 64 fp32 roundings (a sum over D as 8 values per thread
and a tree of at most 10 levels, twice for the layer norm's two passes, the reciprocal root,
the gate's exponential, whose argument's rounding counts up to |z| log2 e ~ 8 half steps, and
the products), each off by at most half a step of the largest value it works on in its row;
bfloat16 results are rounded once more, by half a step of their own value.
"""
import pytest
import torch

import selective_scan_ss2d_amd as ss

pytestmark = pytest.mark.gpu
HALF = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
CHAIN = 64 * 2.0 ** -24

FULL = dict(post=True, gate=True, residual=True, groups=1, pre=True)
PARTS = [FULL, dict(FULL, gate=False, groups=0), dict(FULL, pre=False),
         dict(FULL, residual=False, pre=False, groups=0), dict(FULL, post=False, pre=False),
         dict(FULL, post=False, gate=False), dict(FULL, residual=False, gate=False, groups=2),
         dict(post=False, gate=False, residual=False, groups=0, pre=True)]
TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16),
         (torch.bfloat16, torch.float32)]


def make(R, D, L, parts, dtype, ytype, layer, seed, grad=False):
    """Inputs on the CPU; rows (R, D), or (R / L, D, L) for channels first."""
    gen = torch.Generator().manual_seed(seed)
    shape = (R // L, D, L) if L else (R, D)

    def normal(*s, std=1.0, dtype=torch.float32):
        return (std * torch.randn(s, generator=gen)).to(dtype)

    t = dict(h=normal(*shape, std=1.5, dtype=dtype), z=None, residual=None, res_scale=None,
             w_post=None, b_post=None, w_pre=None, b_pre=None)
    if not parts["residual"]:
        ytype = dtype
    if parts["post"]:
        t["w_post"], t["b_post"] = normal(D) + 1, normal(D) if layer else None
    if parts["gate"]:
        t["z"] = normal(*shape, dtype=dtype)
    if parts["residual"]:
        t["residual"] = normal(*shape, std=3.0, dtype=ytype)
    if parts["groups"]:
        t["res_scale"] = normal(parts["groups"], D)
    if parts["pre"]:
        t["w_pre"], t["b_pre"] = normal(D) + 1, normal(D) if layer else None
    if grad:
        t["y"], t["dy"] = normal(*shape, std=3.0, dtype=ytype), normal(*shape, dtype=ytype)
        t["dn"] = normal(*shape, dtype=dtype) if parts["pre"] else None
    return t


def gpu(t):
    return {n: x.cuda() if x is not None else None for n, x in t.items()}


def last(x, L):
    return None if x is None else (x.double().transpose(1, 2).reshape(-1, x.shape[1]) if L
                                   else x.double())


def unit(x, layer, eps):
    if layer:
        x = x - x.mean(1, keepdim=True)
    return x / (x.square().mean(1, keepdim=True) + eps).sqrt()


def definition(t, L, layer, eps):
    """y, n and the largest magnitude of each row's terms, rows of D, float64."""
    p = last(t["h"], L)
    R, D = p.shape
    if t["w_post"] is not None:
        p = unit(p, layer, eps) * t["w_post"].double()
        p = p if t["b_post"] is None else p + t["b_post"].double()
    if t["z"] is not None:
        z = last(t["z"], L)
        p = p * z * torch.sigmoid(z)
    if t["res_scale"] is not None:
        G = t["res_scale"].shape[0]
        p = (p.reshape(G, -1, D) * t["res_scale"].double()[:, None]).reshape(R, D)
    y = p + last(t["residual"], L) if t["residual"] is not None else p
    n = None
    if t["w_pre"] is not None:
        n = unit(y, layer, eps) * t["w_pre"].double()
        n = n if t["b_pre"] is None else n + t["b_pre"].double()
    big = p.abs().amax(1, keepdim=True)
    if t["residual"] is not None:
        big = big + last(t["residual"], L).abs().amax(1, keepdim=True)
    return y, n, big


def check(got, ref, what, tol, L=0):
    x = last(got.cpu(), L)
    assert torch.isfinite(x).all(), what
    err = (x - ref).abs() - HALF[got.dtype] * ref.abs() - tol
    assert float(err.max()) <= 0, f"{what}: {float((x - ref).abs().max()):.3e}, over by {float(err.max()):.3e}"


def forward(d, L, **kw):
    return ss.ss2d_norm_forward(d["h"], channels_first=L > 0,
                                **{k: d[k] for k in ("residual", "z", "res_scale", "w_post",
                                                     "b_post", "w_pre", "b_pre")}, **kw)


def check_forward(t, L, y, n, layer, eps):
    ry, rn, big = definition(t, L, layer, eps)
    check(y, ry, "y", CHAIN * big, L)
    if rn is not None:
        # the second norm divides by the root mean square of (centred) y: errors of y as large
        # as CHAIN * big reach n times the weight over that root
        c = ry - ry.mean(1, keepdim=True) if layer else ry
        r = 1 / (c.square().mean(1, keepdim=True) + eps).sqrt()
        w = t["w_pre"].double().abs()
        b = 0 if t["b_pre"] is None else t["b_pre"].double().abs()
        check(n, rn, "n", CHAIN * (2 * big * r * w + b), L)


LAST = [(1, 1), (3, 5), (70, 64), (9, 100), (33, 192), (5, 768), (3, 1000), (2, 2048), (3, 4100),
        (2, 8192), (40, 24)]
FIRST = [(2, 1, 3), (2, 33, 5), (4, 64, 64), (2, 96, 49), (2, 192, 196), (2, 250, 130), (2, 400, 36),
         (2, 1000, 20), (2, 512, 7), (1, 768, 16)]


@pytest.mark.parametrize("dtype, ytype", TYPES)
@pytest.mark.parametrize("R, D", LAST)
@pytest.mark.parametrize("layer", [False, True])
def test_forward(R, D, layer, dtype, ytype):
    t = make(R, D, 0, FULL, dtype, ytype, layer, seed=R + D)
    y, n = forward(gpu(t), 0, layer=layer, eps=1e-5)
    assert y.dtype == ytype and n.dtype == dtype
    check_forward(t, 0, y, n, layer, 1e-5)


@pytest.mark.parametrize("dtype, ytype", TYPES)
@pytest.mark.parametrize("B, D, L", FIRST)
@pytest.mark.parametrize("layer", [False, True])
def test_forward_channels_first(B, D, L, layer, dtype, ytype):
    t = make(B * L, D, L, FULL, dtype, ytype, layer, seed=B + D)
    y, n = forward(gpu(t), L, layer=layer, eps=1e-5)
    check_forward(t, L, y, n, layer, 1e-5)


@pytest.mark.parametrize("dtype, ytype", TYPES)
@pytest.mark.parametrize("parts", range(len(PARTS)))
@pytest.mark.parametrize("L", [0, 21])
def test_parts(parts, L, dtype, ytype):
    t = make(42, 96, L, PARTS[parts], dtype, ytype, True, seed=parts)
    y, n = forward(gpu(t), L, layer=True)
    check_forward(t, L, y, n, True, 1e-6)
    assert (n is None) == (not PARTS[parts]["pre"])


def rows_bound(x):
    return x.abs().amax(1, keepdim=True)


def check_backward(t, L, d, layer, eps):
    """Autograd of the definition in float64, with bounds from the same terms."""
    keys = [k for k in ("h", "z", "residual", "res_scale", "w_post", "b_post") if t[k] is not None]
    leaf = {k: t[k].double().requires_grad_() if t[k] is not None else None for k in t}
    total = last(t["dy"], L) if t["dy"] is not None else 0
    amp = rows_bound(total) if t["dy"] is not None else 0
    if t["w_pre"] is not None:
        stored = last(t["y"], L).requires_grad_()
        u = unit(stored, layer, eps)
        n = u * leaf["w_pre"]
        n = n if t["b_pre"] is None else n + leaf["b_pre"]
        dn = last(t["dn"], L)
        names = ["w_pre"] + (["b_pre"] if t["b_pre"] is not None else [])
        got = torch.autograd.grad(n, [stored] + [leaf[k] for k in names], dn)
        total = total + got[0]
        c = stored - stored.mean(1, keepdim=True) if layer else stored
        r = 1 / (c.square().mean(1, keepdim=True) + eps).sqrt()
        amp = amp + (2 * r * rows_bound(dn * t["w_pre"].double()) * (1 + rows_bound(u))).detach()
        check(d["w_pre"][None], got[1][None], "dw_pre", 2 * CHAIN * (dn * u).abs().sum(0).detach())
        if t["b_pre"] is not None:
            check(d["b_pre"][None], got[2][None], "db_pre", 2 * CHAIN * dn.abs().sum(0))
    if t["residual"] is not None:
        check(d["residual"], total.detach(), "dresidual", CHAIN * amp, L)
    y, _, _ = definition({**leaf, "w_pre": None}, L, layer, eps)
    if not y.requires_grad:
        y = y + 0 * leaf["h"].sum()
    got = torch.autograd.grad(y, [leaf[k] for k in keys], total.detach())
    h = last(t["h"], L)
    u = unit(h, layer, eps) if t["w_post"] is not None else h
    w = t["w_post"].double() if t["w_post"] is not None else torch.ones(h.shape[1]).double()
    p = (u * w if t["w_post"] is not None else u)
    p = p if t["b_post"] is None else p + t["b_post"].double()
    s = torch.ones_like(h)
    if t["res_scale"] is not None:
        G = t["res_scale"].shape[0]
        s = t["res_scale"].double().repeat_interleave(h.shape[0] // G, 0)
    z = last(t["z"], L) if t["z"] is not None else None
    gate = z * torch.sigmoid(z) if z is not None else torch.ones_like(h)
    D, R = h.shape[1], h.shape[0]
    for k, ref in zip(keys, got):
        if k == "residual":
            continue
        if k == "z":
            check(d["z"], last(ref, L), "dz", 2 * CHAIN * amp * rows_bound(s * p) * 1.2, L)
        elif k == "h":
            if t["w_post"] is None:
                tol = CHAIN * amp * rows_bound(s * gate)
            else:
                c = h - h.mean(1, keepdim=True) if layer else h
                r = 1 / (c.square().mean(1, keepdim=True) + eps).sqrt()
                tol = 4 * CHAIN * r * amp * rows_bound(s * gate * w) * (1 + rows_bound(u))
            check(d["h"], last(ref, L), "dh", tol, L)
        else:  # sums over rows: of the terms' magnitudes
            term = {"res_scale": p * gate, "w_post": s * gate * u, "b_post": s * gate}[k].abs()
            tol = 2 * CHAIN * (amp + 0 * term) * term
            if k == "res_scale":
                tol = tol.reshape(t[k].shape[0], -1, D).sum(1)
                check(d[k], ref, "d" + k, tol)
            else:
                check(d[k][None], ref[None], "d" + k, tol.sum(0))
    assert R


def backward(d, L, parts, **kw):
    return ss.ss2d_norm_backward(d["h"], d["y"] if d["dn"] is not None else None, d["dy"], d["dn"],
                                 residual=parts["residual"], channels_first=L > 0,
                                 **{k: d[k] for k in ("z", "res_scale", "w_post", "b_post",
                                                      "w_pre", "b_pre")}, **kw)


@pytest.mark.parametrize("dtype, ytype", TYPES)
@pytest.mark.parametrize("R, D", LAST)
@pytest.mark.parametrize("layer", [False, True])
def test_backward(R, D, layer, dtype, ytype):
    t = make(R, D, 0, FULL, dtype, ytype, layer, seed=R + D, grad=True)
    check_backward(t, 0, backward(gpu(t), 0, FULL, layer=layer, eps=1e-5), layer, 1e-5)


@pytest.mark.parametrize("dtype, ytype", TYPES)
@pytest.mark.parametrize("B, D, L", FIRST)
@pytest.mark.parametrize("layer", [False, True])
def test_backward_channels_first(B, D, L, layer, dtype, ytype):
    t = make(B * L, D, L, FULL, dtype, ytype, layer, seed=B + D, grad=True)
    check_backward(t, L, backward(gpu(t), L, FULL, layer=layer, eps=1e-5), layer, 1e-5)


@pytest.mark.parametrize("dtype, ytype", TYPES)
@pytest.mark.parametrize("parts", range(len(PARTS)))
@pytest.mark.parametrize("L", [0, 21])
def test_backward_parts(parts, L, dtype, ytype):
    t = make(42, 96, L, PARTS[parts], dtype, ytype, True, seed=parts, grad=True)
    check_backward(t, L, backward(gpu(t), L, PARTS[parts], layer=True), True, 1e-6)


@pytest.mark.parametrize("L", [0, 50])
@pytest.mark.parametrize("groups", [1, 3, 12, 1500])
def test_many_rows_and_groups(L, groups):
    """Sums over blocks, over several groups per block and several blocks per group."""
    B = 1500 if groups == 1500 else 12
    R = B * 50
    parts = dict(FULL, groups=groups)
    t = make(R, 64, L, parts, torch.float32, torch.float32, True, seed=groups, grad=True)
    d = backward(gpu(t), L, parts, layer=True)
    check_backward(t, L, d, True, 1e-6)
    again = backward(gpu(t), L, parts, layer=True)
    for k in d:
        assert torch.equal(d[k], again[k]), k


def test_against_differences():
    t = make(6, 40, 0, FULL, torch.float32, torch.float32, True, seed=3, grad=True)
    y0, _ = forward(gpu(t), 0, layer=True)
    t["y"] = y0.cpu()
    d = backward(gpu(t), 0, FULL, layer=True)
    gen = torch.Generator().manual_seed(4)
    for k in ("h", "z", "residual", "res_scale", "w_post", "b_post", "w_pre", "b_pre"):
        step = torch.randn(t[k].shape, generator=gen)
        step /= step.norm()
        val = []
        for sign in (1, -1):
            m = dict(t)
            m[k] = t[k] + sign * 1e-2 * step
            y, n = forward(gpu(m), 0, layer=True)
            val.append((y.double().cpu() * t["dy"]).sum() + (n.double().cpu() * t["dn"]).sum())
        want = float(val[0] - val[1]) / 2e-2
        got = float((d[k].double().cpu() * step).sum())
        # third derivatives times 1e-4 / 6, and the outputs' roundings over the step
        assert abs(got - want) <= 2e-3 * max(abs(want), float(d[k].norm()) / step.numel() ** 0.5), k


def test_constant_rows_and_far_means():
    """Rows without spread, and a mean far above it: the centred sum of squares keeps it."""
    h = torch.full((4, 96), 3.0)
    h[1] = 0
    h[2] = 1000 + torch.randn(96, generator=torch.Generator().manual_seed(1))
    h[3] = 1e18
    w = torch.ones(96)
    y, _ = ss.ss2d_norm_forward(h.cuda(), w_post=w.cuda(), layer=True, eps=1e-6)
    ref = unit(h.double()[2:3], True, 1e-6)
    assert torch.isfinite(y).all()
    # 1000 has steps of 2^-14: the mean and differences round to half a step of 1000
    assert float((y[2].cpu().double() - ref).abs().max()) <= 3 * 1000 * 2.0 ** -24 / 1 + 1e-5
    y, n = ss.ss2d_norm_forward(h[:2].cuda(), w_pre=w.cuda(), eps=1e-6)
    assert y.shape == (2, 96) and (n[1] == 0).all()
    assert float((n[0].cpu().double() - 1).abs().max()) <= 1e-6


def test_in_place_and_given_outputs():
    t = make(33, 192, 0, FULL, torch.bfloat16, torch.float32, False, seed=5)
    d = gpu(t)
    y, n = forward(d, 0)
    given = torch.empty_like(n)
    back, m = forward(d, 0, y=d["residual"], n=given)
    assert back is d["residual"] and m is given
    assert torch.equal(back, y) and torch.equal(m, n)


@pytest.mark.parametrize("L", [0, 30])
def test_misaligned_rows(L):
    """Tensors that start off a 16-byte edge take the element-wise path: the same values."""
    t = make(60, 64, L, FULL, torch.bfloat16, torch.bfloat16, True, seed=6, grad=True)
    d = gpu(t)
    y, n = forward(d, L, layer=True)
    g = backward(d, L, FULL, layer=True)
    m = dict(d)
    for k in ("h", "z", "residual", "y", "dy", "dn"):
        b = torch.empty(d[k].numel() + 1, dtype=d[k].dtype, device="cuda")
        m[k] = b[1:].view(d[k].shape)
        m[k].copy_(d[k])
    y2, n2 = forward(m, L, layer=True)
    g2 = backward(m, L, FULL, layer=True)
    check_forward(t, L, y2, n2, True, 1e-6)
    check_backward(t, L, g2, True, 1e-6)
    assert y.shape == y2.shape and set(g) == set(g2) and n.shape == n2.shape


def test_nothing():
    w = torch.ones(8, device="cuda")
    h = torch.empty(0, 8, device="cuda")
    y, n = ss.ss2d_norm_forward(h, w_post=w, w_pre=w)
    assert y.shape == n.shape == (0, 8)
    d = ss.ss2d_norm_backward(h, y, y, n, w_post=w, w_pre=w, res_scale=w[None])
    assert (d["w_post"] == 0).all() and (d["w_pre"] == 0).all() and (d["res_scale"] == 0).all()


def test_a_block_of_the_delta_rule():
    """The operators in a row, as a layer uses them: the norm before, the gated delta rule, its
    heads' gated norm, then the residual with the next norm; against float64."""
    from tests import delta_util as du
    t = du.make_inputs(2, 70, 1, 2, 64, 64, torch.bfloat16, seed=7)
    d = du.to_gpu(t)
    gen = torch.Generator().manual_seed(8)
    z = torch.randn(2, 70, 2, 64, generator=gen).bfloat16()
    res = torch.randn(2, 70, 128, generator=gen)
    w, w2 = torch.rand(64, generator=gen) + 0.5, torch.rand(128, generator=gen) + 0.5
    gamma = torch.rand(128, generator=gen)
    o = ss.ss1d_delta_forward(*[d[n] for n in du.NAMES])
    p, _ = ss.ss2d_norm_forward(o, w_post=w.cuda(), z=z.cuda())
    y, n = ss.ss2d_norm_forward(p.reshape(2, 70, 128), residual=res.cuda(),
                                res_scale=gamma.cuda()[None], w_pre=w2.cuda(), layer=True)
    ro, _ = du.reference(t, 64 ** -0.5)
    rp = unit(ro.reshape(-1, 64), False, 1e-6) * w * torch.nn.functional.silu(z.double()).reshape(-1, 64)
    # o and p are each rounded to bfloat16; the norm divides by o's root mean square
    rms = 1 / ro.reshape(-1, 64).square().mean(1, keepdim=True).sqrt()
    tol = du.o_bounds(64, ro, torch.bfloat16)[0] * rms * 2 + 2 * 2.0 ** -8 * rp.abs().amax(1, keepdim=True)
    err = (p.double().cpu().reshape(-1, 64) - rp).abs()
    assert float((err - tol * (1 + z.double().abs().reshape(-1, 64))).max()) <= 0
    py = p.double().cpu().reshape(-1, 128) * gamma + res.double().reshape(-1, 128)
    check(y.reshape(-1, 128), py, "y", CHAIN * py.abs().amax(1, keepdim=True))
    check(n.reshape(-1, 128), unit(py, True, 1e-6) * w2, "n", CHAIN * 2 * py.abs().amax(1, keepdim=True)
          * (1 / py.var(1, unbiased=False, keepdim=True).sqrt()))


def test_graph_of_forward_and_backward():
    t = gpu(make(60, 192, 0, FULL, torch.bfloat16, torch.float32, True, seed=9, grad=True))

    def work():
        y, n = forward(t, 0, layer=True)
        return [y, n] + list(backward(t, 0, FULL, layer=True).values())

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = work()
    for i in range(3):
        t["h"].copy_(torch.randn_like(t["h"]))
        t["dn"].copy_(torch.randn_like(t["dn"]))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        for x, y in zip(got, work()):
            assert torch.equal(x, y), i
        torch.cuda.synchronize()
