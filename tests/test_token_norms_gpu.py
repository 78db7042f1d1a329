"""Gradients of the token-order scan, its convolution and the group norm against 64 bits by norms, whose bounds
stay far below the gradients (the absolute bounds of the parameters' gradients beside them may not), and the
kernels' paths that only large calls take: steps of several rows a block, deep rows of the group norm,
several units a thread of the convolution's backward."""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import scan_util as su
from tests import test_group_norm_gpu as gn
from tests import token_util as tu
from tests.test_conv_gpu import CASES as CONV_CASES
from tests.test_conv_gpu import gpu as conv_gpu
from tests.test_scan_gpu import CASES, PACKED, args, gpu

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def scan_both(t, seg, cu=None):
    d = gpu(t)
    at = torch.tensor(cu, dtype=torch.int32).cuda() if cu is not None else None
    kw = dict(z=d["z"], initial_state=d["h0"], cu_seqlens=at)
    with su.plan(seg):
        y, end, saved = ss.ss1d_scan_forward_save(*args(d), final_state=True, y=torch.zeros_like(d["u"]), **kw)
        got = ss.ss1d_scan_backward(*args(d), d["dy"], dstate=d["dht"], saved=saved, **kw)
    tu.check_scan(t, y, end, got, cu)


@pytest.mark.parametrize("case", CASES)
def test_scan(case):
    B, L, D, G, N, dtype, gate, h0, views, seg = case
    scan_both(su.make_inputs(B, L, D, G, N, dtype, seed=L + N, gate=gate, h0=B if h0 else 0, views=views), seg)


@pytest.mark.parametrize("case", PACKED)
def test_packed_scan(case):
    T, cu, D, G, N, dtype, gate, seg = case
    scan_both(su.make_inputs(1, T, D, G, N, dtype, seed=T + N, gate=gate, h0=len(cu) - 1), seg, cu)


@pytest.mark.parametrize("seg", [-1, 0, 64])
@pytest.mark.parametrize("first", [True, False])
def test_a_prompt_among_single_tokens(first, seg):
    """Continuous batching: one prompt of 700 tokens and 150 sequences of one token or none."""
    singles = [n % 5 != 3 for n in range(150)]
    lengths = [700] + singles if first else singles + [700]
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + int(n))
    scan_both(su.make_inputs(1, cu[-1], 24, 1, 16, F32, seed=11, h0=len(lengths)), seg, cu)


# B, L, D, N, segment, offsets: 69, 130 and 75 or so units, whose sums go four at a time and some alone
@pytest.mark.parametrize("B, L, D, N, seg, cu", [
    (1, 1100, 20, 16, 16, None), (65, 20, 9, 4, 16, None), (1, 1000, 12, 16, 16, [0, 3, 400, 400, 401, 993]),
    (1, 530, 8, 32, 8, None)])
def test_parameter_sums_of_many_units(B, L, D, N, seg, cu):
    S = B if cu is None else len(cu) - 1
    scan_both(su.make_inputs(B, L, D, 1, N, F32, seed=L, h0=S), seg, cu)


def step_reference(t, state, slots):
    """y and the states in float64 on the GPU: the first row of every slot, then the second, ..."""
    c = {n: x.double() for n, x in t.items() if isinstance(x, torch.Tensor)}
    A, rep = -c["A_log"].exp(), c["u"].shape[2] // c["Bs"].shape[2]
    delta = torch.nn.functional.softplus(c["dt_raw"] + c["dt_bias"], threshold=1e3)
    h, y = state.double(), torch.zeros_like(c["u"])
    order, seen = {}, {}
    for b, slot in enumerate(slots.tolist()):
        if 0 <= slot < state.shape[0]:
            seen[slot] = seen.get(slot, -1) + 1
            order.setdefault(seen[slot], []).append(b)
    hm = su.top(h)
    for rows in order.values():
        at = slots[rows].long().to(h.device)
        now = h[at]
        for i in range(c["u"].shape[1]):
            Bt, Ct = (c[n][rows, i].repeat_interleave(rep, 1) for n in ("Bs", "Cs"))
            now = (delta[rows, i][..., None] * A).exp() * now + (delta[rows, i] * c["u"][rows, i])[..., None] * Bt
            hm = max(hm, su.top(now))
            y[rows, i] = (now * Ct).sum(-1) + c["Ds"] * c["u"][rows, i]
        h[at] = now
    if "z" in c:
        y = y * c["z"] * torch.sigmoid(c["z"])
    wm = su.top(delta) * su.top(c["u"]) * su.top(c["Bs"])
    eh = su.F32_HALF * (len(order) * c["u"].shape[1] + 1) * (8 * hm + 6 * wm)  # as su.state_bound's
    N, cm = A.shape[1], su.top(c["Cs"])
    ey = N * cm * eh + su.F32_HALF * (N + 8) * (N * cm * hm + 2 * su.top(c["u"]) * su.top(c["Ds"]))
    return y, h, eh, ey * (max(1.0, su.top(c["z"])) if "z" in c else 1.0)


# rows of a block: 8, 6, 2 and 16
@pytest.mark.parametrize("B, T, D, G, N, dtype", [(256, 1, 4096, 1, 16, BF16), (300, 2, 3000, 3, 12, F32),
                                                  (4101, 1, 64, 1, 8, F32), (2100, 1, 1000, 1, 32, BF16)])
def test_steps_of_several_rows_a_block(B, T, D, G, N, dtype):
    t = gpu(su.make_inputs(B, T, D, G, N, dtype, seed=D))
    gen = torch.Generator(device="cuda").manual_seed(B)
    S = B + 40
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(2))[:B].to(torch.int32)
    # repeats within a block, in the next one and in the last; padding alone, side by side, and next to repeats
    for row, of in ((3, 1), (4, 1), (21, 1), (100, 99), (B - 1, 0), (B - 2, 2)):
        slots[row] = slots[of]
    slots[5] = slots[6] = -1
    slots[7] = S
    slots[200:217] = -7
    slots[B - 4] = S + 9
    state = torch.randn(S, D, N, generator=gen, device="cuda")
    ref, ends, eh, ey = step_reference(t, state, slots)
    before = state.clone()
    y = ss.ss1d_scan_step(*args(t), state, z=t["z"], slots=slots.cuda(), y=torch.full_like(t["u"], 7.0))
    pad = (slots < 0) | (slots >= S)
    ref[pad.cuda()] = 7.0
    err = (y.double() - ref).abs() - su.half(dtype) * ref.abs()
    assert float(err.max()) <= ey
    assert float((state.double() - ends).abs().max()) <= eh
    idle = torch.ones(S, dtype=torch.bool)
    idle[slots[~pad].long()] = False
    assert torch.equal(state[idle.cuda()], before[idle.cuda()])
    assert (y[pad.cuda()] == 7.0).all()


def group_gradients(case):
    """The norms of dweight's and dbias's errors, on the GPU in float64, at a mean near the deviation."""
    shape, G, dtype, silu, _ = case
    half, eps = su.F32_HALF, 1e-5
    x, dy, w, b = gn.make(shape, dtype, True, seed=len(shape) + shape[-1])
    xc, dc, wc, bc = (v.cuda() for v in (x, dy, w, b))
    B, C = shape[0], shape[-1]
    v = xc.double().reshape(B, -1, G, C // G)
    mean = v.mean((1, 3), keepdim=True)
    r = ((v - mean).square().mean((1, 3), keepdim=True) + eps).rsqrt()
    n = ((v - mean) * r).reshape(B, -1, C)
    g = dc.double().reshape(B, -1, C)
    w64, b64 = wc.double(), bc.double()
    d = g
    if silu:
        pre = n * w64 + b64
        s = torch.sigmoid(pre)
        d = g * s * (1 + pre * (1 - s))
    count, total = v[0, :, 0].numel(), B * n.shape[1]
    # half steps in quadrature of sums over a group and over all tokens, and those of a value
    k, kt = (8 + gn.summed(m) ** 0.5 for m in (count, total))
    en = half * k * (su.top(v) * float(r.max()) + n.abs())
    ed = g.abs() * ((0.5 * w64.abs() * en if silu else 0.0) + 12 * half)
    for given in (True, False):
        stats = ss.ss2d_group_norm_forward(xc, G, wc, bc, silu, eps, stats=True)[1] if given else None
        got = ss.ss2d_group_norm_backward(xc, dc, G, wc, bc, silu, eps, stats=stats)
        for name, term, off in (("weight", d * n, ed * n.abs() + d.abs() * en), ("bias", d, ed)):
            ref = term.sum((0, 1))
            bound = float((off.sum((0, 1)) + half * kt * term.abs().sum((0, 1))).norm())
            # (groups of one value have unit values, and dweight, of exactly 0)
            assert bound <= 0.05 * float(ref.norm()) or not ref.any(), "the bound says nothing"
            err = float((got[name].double() - ref).norm())
            assert err <= bound, f"d{name}: off by {err:.3e} against {bound:.3e}"


@pytest.mark.parametrize("case", [c for c in gn.CASES if c[-1]])
def test_group_norm_parameters(case):
    group_gradients(case)


# rows of a thread forward and backward: bf16 10 and 10, 10 and 10, 4 and 8; fp32 20 and 10, 8 and 8, 16 and 4, 14 and chunks
DEEP = [((64, 28, 28, 384), 32, BF16, True, True), ((64, 1500, 96), 16, BF16, True, True),
        ((48, 32, 32, 96), 16, BF16, True, True), ((64, 28, 28, 384), 32, F32, True, True),
        ((48, 32, 32, 96), 16, F32, True, True), ((64, 32, 32, 256), 32, F32, False, True),
        ((64, 2300, 96), 16, F32, True, True)]


@pytest.mark.parametrize("case", DEEP)
def test_group_norm_of_deep_rows(case):
    gn.test_both_directions(case, 0.5)
    group_gradients(case)


def test_group_norm_by_chunks_off_16_bytes():
    """Rows that start off 16 bytes, of groups too large for registers: by single values."""
    x, dy, w, b = (v.cuda() for v in gn.make((2, 20000, 64), BF16, True))
    off = torch.zeros(x.numel() + 1, dtype=BF16, device="cuda")[1:].view(x.shape)
    off.copy_(x)
    assert off.data_ptr() % 16 and off.is_contiguous()
    kw = dict(weight=w, bias=b)
    y, stats = ss.ss2d_group_norm_forward(off, 2, stats=True, **kw)
    want, same = ss.ss2d_group_norm_forward(x, 2, stats=True, **kw)
    d, dwant = ss.ss2d_group_norm_backward(off, dy, 2, **kw), ss.ss2d_group_norm_backward(x, dy, 2, **kw)
    # sums of 640,000 values in another order: their roundings in quadrature
    e = (8 + gn.summed(640000) ** 0.5) * su.F32_HALF
    assert float((stats / same - 1).abs()[..., 1].max()) <= 2 * e
    for got, ref, rel in [(y, want, su.BF16_HALF), (d["x"], dwant["x"], su.BF16_HALF)] + [
            (d[n], dwant[n], 0.0) for n in ("weight", "bias")]:
        got, ref = got.double(), ref.double()
        # both are rounded to bfloat16; the parameters' sums go over 40,000 positions, whose terms
        # of both signs leave 1 / 200 of their magnitudes
        bound = (2 * rel + 8 * e) * float(ref.norm()) if rel else 200 * 2 * e * float(ref.norm())
        assert float((got - ref).norm()) <= bound


def conv_parameters(t, silu):
    """The norms of the errors of dconv_w and dconv_b, on the GPU in float64, and x's gradient."""
    half, dtype = su.F32_HALF, t["x"].dtype
    got = ss.ss1d_conv_backward(t["x"], t["conv_w"], t["dy"], t["conv_b"], silu=silu, initial_state=t["h0"],
                                dstate=t["dht"])
    x, w, dy = (t[n].double() for n in ("x", "conv_w", "dy"))
    (B, L, D), KW = x.shape, w.shape[1]
    before = t["h0"].double() if t["h0"] is not None else x.new_zeros(B, KW - 1, D)
    whole = torch.cat([before, x], 1)
    d, off = dy, 12 * half * dy.abs()
    if silu:
        pre = sum(whole[:, j:j + L] * w[:, j] for j in range(KW)) + (t["conv_b"].double() if t["conv_b"] is not None else 0)
        size = sum(whole[:, j:j + L].abs() * w[:, j].abs() for j in range(KW)) + (
            t["conv_b"].double().abs() if t["conv_b"] is not None else 0)
        s = torch.sigmoid(pre)
        d = dy * s * (1 + pre * (1 - s))
        off = dy.abs() * (0.5 * half * (KW + 8) * size + 12 * half)  # the slope's own slope is at most 0.5
    # a sum over B L tokens: a thread's runs and 2048 blocks' parts one after the other, in quadrature
    k = 16 + (B * L) ** 0.5
    sums = [("conv_b", d, off)] if t["conv_b"] is not None else []
    sums += [(j, d * whole[:, j:j + L], off * whole[:, j:j + L].abs()) for j in range(KW)]
    for name, term, e in sums:
        ref = term.sum((0, 1))
        bound = float((e.sum((0, 1)) + half * k * term.abs().sum((0, 1)) / max(1.0, (B * L) ** 0.5)).norm())
        bound += half * k * float(term.square().sum((0, 1)).sqrt().norm())
        assert bound <= 0.02 * float(ref.norm()), "the bound says nothing"
        mine = got["conv_b"] if name == "conv_b" else got["conv_w"][:, name]
        err = float((mine.double() - ref).norm())
        assert err <= bound, f"d{name}: off by {err:.3e} against {bound:.3e}"
    behind = torch.cat([d, d.new_zeros(B, KW - 1, D)], 1)
    wide = sum(behind[:, i:i + whole.shape[1] - KW + 1] * w[:, KW - 1 - i] for i in range(KW))
    if t["dht"] is not None:
        tail = t["dht"].double()
        keep = min(L, KW - 1)
        wide[:, L - keep:] += tail[:, KW - 1 - keep:]
    err = float((got["x"].double() - wide).norm())
    assert err <= (tu.STEPS + su.half(dtype)) * float(wide.norm())


@pytest.mark.parametrize("case", CONV_CASES)
def test_conv_parameters(case):
    B, L, D, KW, dtype, silu, bias, h0, views = case
    conv_parameters(conv_gpu(su.conv_inputs(B, L, D, KW, dtype, seed=L, bias=bias, h0=B if h0 else 0, views=views)), silu)


# units of 24 tokens of a thread: 1.95, 2.4 and 1.5 on average, of four channels and of one
@pytest.mark.parametrize("B, L, D, KW, dtype", [(4, 3000, 8192, 4, BF16), (3, 5000, 8192, 8, F32), (4, 1100, 4099, 3, BF16)])
def test_conv_of_several_units_a_thread(B, L, D, KW, dtype):
    gen = torch.Generator(device="cuda").manual_seed(L)
    x, dy = (torch.randn(B, L, D, generator=gen, device="cuda").to(dtype) for _ in range(2))
    w, b = torch.randn(D, KW, generator=gen, device="cuda"), torch.randn(D, generator=gen, device="cuda")
    conv_parameters(dict(x=x, dy=dy, conv_w=w, conv_b=b, h0=None, dht=None), True)
