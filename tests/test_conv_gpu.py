"""The short causal convolution on the GPU against its definition in 64 bits."""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import scan_util as su

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def gpu(t):
    out = {}
    for n, x in t.items():
        if x is not None and not x.is_contiguous():
            wide = torch.zeros(*x.shape[:2], 16 + x.shape[2], dtype=x.dtype, device="cuda")
            wide[..., 8:8 + x.shape[2]] = x
            x = wide[..., 8:8 + x.shape[2]]
        out[n] = x.cuda() if x is not None else None
    return out


def bounds(t, ref, dtype):
    """Sums of KW products and a bias in fp32, the activation's 6 half steps, the rounding."""
    KW = t["conv_w"].shape[1]
    size = su.top(t["x"].double()) + su.top(t["h0"].double() if t["h0"] is not None else None)
    pre = KW * su.top(t["conv_w"]) * max(size, 1e-6) + su.top(t["conv_b"])
    return su.F32_HALF * (KW + 8) * 1.1 * pre, su.half(dtype)


# B, L, D, KW, type, SiLU, bias, initial states, views
CASES = [
    (1, 1, 1, 1, F32, True, False, False, False), (2, 3, 5, 2, BF16, True, True, True, False),
    (2, 31, 8, 4, BF16, True, True, False, False), (1, 32, 16, 4, F32, True, True, True, True),
    (3, 33, 70, 4, BF16, False, True, True, True), (2, 70, 64, 3, F32, True, False, True, False),
    (1, 100, 264, 4, BF16, True, True, True, True), (2, 65, 130, 8, F32, True, True, True, False),
    (2, 2, 24, 8, BF16, True, True, True, False), (1, 97, 1100, 5, BF16, True, True, False, True),
    (2, 40, 40, 6, F32, False, False, True, True), (1, 64, 136, 7, BF16, True, True, True, False),
    (8, 197, 8192, 4, BF16, True, True, True, False), (3, 900, 2050, 8, F32, True, True, False, True),  # longer runs
]


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    B, L, D, KW, dtype, silu, bias, h0, views = case
    t = su.conv_inputs(B, L, D, KW, dtype, seed=L, bias=bias, h0=B if h0 else 0, views=views)
    ref, ends = su.conv_reference(t, silu)
    d = gpu(t)
    y, end = ss.ss1d_conv_forward(d["x"], d["conv_w"], d["conv_b"], silu=silu, initial_state=d["h0"], final_state=True)
    su.check(y, ref, "y", *bounds(t, ref, dtype))
    assert torch.equal(end.double().cpu(), ends)
    assert torch.equal(y, ss.ss1d_conv_forward(d["x"], d["conv_w"], d["conv_b"], silu=silu, initial_state=d["h0"]))


def check_gradients(t, got, ref, dtype):
    KW, T = t["conv_w"].shape[1], t["x"].shape[0] * t["x"].shape[1]
    wm, gm = su.top(t["conv_w"]), su.top(t["dy"].double())
    pre, rel = bounds(t, None, dtype)
    # the activation's slope is off by its argument's error (its own slope is at most 0.5) and 12
    # half steps; KW such terms make x's gradient, T of them a tap's
    e = 1.1 * gm * (0.5 * pre + 12 * su.F32_HALF)
    xm = max(su.top(t["x"].double()), su.top(t["h0"].double() if t["h0"] is not None else None))
    wide = KW * wm * e + su.F32_HALF * (KW + 1) * KW * wm * 1.1 * gm + su.F32_HALF * 2 * su.top(t["dht"].double() if t["dht"] is not None else None)
    su.check(got["x"], ref["x"], "dx", wide, rel)
    total = max(T, 1)
    su.check(got["conv_w"], ref["conv_w"], "dw", total * xm * (e + su.F32_HALF * total * 1.1 * gm))
    if "conv_b" in ref:
        su.check(got["conv_b"], ref["conv_b"], "db", total * (e + su.F32_HALF * total * 1.1 * gm))
    if "h0" in ref:
        su.check(got["initial_state"], ref["h0"], "dh0", wide, rel)


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    B, L, D, KW, dtype, silu, bias, h0, views = case
    t = su.conv_inputs(B, L, D, KW, dtype, seed=L, bias=bias, h0=B if h0 else 0, views=views)
    d = gpu(t)
    got = ss.ss1d_conv_backward(d["x"], d["conv_w"], d["dy"], d["conv_b"], silu=silu, initial_state=d["h0"],
                                dstate=d["dht"])
    check_gradients(t, got, su.conv_reference(t, silu, grads=True), dtype)


PACKED = [
    (40, [0, 40], 16, 4, F32), (50, [0, 0, 7, 7, 40, 50, 50], 24, 4, BF16), (120, [3, 20, 20, 61, 115], 70, 3, F32),
    (90, [0, 1, 2, 3, 90], 64, 8, BF16), (0, [0, 0, 0], 8, 4, F32), (64, [0, 32, 64], 33, 4, BF16),
]


@pytest.mark.parametrize("case", PACKED)
def test_packed(case):
    T, cu, D, KW, dtype = case
    t = su.conv_inputs(1, T, D, KW, dtype, seed=T, h0=len(cu) - 1)
    ref, ends = su.conv_reference(t, True, cu)
    d, at = gpu(t), torch.tensor(cu, dtype=torch.int32).cuda()
    y = torch.full_like(d["x"], 7.0)  # tokens outside of every sequence stay
    state = d["h0"].clone()
    y, end = ss.ss1d_conv_forward(d["x"], d["conv_w"], d["conv_b"], cu_seqlens=at, initial_state=state,
                                  final_state=state, y=y)
    assert end is state and torch.equal(end.double().cpu(), ends)
    ref[0, :cu[0]] = 7.0
    ref[0, cu[-1]:] = 7.0
    su.check(y, ref, "y", *bounds(t, ref, dtype))
    got = ss.ss1d_conv_backward(d["x"], d["conv_w"], d["dy"], d["conv_b"], cu_seqlens=at, initial_state=d["h0"],
                                dstate=d["dht"])
    check_gradients(t, got, su.conv_reference(t, True, cu, grads=True), dtype)


@pytest.mark.parametrize("case", [(1, 1, 1, 1, F32), (3, 1, 64, 4, BF16), (5, 5, 70, 4, BF16), (4, 2, 520, 3, F32),
                                  (2, 9, 24, 8, BF16), (70, 2, 16, 4, F32)])
def test_step(case):
    B, T, D, KW, dtype = case
    t = su.conv_inputs(B, T, D, KW, dtype, seed=D, h0=B, views=D > 60)
    ref, ends = su.conv_reference(t)
    d = gpu(t)
    state = d["h0"].clone()
    y = ss.ss1d_conv_step(d["x"], d["conv_w"], state, d["conv_b"])
    su.check(y, ref, "y", *bounds(t, ref, dtype))
    assert torch.equal(state.double().cpu(), ends)
    slots = torch.randperm(B + 2, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    pad = B // 2 if B > 1 else -1
    if pad >= 0:
        slots[pad] = B + 2 + 5
    real = torch.tensor([i != pad for i in range(B)]).cuda()
    at = slots.long().cuda()[real]
    pool = torch.full((B + 2, KW - 1, D), 9.0, device="cuda").to(dtype)
    pool[at] = d["h0"][real]
    out = ss.ss1d_conv_step(d["x"], d["conv_w"], pool, d["conv_b"], slots=slots.cuda(), y=torch.full_like(y, 5.0))
    assert torch.equal(out[real], y[real]) and (out[~real] == 5.0).all()
    assert torch.equal(pool[at], state[real])
    if KW > 1:
        others = [i for i in range(B + 2) if i not in slots.tolist()]
        assert (pool[others] == 9.0).all()


def test_step_rows_of_one_slot_are_successive_tokens():
    B, D, KW = 70, 24, 4
    t = su.conv_inputs(B, 2, D, KW, F32, seed=3, h0=1)
    slots = torch.full((B,), 1, dtype=torch.int32)
    slots[5:60] = -1
    d = gpu(t)
    state = torch.zeros(2, KW - 1, D, device="cuda")
    state[1] = d["h0"][0]
    rows = torch.nonzero(slots == 1).flatten()
    seq = {**t, "x": t["x"][rows].flatten(0, 1)[None], "dht": None}
    ref, ends = su.conv_reference(seq)
    y = ss.ss1d_conv_step(d["x"], d["conv_w"], state, d["conv_b"], slots=slots.cuda())
    su.check(y[rows.cuda()].flatten(0, 1)[None], ref, "y", *bounds(seq, ref, F32))
    assert torch.equal(state[1:].double().cpu(), ends) and not state[0].any()


def test_nan_reaches_its_taps_only():
    t = gpu(su.conv_inputs(2, 60, 16, 4, F32, seed=4))
    clean = ss.ss1d_conv_forward(t["x"], t["conv_w"], t["conv_b"])
    t["x"][1, 30, 3] = float("nan")
    y = ss.ss1d_conv_forward(t["x"], t["conv_w"], t["conv_b"])
    hit = torch.zeros_like(y, dtype=torch.bool)
    hit[1, 30:34, 3] = True
    assert y[hit].isnan().all() and torch.equal(y[~hit], clean[~hit])
