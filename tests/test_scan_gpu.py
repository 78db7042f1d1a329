"""The token-order scan on the GPU against its definition in 64 bits: forward, states, packed
sequences, segments, gradients, and the form for single tokens."""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import scan_util as su

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def gpu(t):
    """The same on the GPU, views kept views."""
    out = {}
    for n, x in t.items():
        if x is not None and not x.is_contiguous():
            wide = torch.zeros(*x.shape[:2], 7 + x[0, 0].numel(), dtype=x.dtype, device="cuda")
            y = wide[..., 7:].unflatten(-1, x.shape[2:])
            y.copy_(x)
            out[n] = y
        else:
            out[n] = x.cuda() if x is not None else None
    return out


def args(t):
    return [t[n] for n in su.NAMES]


# B, L, D, G, N, type, gate, initial states, views, segment
CASES = [
    (1, 1, 1, 1, 1, F32, False, False, False, -1),
    (2, 2, 5, 1, 2, BF16, True, False, False, -1),
    (1, 15, 16, 1, 3, F32, True, True, True, -1),
    (3, 16, 17, 1, 4, BF16, False, True, False, 0),
    (2, 17, 63, 3, 7, F32, True, False, False, 0),
    (1, 33, 64, 2, 8, BF16, True, True, True, 16),
    (2, 70, 65, 5, 12, F32, False, True, True, 32),
    (2, 100, 130, 1, 16, BF16, True, True, True, -1),
    (1, 100, 130, 2, 16, F32, True, True, False, 48),
    (2, 64, 80, 1, 16, F32, True, False, True, 16),
    (1, 41, 40, 1, 17, F32, True, True, False, 8),
    (2, 50, 70, 1, 32, BF16, True, True, True, 16),
    (1, 50, 130, 2, 32, F32, False, True, False, 0),
    (2, 331, 20, 1, 16, F32, True, True, False, 8),  # 42 segments, joined by 16 waves
    (1, 270, 33, 1, 5, BF16, True, True, False, 8),
]


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    B, L, D, G, N, dtype, gate, h0, views, seg = case
    t = su.make_inputs(B, L, D, G, N, dtype, seed=L + N, gate=gate, h0=B if h0 else 0, views=views)
    ref, ends, hm = su.reference(t)
    d = gpu(t)
    for lanes in (16, 4):
        with su.plan(seg, lanes):
            y, end = ss.ss1d_scan_forward(*args(d), z=d["z"], initial_state=d["h0"], final_state=True)
            alone = ss.ss1d_scan_forward(*args(d), z=d["z"], initial_state=d["h0"])
        su.check(y, ref, "y", *su.y_bounds(t, hm))
        su.check(end, ends, "end states", su.state_bound(t, hm))
        assert torch.equal(y, alone)
    with su.plan(seg):
        y2, end2, saved = ss.ss1d_scan_forward_save(*args(d), z=d["z"], initial_state=d["h0"], final_state=True)
    assert torch.equal(y, y2) and torch.equal(end, end2)  # both by four lanes


PACKED = [
    (40, [0, 40], 16, 1, 16, F32, True, -1),
    (50, [0, 0, 7, 7, 40, 50, 50], 20, 1, 16, BF16, True, -1),
    (90, [3, 20, 20, 61, 85], 70, 2, 16, F32, True, 16),
    (90, [0, 1, 2, 3, 90], 65, 1, 8, F32, False, 32),
    (64, [0, 16, 32, 64], 64, 1, 4, BF16, True, 16),
    (33, [0, 0, 0, 33], 40, 1, 32, F32, True, 8),
    (560, [0, 200, 200, 203, 560], 24, 1, 7, F32, True, 8),  # the same join for sequences of 0 to 45 segments
    (0, [0, 0, 0], 20, 1, 16, F32, True, -1),
]


@pytest.mark.parametrize("case", PACKED)
def test_packed_forward(case):
    T, cu, D, G, N, dtype, gate, seg = case
    t = su.make_inputs(1, T, D, G, N, dtype, seed=T + N, gate=gate, h0=len(cu) - 1)
    ref, ends, hm = su.reference(t, cu)
    d, at = gpu(t), torch.tensor(cu, dtype=torch.int32).cuda()
    ref[0, :cu[0]] = 7.0  # tokens outside of every sequence stay
    ref[0, cu[-1]:] = 7.0
    for lanes in (4, 16):
        y, state = torch.full_like(d["u"], 7.0), d["h0"].clone()
        with su.plan(seg, lanes):
            y, end = ss.ss1d_scan_forward(*args(d), z=d["z"], cu_seqlens=at, initial_state=state, final_state=state,
                                          y=y)
        assert end is state
        su.check(y, ref, "y", *su.y_bounds(t, hm, cu))
        su.check(end, ends, "end states", su.state_bound(t, hm, cu))


def check_gradients(t, got, cu=None):
    ref, bounds = su.adjoint(t, cu)
    for n in list(su.NAMES) + (["z"] if t["z"] is not None else []):
        rel = su.half(t["u"].dtype) if n in ("u", "dt_raw", "Bs", "Cs", "z") else 0.0
        su.check(got[n], ref[n], "d" + n, bounds[n], rel)
    if t["h0"] is not None:
        su.check(got["initial_state"], ref["h0"], "dh0", bounds["h0"])


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    B, L, D, G, N, dtype, gate, h0, views, seg = case
    t = su.make_inputs(B, L, D, G, N, dtype, seed=L + N, gate=gate, h0=B if h0 else 0, views=views)
    d = gpu(t)
    kw = dict(z=d["z"], initial_state=d["h0"])
    with su.plan(seg):
        _, saved = ss.ss1d_scan_forward_save(*args(d), **kw)
        got = ss.ss1d_scan_backward(*args(d), d["dy"], dstate=d["dht"], saved=saved, **kw)
        again = ss.ss1d_scan_backward(*args(d), d["dy"], dstate=d["dht"], **kw)
    check_gradients(t, got)
    for n in got:
        assert torch.equal(got[n], again[n]), n


@pytest.mark.parametrize("case", PACKED)
def test_packed_backward(case):
    T, cu, D, G, N, dtype, gate, seg = case
    t = su.make_inputs(1, T, D, G, N, dtype, seed=T + N, gate=gate, h0=len(cu) - 1)
    d, at = gpu(t), torch.tensor(cu, dtype=torch.int32).cuda()
    kw = dict(z=d["z"], initial_state=d["h0"], cu_seqlens=at)
    with su.plan(seg):
        _, saved = ss.ss1d_scan_forward_save(*args(d), **kw)
        got = ss.ss1d_scan_backward(*args(d), d["dy"], dstate=d["dht"], saved=saved, **kw)
        again = ss.ss1d_scan_backward(*args(d), d["dy"], dstate=d["dht"], **kw)
    check_gradients(t, got, cu)
    for n in got:
        assert torch.equal(got[n], again[n]), n


def test_gradients_against_differences():
    """Central differences of the forward along random directions, fp32."""
    t = gpu(su.make_inputs(2, 37, 24, 2, 16, F32, seed=5, h0=2))
    names = list(su.NAMES) + ["z", "h0"]

    def loss(s):
        y, end = ss.ss1d_scan_forward(*args(s), z=s["z"], initial_state=s["h0"], final_state=True)
        return float((y.double() * t["dy"].double()).sum() + (end.double() * t["dht"].double()).sum())

    got = ss.ss1d_scan_backward(*args(t), t["dy"], z=t["z"], initial_state=t["h0"], dstate=t["dht"])
    got["h0"] = got["initial_state"]
    eps = 1e-2
    for n in names:
        gen = torch.Generator(device="cuda").manual_seed(len(n))
        v = torch.randn(t[n].shape, generator=gen, device="cuda")
        v = v / v.norm()
        up, down = (loss({**t, n: t[n] + s * eps * v}) for s in (1, -1))
        want, mine = (up - down) / (2 * eps), float((got[n].double() * v.double()).sum())
        # the difference's own error: eps^2 / 6 of the third derivative along v (of the loss's scale
        # at most) and the forward's roundings over 2 eps
        scale = float(got[n].double().norm()) + 1.0
        assert abs(want - mine) <= scale * (eps ** 2 + 1e-3), n


STEPS = [
    (1, 1, 1, 1, 1, F32, False), (3, 1, 17, 1, 4, BF16, True), (2, 5, 64, 2, 8, F32, True),
    (5, 3, 70, 5, 16, BF16, True), (4, 2, 33, 1, 12, F32, True), (2, 2, 40, 1, 32, BF16, False),
    (2, 1, 40, 1, 20, F32, True),
]


@pytest.mark.parametrize("views", [False, True])
@pytest.mark.parametrize("case", STEPS)
def test_step(case, views):
    B, T, D, G, N, dtype, gate = case
    t = su.make_inputs(B, T, D, G, N, dtype, seed=D, gate=gate, h0=B, views=views)
    ref, ends, hm = su.reference(t)
    d = gpu(t)
    state = d["h0"].clone()
    y = ss.ss1d_scan_step(*args(d), state, z=d["z"])
    su.check(y, ref, "y", *su.y_bounds(t, hm))
    su.check(state, ends, "state", su.state_bound(t, hm))
    # the same through slots of a pool, in another order, with padding rows among them
    S = B + 3
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(1))[:B].to(torch.int32)
    slots[B // 2] = -1 if B > 1 else slots[0]
    pool = torch.full((S, D, N), 9.0, device="cuda")
    real = slots >= 0
    pool[slots[real].long().cuda()] = d["h0"][real.cuda()]
    out = ss.ss1d_scan_step(*args(d), pool, z=d["z"], slots=slots.cuda(), y=torch.full_like(y, 5.0))
    assert torch.equal(out[real.cuda()], y[real.cuda()]) and (out[~real.cuda()] == 5.0).all()
    assert torch.equal(pool[slots[real].long().cuda()], state[real.cuda()])
    others = [i for i in range(S) if i not in slots.tolist()]
    assert (pool[others] == 9.0).all()


def test_step_rows_of_one_slot_are_successive_tokens():
    B, D, N = 70, 20, 16
    t = su.make_inputs(B, 2, D, 1, N, F32, seed=3, h0=1)
    slots = torch.full((B,), 1, dtype=torch.int32)
    slots[5:60] = -1
    slots[7] = 2  # past the pool: padding as well
    d = gpu(t)
    state = torch.zeros(2, D, N, device="cuda")
    state[1] = d["h0"][0]
    rows = torch.nonzero(slots == 1).flatten()
    seq = {n: (x[rows].flatten(0, 1)[None] if n in ("u", "dt_raw", "Bs", "Cs", "z", "dy") else x) for n, x in t.items()}
    ref, ends, hm = su.reference(seq)
    y = ss.ss1d_scan_step(*args(d), state, z=d["z"], slots=slots.cuda())
    su.check(y[rows.cuda()].flatten(0, 1)[None], ref, "y", *su.y_bounds(seq, hm))
    su.check(state[1:], ends, "state", su.state_bound(seq, hm))
    assert not state[0].any()


def test_steps_continue_a_prompt():
    t = su.make_inputs(2, 50, 40, 1, 16, F32, seed=9)
    d = gpu(t)
    whole = ss.ss1d_scan_forward(*args(d), z=d["z"])

    def part(a, e):
        return [d[n][:, a:e].contiguous() if n in ("u", "dt_raw", "Bs", "Cs") else d[n] for n in su.NAMES], \
            d["z"][:, a:e].contiguous()

    seq, z = part(0, 44)
    y, state = ss.ss1d_scan_forward(*seq, z=z, final_state=True)
    ys = [y]
    for i in range(44, 50):
        seq, z = part(i, i + 1)
        ys.append(ss.ss1d_scan_step(*seq, state, z=z))
    _, _, hm = su.reference(t)
    su.check(torch.cat(ys, 1), whole.double().cpu(), "y", 2 * su.y_bounds(t, hm)[0])


def test_extreme_steps():
    """delta of 0 and infinity, A of 0: nothing forgotten, everything forgotten."""
    t = su.make_inputs(1, 40, 16, 1, 16, F32, seed=2, h0=1)
    t["dt_raw"][0, 10] = -float("inf")   # delta 0: the state stays
    t["dt_raw"][0, 20] = 300.0           # the state is forgotten
    t["A_log"][3] = -float("inf")        # no decay at all
    ref, ends, hm = su.reference(t)
    d = gpu(t)
    for seg, lanes in ((0, 4), (16, 4), (0, 16), (16, 16)):
        with su.plan(seg, lanes):
            y, end = ss.ss1d_scan_forward(*args(d), z=d["z"], initial_state=d["h0"], final_state=True)
        su.check(y, ref, "y", *su.y_bounds(t, hm))
        su.check(end, ends, "end", su.state_bound(t, hm))


@pytest.mark.parametrize("name", ["u", "dt_raw", "z", "Bs", "Cs"])
@pytest.mark.parametrize("seg, lanes", [(0, 4), (16, 4), (0, 16), (16, 16)])
def test_nan_reaches_no_earlier_token_nor_other_sequence(name, seg, lanes):
    t = su.make_inputs(2, 60, 40, 2, 16, F32, seed=4)
    d = gpu(t)
    with su.plan(seg, lanes):
        clean, end0 = ss.ss1d_scan_forward(*args(d), z=d["z"], final_state=True)
        d[name][1, 30].view(-1)[3] = float("nan")
        y, end = ss.ss1d_scan_forward(*args(d), z=d["z"], final_state=True)
    assert torch.equal(y[0], clean[0]) and torch.equal(end[0], end0[0])
    assert torch.equal(y[1, :30], clean[1, :30])
    wide = slice(3, 4) if name in ("u", "dt_raw", "z") else slice(0, 20)  # its channel, or its group
    rest = torch.ones(40, dtype=torch.bool)
    rest[wide] = False
    assert torch.equal(y[1][:, rest], clean[1][:, rest]) and torch.equal(end[1][rest], end0[1][rest])
    assert y[1, 30, wide].isnan().all()
    if name not in ("z", "Cs"):
        assert y[1, 30:, wide].isnan().all() and end[1][wide].isnan().any()


def test_padded_offsets_touch_nothing_else():
    """Offsets out of order and out of range stay inside the tensors."""
    t = gpu(su.make_inputs(1, 64, 40, 1, 16, F32, seed=6))
    big = torch.full((3, 64, 40), 3.0, device="cuda")
    cu = torch.tensor([-5, 40, 20, 900, 64], dtype=torch.int32, device="cuda")
    for seg in (0, 16):
        with su.plan(seg):
            ss.ss1d_scan_forward(*args(t), z=t["z"], cu_seqlens=cu, final_state=True, y=big[1:2])
            ss.ss1d_scan_backward(*args(t), t["dy"], z=t["z"], cu_seqlens=cu)
    assert (big[0] == 3.0).all() and (big[2] == 3.0).all()
