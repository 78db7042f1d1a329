"""Calls of the token-order scan, its convolution and the group norm at the ends of what their definitions
cover: decays past fp32, no positions, no channels, views whose unused strides are wide."""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import scan_util as su
from tests import token_util as tu
from tests.test_scan_gpu import args, gpu

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("L, N", [(41, 16), (48, 16), (21, 32), (70, 5)])
@pytest.mark.parametrize("seg, lanes", [(0, 4), (16, 4), (0, 16), (16, 16)])
def test_decays_past_fp32(L, N, seg, lanes):
    """exp(A_log) above the largest fp32: the state forgets everything at each token, whether or not the
    length is whole tiles; channels up to the block's last, whose values idle lanes copy."""
    t = su.make_inputs(2, L, 70, 1, N, F32, seed=L, h0=2)
    t["A_log"][3, :2], t["A_log"][40], t["A_log"][69] = 89.0, 200.0, 500.0
    d = gpu(t)
    kw = dict(z=d["z"], initial_state=d["h0"])
    with su.plan(seg, lanes):
        y, end = ss.ss1d_scan_forward(*args(d), final_state=True, **kw)
        _, saved = ss.ss1d_scan_forward_save(*args(d), **kw)
        got = ss.ss1d_scan_backward(*args(d), d["dy"], dstate=d["dht"], saved=saved, **kw)
    tu.check_scan(t, y, end, got)


def test_infinite_decay():
    """A_log of +infinity: the same as any that forgets everything; of NaN: its channel is NaN, no other."""
    t = gpu(su.make_inputs(1, 41, 40, 1, 16, F32, seed=3, h0=1))
    t["A_log"][7] = 300.0
    want = ss.ss1d_scan_forward(*args(t), z=t["z"], initial_state=t["h0"], final_state=True)
    t["A_log"][7] = float("inf")
    for seg, lanes in ((0, 4), (16, 4), (0, 16)):
        with su.plan(seg, lanes):
            got = ss.ss1d_scan_forward(*args(t), z=t["z"], initial_state=t["h0"], final_state=True)
        assert torch.allclose(got[0], want[0], rtol=1e-4, atol=1e-4) and torch.allclose(got[1], want[1], rtol=1e-4, atol=1e-4)
    t["A_log"][7, 3] = float("nan")
    state = t["h0"].clone()
    one = [t[n][:, :1].contiguous() if n in ("u", "dt_raw", "Bs", "Cs") else t[n] for n in su.NAMES]
    for y, end in (ss.ss1d_scan_forward(*args(t), z=t["z"], initial_state=t["h0"], final_state=True),
                   (ss.ss1d_scan_step(*one, state, z=t["z"][:, :1].contiguous()), state)):
        assert y[:, :, 7].isnan().all() and end[:, 7, 3].isnan().all()
        assert int(y.isnan().sum()) == y.shape[1] and int(end.isnan().sum()) == 1


def test_step_decays_past_fp32():
    t = su.make_inputs(3, 2, 40, 1, 16, F32, seed=5, h0=3)
    t["A_log"][3], t["A_log"][39] = 89.0, 200.0
    d = gpu(t)
    state = d["h0"].clone()
    y = ss.ss1d_scan_step(*args(d), state, z=d["z"])
    tu.check_scan(t, y, state, None)


def test_wide_strides_of_one_token_and_of_one_group():
    """Time-first projections viewed batch-first, of one token; groups behind tokens, of one group."""
    B, D, N = 1100, 8192, 16
    assert B * 2 * D > 1 << 24
    gen = torch.Generator(device="cuda").manual_seed(2)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(BF16)

    u, dt = (normal(1, B, 2 * D).transpose(0, 1)[..., :D] for _ in range(2))
    Bs, Cs = (normal(B, 1, 1, N) for _ in range(2))
    par = (torch.zeros(D, N, device="cuda"), torch.ones(D, device="cuda"), torch.full((D,), -2.0, device="cuda"))

    def step(u, dt):
        state = torch.zeros(B, D, N, device="cuda")
        return ss.ss1d_scan_step(u, dt, par[0], Bs, Cs, par[1], par[2], state), state

    for got, want in zip(step(u, dt), step(u.contiguous(), dt.contiguous())):
        assert torch.equal(got, want)
    L, W, D = 20, 1 << 20, 40
    wide = normal(1, 1, L, W).transpose(1, 2)  # group stride L W, token stride W
    u, dt = (normal(1, L, D) for _ in range(2))
    par = (torch.zeros(D, N, device="cuda"), torch.ones(D, device="cuda"), torch.full((D,), -2.0, device="cuda"))
    assert wide.stride(2) > 1 << 24

    def both(Bs, Cs):
        a = (u, dt, par[0], Bs, Cs, par[1], par[2])
        return [ss.ss1d_scan_forward(*a)] + list(ss.ss1d_scan_backward(*a, u).values())

    views = wide[..., :N], wide[..., N:2 * N]
    for got, want in zip(both(*views), both(*[v.contiguous() for v in views])):
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_group_statistics_without_positions(dtype):
    for shape, G, eps in (((2, 0, 8), 2, 1e-5), ((3, 5, 0, 33), 33, 0.25), ((1, 0, 4096), 1, 1e-3), ((0, 4, 8), 2, 1e-5)):
        torch.full((1 << 18,), 7.0, device="cuda")  # what the allocator hands out next
        y, stats = ss.ss2d_group_norm_forward(torch.zeros(shape, device="cuda", dtype=dtype), G, eps=eps, stats=True)
        assert y.shape == shape and stats.shape == (shape[0], G, 2)
        assert not stats[..., 0].any()
        assert torch.allclose(stats[..., 1], torch.full_like(stats[..., 1], eps ** -0.5), rtol=4 * su.F32_HALF)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("cu", [None, [0, 2, 2, 5]])
def test_gradients_without_channels(cu, dtype):
    """dBs and dCs are sums over the channels, of which there may be none."""
    B, S = (2, 2) if cu is None else (1, 3)
    u, bc = torch.zeros(B, 5, 0, device="cuda", dtype=dtype), torch.ones(B, 5, 2, 16, device="cuda", dtype=dtype)
    none, A = torch.zeros(0, device="cuda"), torch.zeros(0, 16, device="cuda")
    at = torch.tensor(cu, dtype=torch.int32, device="cuda") if cu else None
    for z, h0 in ((None, None), (u, torch.zeros(S, 0, 16, device="cuda"))):
        kw = dict(z=z, initial_state=h0, cu_seqlens=at)
        y, saved = ss.ss1d_scan_forward_save(u, u, A, bc, bc, none, none, **kw)
        assert y.shape == u.shape
        for kept in (saved, None):
            torch.full((1 << 18,), 7.0, device="cuda")  # what the allocator hands out next
            d = ss.ss1d_scan_backward(u, u, A, bc, bc, none, none, u, saved=kept, **kw)
            assert d["Bs"].shape == bc.shape and not d["Bs"].any() and not d["Cs"].any()
            assert d["u"].shape == u.shape and d["A_log"].shape == A.shape


def test_scan_of_more_states_than_threads_of_a_launch():
    """70,000 sequences of 4096 channels of 16 states, which nothing joins: each is that of a call of few."""
    B, L, D, N = 70000, 2, 4096, 16
    assert B * D * N > 1 << 32
    gen = torch.Generator(device="cuda").manual_seed(4)
    u, dt = (torch.randn(B, L, D, generator=gen, device="cuda", dtype=BF16) for _ in range(2))
    Bs, Cs = (torch.randn(B, L, 1, N, generator=gen, device="cuda", dtype=BF16) for _ in range(2))
    par = (torch.zeros(D, N, device="cuda"), torch.ones(D, device="cuda"), torch.full((D,), -2.0, device="cuda"))

    def run(rows, lanes):
        with su.plan(-1, lanes):
            return ss.ss1d_scan_forward(u[rows], dt[rows], par[0], Bs[rows], Cs[rows], par[1], par[2], final_state=True)

    y, end = run(slice(0, B), 0)
    for rows in (slice(0, 3), slice(B - 3, B), slice(B // 2, B // 2 + 3)):
        want, state = run(rows, 4)
        assert torch.equal(y[rows], want) and torch.equal(end[rows], state)
    del end

    def back(rows):
        return ss.ss1d_scan_backward(u[rows], dt[rows], par[0], Bs[rows], Cs[rows], par[1], par[2], y[rows])

    got = back(slice(0, B))
    for rows in (slice(0, 3), slice(B - 3, B)):
        want = back(rows)
        for n in ("u", "dt_raw", "Bs", "Cs"):
            assert torch.equal(got[n][rows], want[n]), n
    # dDs in 64 bits, by parts; sums of 140,000 terms of both signs in fp32
    ref = sum((y[i:i + 1000].double() * u[i:i + 1000].double()).sum((0, 1)) for i in range(0, B, 1000))
    mag = sum((y[i:i + 1000].double() * u[i:i + 1000].double()).abs().sum((0, 1)) for i in range(0, B, 1000))
    assert float((got["Ds"] - ref).norm()) <= 16 * su.F32_HALF * float(mag.norm()) <= 1e-3 * float(ref.norm())


@pytest.mark.parametrize("B, D, KW, dtype", [(3, 5, 4, F32), (2, 7, 2, BF16), (80000, 8192, 8, BF16)])
def test_conv_states_of_rows_without_tokens(B, D, KW, dtype):
    """The states, and back their gradients, pass through, more than 2^33 bytes of them as well."""
    state = torch.randn(B, KW - 1, D, device="cuda", dtype=dtype)
    x, w = torch.zeros(B, 0, D, device="cuda", dtype=dtype), torch.ones(D, KW, device="cuda")
    y, end = ss.ss1d_conv_forward(x, w, initial_state=state, final_state=True)
    assert y.shape == x.shape and torch.equal(end, state)
    del end
    d = ss.ss1d_conv_backward(x, w, x, initial_state=state, dstate=state)
    assert torch.equal(d["initial_state"], state) and not d["conv_w"].any()
    del d
    assert not ss.ss1d_conv_forward(x, w, final_state=True)[1].any()


@pytest.mark.parametrize("channel", [3, 69])
@pytest.mark.parametrize("seg", [0, 16])
def test_nan_in_u_reaches_no_other_gradient(channel, seg):
    """What does not read u of that token and channel, or the states behind it, is as without the NaN: the
    last channel's too, whose values idle lanes copy."""
    t = gpu(su.make_inputs(2, 60, 70, 1, 16, F32, seed=4))

    def both():
        with su.plan(seg):
            _, saved = ss.ss1d_scan_forward_save(*args(t), z=t["z"])
            return ss.ss1d_scan_backward(*args(t), t["dy"], z=t["z"], saved=saved)

    clean = both()
    t["u"][1, 30, channel] = float("nan")
    got = both()
    rest = [i for i in range(70) if i != channel]
    for n in ("u", "dt_raw", "z"):
        assert torch.equal(got[n][0], clean[n][0]) and torch.equal(got[n][1][:, rest], clean[n][1][:, rest]), n
        assert torch.equal(got[n][1, :30], clean[n][1, :30]), n
    assert torch.equal(got["u"], clean["u"])  # the adjoint does not read the states
    for n in ("A_log", "Ds", "dt_bias"):
        assert torch.equal(got[n][rest], clean[n][rest]), n
    for n in ("Bs", "Cs"):
        assert torch.equal(got[n][0], clean[n][0]) and torch.equal(got[n][1, :30], clean[n][1, :30]), n
    assert torch.equal(got["Bs"][1, 31:], clean["Bs"][1, 31:])
    assert got["Bs"][1, 30].isnan().all() and got["Cs"][1, 30:].isnan().all() and got["z"][1, 30:, channel].isnan().all()
