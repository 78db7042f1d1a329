"""NaN and infinities inside the gated delta rule's sequences: what the definition makes NaN or
infinite is so, and nothing else is."""
import math

import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import delta_util as du

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]
BAD = [("g", math.nan), ("g", math.inf), ("beta", math.nan), ("beta", -math.inf), ("k", math.nan),
       ("k", math.inf), ("v", math.nan), ("v", -math.inf), ("q", math.nan)]


def planted(t, name, value, b, token, head):
    """A copy with one value of token `token`, head `head` (q, k: its key head) of row b replaced."""
    m = dict(t)
    x = t[name].clone()
    if name in ("q", "k"):
        head //= t["v"].shape[2] // t["q"].shape[2]
    x[(b, token, head) if name in ("g", "beta") else (b, token, head, 5)] = value
    m[name] = x
    return m


def forward(t, scale=0.6, **kw):
    d = du.to_gpu(t)
    return ss.ss1d_delta_forward(*[d[n] for n in du.NAMES], scale=scale, initial_state=d["h0"],
                                 final_state=True, **kw)


def check_like(got, ref, clean, what, tol, rel):
    """got is finite exactly where the definition is, near it there; what the planted value
    does not reach in the definition (equal to the clean one) has the clean run's bits."""
    got = got.double().cpu()
    fine = torch.isfinite(ref)
    wrong = fine != torch.isfinite(got)
    assert not wrong.any(), f"{what}: finite or not unlike the definition at {wrong.nonzero()[:3].tolist()}"
    if clean is not None:
        assert torch.equal(got[fine], clean.double().cpu()[fine]), f"{what}: unreached values changed"
    big = ref[fine].abs().max() if fine.any() else torch.tensor(1.0)
    over = (got[fine] - ref[fine]).abs() - rel * ref[fine].abs() - tol(big)
    assert not fine.any() or float(over.max()) <= 0, what


def check_forward(t, dtype, got, clean, cu=None):
    ref_o, ref_s = du.reference(t, 0.6, cu)
    DK = t["q"].shape[3]
    check_like(got[0], ref_o, clean[0], "o", lambda big: du.o_bounds(DK, big, dtype)[0],
               du.o_bounds(DK, ref_o, dtype)[1])
    check_like(got[1], ref_s, clean[1], "end states", lambda big: du.f32_bound(DK, big), 0.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name, value", BAD)
@pytest.mark.parametrize("chunks", [0, 2])
def test_forward_hides_nothing(name, value, chunks, dtype):
    """What the definition makes NaN or infinite is so; other rows and key heads keep their bits."""
    t = du.make_inputs(2, 200, 2, 4, 64, 48, dtype, seed=2, h0=2)
    m = planted(t, name, value, 1, 100, 2)
    ref_o, ref_s = du.reference(m, 0.6)
    with du.segments(chunks):
        got, clean = forward(m), forward(t)
    for x, c, ref in zip(got, clean, (ref_o, ref_s)):
        assert not torch.isfinite(x.cpu())[~torch.isfinite(ref)].any()
        assert torch.equal(x[0], c[0])
    assert torch.equal(got[0][1, :, :2], clean[0][1, :, :2]) and torch.equal(got[1][1, :2], clean[1][1, :2])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name, value", BAD)
@pytest.mark.parametrize("token", [0, 31, 32, 45, 99])
def test_forward_only_later_tokens(name, value, token, dtype):
    """One bad value: the tokens before it, other rows, other heads and (for v) other columns
    keep their bits."""
    t = du.make_inputs(2, 100, 2, 4, 64, 48, dtype, seed=token, h0=2)
    m = planted(t, name, value, 1, token, 2)
    check_forward(m, dtype, forward(m), forward(t))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name, value", BAD)
@pytest.mark.parametrize("shape", [(1, 70, 1, 1, 16, 31), (1, 70, 1, 2, 128, 100), (1, 40, 1, 1, 33, 160)])
def test_forward_of_other_widths(shape, name, value, dtype):
    t = du.make_inputs(*shape, dtype, seed=3)
    m = planted(t, name, value, 0, 37, 0)
    check_forward(m, dtype, forward(m), forward(t))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name, value", BAD)
def test_forward_in_segments(name, value, dtype):
    t = du.make_inputs(1, 300, 1, 2, 64, 64, dtype, seed=4, h0=1)
    m = planted(t, name, value, 0, 150, 1)
    with du.segments(2):
        check_forward(m, dtype, forward(m), forward(t))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name, value", BAD)
def test_other_packed_sequences_keep_their_bits(name, value, dtype):
    cu = torch.tensor([0, 20, 75, 90], dtype=torch.int32)
    t = du.make_inputs(1, 90, 1, 2, 64, 64, dtype, seed=5, h0=3)
    m = planted(t, name, value, 0, 41, 1)
    check_forward(m, dtype, forward(m, cu_seqlens=cu.cuda()), forward(t, cu_seqlens=cu.cuda()), cu)


@pytest.mark.parametrize("dtype", TYPES)
def test_padding_behind_a_row(dtype):
    """A padded batch: rows whose ends hold NaN in all inputs."""
    lens = [70, 100, 1, 33]
    t = du.make_inputs(4, 100, 1, 2, 64, 64, dtype, seed=6)
    m = {n: t[n].clone() if t[n] is not None else None for n in t}
    for b, n in enumerate(lens):
        for name in du.NAMES:
            m[name][b, n:] = math.nan
    o, _ = forward(m)
    clean, _ = forward(t)
    for b, n in enumerate(lens):
        assert torch.equal(o[b, :n], clean[b, :n]), b
        assert torch.isnan(o[b, n:]).all(), b


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name, value", BAD)
def test_training_forward(name, value, dtype):
    t = du.make_inputs(1, 100, 1, 2, 64, 48, dtype, seed=9, h0=1)

    def run(x):
        d = du.to_gpu(x)
        return ss.ss1d_delta_forward_save(*[d[n] for n in du.NAMES], scale=0.6, final_state=True,
                                          initial_state=d["h0"])[:2]

    m = planted(t, name, value, 0, 45, 1)
    check_forward(m, dtype, run(m), run(t))


@pytest.mark.parametrize("dtype", TYPES)
def test_sums_past_the_largest_value(dtype):
    """Finite inputs whose products overflow from token 40 on reach no token before it."""
    t = du.make_inputs(1, 100, 1, 1, 64, 64, dtype, seed=10)
    m = {n: t[n].clone() if t[n] is not None else None for n in t}
    m["k"][0, 40:44] *= 2.0 ** 100
    m["v"][0, 50] *= 2.0 ** 126
    got, clean = forward(m), forward(t)
    assert torch.equal(got[0][0, :40], clean[0][0, :40])
    assert not torch.isfinite(got[0][0, 60:]).any() and not torch.isfinite(got[1]).any()


def test_the_largest_values_are_values():
    """fp32 values up to the largest one are neither cut nor taken for infinite: exact here, one token
    at a time with orthogonal keys."""
    big = torch.finfo(torch.float32).max
    t = du.make_inputs(1, 3, 1, 1, 8, 32, torch.float32, seed=11, decay=0.0)
    for n in ("q", "k"):
        t[n] = torch.eye(8)[None, :3, None].clone()
    t["beta"][:] = 1.0
    t["v"][0, 1, 0, 3], t["v"][0, 2, 0, 4] = big, -big
    o, end = forward(t, scale=1.0)
    assert torch.equal(o.cpu(), t["v"])
    assert torch.equal(end.cpu()[0, 0, :3], t["v"][0, :, 0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name, value", BAD)
def test_step(name, value, dtype):
    """The form for single tokens: the same definition, its 3 tokens in order."""
    t = du.make_inputs(2, 3, 2, 4, 64, 48, dtype, seed=7, h0=2)

    def run(x):
        d = du.to_gpu(x)
        return ss.ss1d_delta_step(*[d[n] for n in du.NAMES], d["h0"], scale=0.6), d["h0"]

    m = planted(t, name, value, 1, 1, 2)
    check_forward(m, dtype, run(m), run(t))


def backward(t, keep, cu=None):
    d = du.to_gpu(t)
    args, saved = [d[n] for n in du.NAMES], None
    kw = dict(scale=0.6, initial_state=d["h0"], cu_seqlens=cu.cuda() if cu is not None else None)
    if keep:
        _, saved = ss.ss1d_delta_forward_save(*args, **kw)
    return ss.ss1d_delta_backward(*args, d["do"], saved=saved, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name, value", BAD + [("do", math.nan)])
@pytest.mark.parametrize("keep", [True, False])
def test_backward_hides_nothing(name, value, keep, dtype):
    """What the definition's adjoint makes NaN or infinite is so; other rows and key heads keep
    their bits, and so does what it leaves finite outside of the bad token's block of 64."""
    t = du.make_inputs(2, 200, 2, 4, 64, 48, dtype, seed=8, h0=2)
    m = planted(t, name, value, 1, 100, 2)
    got, clean = backward(m, keep), backward(t, keep)
    ref, ref0 = du.adjoint(m, 0.6)
    for n in du.NAMES:
        x, c = got[n].cpu(), clean[n].cpu()
        fine = torch.isfinite(ref[n])
        assert not torch.isfinite(x)[~fine].any(), f"d{n} hides it"
        assert torch.equal(x[0], c[0]), n
        other = slice(0, 2) if n not in ("q", "k") else slice(0, 1)
        assert torch.equal(x[1][:, other], c[1][:, other]), n
        block = torch.zeros_like(fine)
        block[1, 64:128] = True
        assert torch.isfinite(x)[fine & ~block].all(), f"d{n} outside of the block"
    assert not torch.isfinite(got["initial_state"].cpu())[~torch.isfinite(ref0)].any()
    assert torch.equal(got["initial_state"][0], clean["initial_state"][0])
