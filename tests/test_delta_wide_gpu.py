"""The gated delta rule with values wider than 128: several blocks of columns per head."""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import delta_util as du
from tests.test_delta_backward_gpu import check_grads

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16]
SHAPES = [(1, 100, 1, 2, 64, 160), (2, 70, 1, 1, 128, 192), (1, 130, 1, 1, 32, 257), (1, 200, 1, 3, 96, 130)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("chunks", [-1, 2])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, chunks, dtype):
    B, L, HK, H, DK, DV = shape
    t = du.make_inputs(*shape, dtype, seed=DV, h0=B)
    dstate = 0.1 * torch.randn(B, H, DK, DV, generator=torch.Generator().manual_seed(1))
    d = du.to_gpu(t)
    args, scale = [d[n] for n in du.NAMES], DK ** -0.5
    with du.segments(chunks):
        o, end, saved = ss.ss1d_delta_forward_save(*args, initial_state=d["h0"], final_state=True)
        p, pend = ss.ss1d_delta_forward(*args, initial_state=d["h0"], final_state=True)
        got = ss.ss1d_delta_backward(*args, d["do"], initial_state=d["h0"], dstate=dstate.cuda(), saved=saved)
    ref_o, ref_s = du.reference(t, scale)
    for x in (o, p):
        du.check(x, ref_o, "o", *du.o_bounds(DK, ref_o, dtype))
    for x in (end, pend):
        du.check(x, ref_s, "end states", du.f32_bound(DK, ref_s))
    check_grads(t, got, dtype, scale, dstate=dstate)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("DV", [160, 257])
def test_step(DV, dtype):
    t = du.make_inputs(3, 2, 1, 2, 100, DV, dtype, seed=DV, h0=3)
    d = du.to_gpu(t)
    o = ss.ss1d_delta_step(*[d[n] for n in du.NAMES], d["h0"])
    ref_o, ref_s = du.reference(t, 0.1)
    du.check(o, ref_o, "o", du.f32_bound(100, ref_o), du.BF16_HALF if dtype == torch.bfloat16 else 0.0)
    du.check(d["h0"], ref_s, "state", du.f32_bound(100, ref_s))


@pytest.mark.parametrize("dtype", TYPES)
def test_packed_training_with_shared_heads_of_128(dtype):
    lens = [0, 40, 1, 150, 64]
    cu = torch.tensor([2] + [0] * len(lens), dtype=torch.int32)
    for i, n in enumerate(lens):
        cu[i + 1] = cu[i] + n
    t = du.make_inputs(1, int(cu[-1]) + 3, 2, 4, 128, 128, dtype, seed=8, h0=len(lens))
    d = du.to_gpu(t)
    args = [d[n] for n in du.NAMES]
    kw = dict(scale=0.1, cu_seqlens=cu.cuda(), initial_state=d["h0"])
    _, saved = ss.ss1d_delta_forward_save(*args, **kw)
    check_grads(t, ss.ss1d_delta_backward(*args, d["do"], saved=saved, **kw), dtype, 0.1, cu)
