"""How the gated delta rule and the block norm are called."""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import delta_util as du

pytestmark = pytest.mark.gpu


def norm_inputs(seed=0, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = {n: torch.randn(40, 96, generator=gen, device="cuda").to(dtype) for n in
         ("h", "z", "residual", "dy", "dn")}
    t.update({n: torch.randn(96, generator=gen, device="cuda") for n in ("w_post", "w_pre", "res_scale")})
    return t


def norm_forward(t, **kw):
    return ss.ss2d_norm_forward(t["h"], residual=t["residual"], z=t["z"], w_post=t["w_post"],
                                w_pre=t["w_pre"], res_scale=t["res_scale"], **kw)


def norm_backward(t, y, **kw):
    return ss.ss2d_norm_backward(t["h"], y, t["dy"], t["dn"], z=t["z"], w_post=t["w_post"],
                                 w_pre=t["w_pre"], res_scale=t["res_scale"], **kw)


def test_every_given_tensor_is_recorded_on_the_calls_stream(monkeypatch):
    """With stream= the caller's tensors, the outputs that it gives among them, are kept from
    reuse until the call has run."""
    seen = set()
    record = torch.Tensor.record_stream

    def spy(self, stream):
        seen.add((self.data_ptr(), stream.cuda_stream))
        record(self, stream)

    monkeypatch.setattr(torch.Tensor, "record_stream", spy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def check(*tensors):
        torch.cuda.synchronize()
        for i, x in enumerate(tensors):
            assert (x.data_ptr(), s.cuda_stream) in seen, i
        seen.clear()

    t = norm_inputs()
    y, n = torch.empty_like(t["h"]), torch.empty_like(t["h"])
    norm_forward(t, y=y, n=n, stream=s)
    check(*[x for k, x in t.items() if k not in ("dy", "dn")], y, n)
    norm_backward(t, y, stream=s)
    check(*[x for k, x in t.items() if k != "residual"], y)
    d = du.to_gpu(du.make_inputs(1, 40, 1, 2, 64, 64, torch.bfloat16, h0=1))
    seq = [d[x] for x in du.NAMES]
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    o, end = torch.empty_like(d["v"]), torch.empty_like(d["h0"])
    ss.ss1d_delta_forward(*seq, cu_seqlens=cu, initial_state=d["h0"], final_state=end, o=o, stream=s)
    check(*seq, cu, d["h0"], end, o)
    _, _, saved = ss.ss1d_delta_forward_save(*seq, final_state=end, o=o, stream=s)
    check(*seq, end, o)
    ss.ss1d_delta_backward(*seq, d["do"], dstate=end, saved=saved, stream=s)
    check(*seq, d["do"], end, saved)
    slots = torch.zeros(1, dtype=torch.int32, device="cuda")
    ss.ss1d_delta_step(*[x[:, :1].contiguous() for x in seq], end, slots=slots, o=o[:, :1].contiguous(), stream=s)
    assert {(x.data_ptr(), s.cuda_stream) for x in (end, slots)} <= seen


@pytest.mark.parametrize("chunks", [-1, 0, 2])
@pytest.mark.parametrize("packed", [False, True])
def test_rows_without_tokens(packed, chunks):
    """No token at all, in whole sequences and in segments: the states pass through."""
    t = du.to_gpu(du.make_inputs(1 if packed else 3, 0, 1, 2, 64, 48, torch.float32, h0=3))
    seq = [t[n] for n in du.NAMES]
    kw = dict(initial_state=t["h0"])
    if packed:
        kw["cu_seqlens"] = torch.zeros(4, dtype=torch.int32, device="cuda")
    with du.segments(chunks):
        o, end = ss.ss1d_delta_forward(*seq, final_state=True, **kw)
        assert o.shape == t["v"].shape and torch.equal(end, t["h0"])
        o, end, saved = ss.ss1d_delta_forward_save(*seq, final_state=True, **kw)
        assert torch.equal(end, t["h0"])
        g = torch.randn_like(end)
        for kept in (saved, None):
            d = ss.ss1d_delta_backward(*seq, t["do"], dstate=g, saved=kept, **kw)
            assert torch.equal(d["initial_state"], g) and d["v"].shape == t["v"].shape


def test_a_second_output_without_its_norm_is_refused():
    t = norm_inputs()
    with pytest.raises(ValueError, match="n needs w_pre"):
        ss.ss2d_norm_forward(t["h"], residual=t["residual"], n=torch.empty_like(t["h"]))
