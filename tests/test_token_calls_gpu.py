"""How the token-order scan, its convolution and the group norm are called: streams, threads, captured
graphs, tensors past 2^31 elements; and a block of them together."""
import threading

import pytest
import torch

import selective_scan_ss2d_amd as ss
from selective_scan_ss2d_amd import _binding as bnd
from tests import scan_util as su
from tests.test_scan_gpu import args, gpu
from tests.test_sequence_calls_gpu import node_types

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def inputs(seed, L=150, dtype=BF16):
    """Packed sequences of the scan and the convolution, and a map of the group norm."""
    t = gpu(su.make_inputs(1, L, 96, 2, 16, dtype, seed=seed, h0=3))
    t.update({"c_" + n: v.cuda() for n, v in su.conv_inputs(1, L, 96, 4, dtype, seed=seed, h0=3).items()})
    t["cu"] = torch.tensor([0, L // 3, L // 2, L - 10], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t["map"], t["dmap"], t["long"] = (torch.randn(shape, generator=gen, device="cuda").to(dtype)
                                      for shape in ((2, 9, 9, 96), (2, 9, 9, 96), (1, 30000, 8)))
    t["w"], t["b"] = (torch.rand(96, generator=gen, device="cuda") for _ in range(2))
    return t


def everything(t, stream=None):
    """One call of every entry point; the outputs."""
    kw = dict(stream=stream)
    packed = dict(z=t["z"], cu_seqlens=t["cu"], initial_state=t["h0"], **kw)
    # (tokens outside of the packed sequences are left as they are in a given y)
    y, end = ss.ss1d_scan_forward(*args(t), final_state=True, y=torch.zeros_like(t["u"]), **packed)
    y2, saved = ss.ss1d_scan_forward_save(*args(t), y=torch.zeros_like(t["u"]), **packed)
    out = [y, end, y2]
    with su.plan(32):
        out += list(ss.ss1d_scan_forward(*args(t), final_state=True, y=torch.zeros_like(y), **packed))
        out += list(ss.ss1d_scan_backward(*args(t), t["dy"], dstate=t["dht"], saved=saved, **packed).values())
    out += list(ss.ss1d_scan_backward(*args(t), t["dy"], **packed).values())
    one = [t[n][:, :1].contiguous() if n in ("u", "dt_raw", "Bs", "Cs") else t[n] for n in su.NAMES]
    state, slot = t["h0"].clone(), torch.ones(1, dtype=torch.int32, device="cuda")
    out += [ss.ss1d_scan_step(*one, state, z=t["z"][:, :1].contiguous(), slots=slot, **kw), state]
    conv = dict(cu_seqlens=t["cu"], initial_state=t["c_h0"], **kw)
    x, w, b = t["c_x"], t["c_conv_w"], t["c_conv_b"]
    out += list(ss.ss1d_conv_forward(x, w, b, final_state=True, y=torch.zeros_like(x), **conv))
    out += list(ss.ss1d_conv_backward(x, w, t["c_dy"], b, dstate=t["c_dht"], **conv).values())
    held = t["c_h0"].clone()
    out += [ss.ss1d_conv_step(x[:, :2].contiguous(), w, held, b, slots=slot, **kw), held]
    aff = dict(weight=t["w"], bias=t["b"], **kw)
    y, stats = ss.ss2d_group_norm_forward(t["map"], 8, stats=True, **aff)
    out += [y, stats] + list(ss.ss2d_group_norm_backward(t["map"], t["dmap"], 8, stats=stats, **aff).values())
    out += list(ss.ss2d_group_norm_backward(t["map"], t["dmap"], 8, **aff).values())
    out += [ss.ss2d_group_norm_forward(t["long"], 1, **kw)]  # by chunks
    out += list(ss.ss2d_group_norm_backward(t["long"], t["long"], 1, **kw).values())
    return out


def on_stream(t, stream):
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):  # the clones and zeros that the calls are given
        out = everything(t, stream)
    stream.synchronize()
    return out


def same(a, b):
    assert len(a) == len(b)
    for i, (x, y) in enumerate(zip(a, b)):
        assert torch.equal(x, y), i


def test_every_call_on_a_given_stream():
    t = inputs(1)
    want = everything(t)
    torch.cuda.synchronize()
    for _ in range(3):
        same(on_stream(t, torch.cuda.Stream()), want)


def test_results_repeat():
    t = inputs(2, dtype=F32)
    want = everything(t)
    for _ in range(3):
        same(everything(t), want)


def test_calls_from_several_threads():
    """Each thread on a stream of its own, at once."""
    ts = [inputs(i) for i in range(4)]
    want = [everything(t) for t in ts]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        stream = torch.cuda.Stream()
        for _ in range(4):
            out = on_stream(ts[i], stream)
            if not all(torch.equal(a, b) for a, b in zip(out, want[i])):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not bad


def test_every_given_tensor_is_recorded_on_the_calls_stream(monkeypatch):
    seen = set()
    record = torch.Tensor.record_stream

    def spy(self, stream):
        seen.add((self.data_ptr(), stream.cuda_stream))
        record(self, stream)

    t = inputs(3)
    monkeypatch.setattr(torch.Tensor, "record_stream", spy)
    s = torch.cuda.Stream()
    on_stream(t, s)
    steps = ("u", "dt_raw", "Bs", "Cs", "z")  # steps are given copies of these as well
    for n, x in t.items():
        assert (x.data_ptr(), s.cuda_stream) in seen, n
    assert len(steps) < len(seen)


def captured(t, stream):
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        everything(t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph, stream=stream):
        out = everything(t)
    return graph, out


def test_a_captured_call_holds_kernels_and_replays():
    t = inputs(4)
    graph, out = captured(t, torch.cuda.Stream())
    types = node_types(graph)
    # clones of the states are copies between device tensors, which torch records as such
    assert len(types) > 40 and types.count(0) >= len(types) - 2
    graph.instantiate()
    for i in range(4):
        for n in ("u", "c_x", "map"):
            t[n].normal_()
        want = [x.clone() for x in everything(t)]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        same(out, want)


def test_c_calls_without_scratch_are_refused_under_capture():
    lib = bnd.load_library()
    t = gpu(su.make_inputs(1, 2048, 64, 1, 16, BF16, seed=1))
    p = [t[n].data_ptr() for n in su.NAMES]
    y = torch.empty_like(t["u"])
    g = [torch.empty_like(t[n]) for n in su.NAMES]
    c = su.conv_inputs(1, 64, 64, 4, BF16, device="cuda")
    dx, dw, db = (torch.empty_like(c[n]) for n in ("x", "conv_w", "conv_b"))
    stream, x = torch.cuda.Stream(), torch.zeros(8, device="cuda")
    sizes = (1, 2048, 1, 64, 1, 16)
    assert lib.ss1d_scan_scratch_bytes(0, 0, *sizes, 1, 0) > 0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s = stream.cuda_stream
        codes = [lib.ss1d_scan_forward(*p, None, None, None, y.data_ptr(), None, None, None, 0, *sizes, None, 1, s),
                 lib.ss1d_scan_backward(*p, None, None, None, None, t["dy"].data_ptr(), None, g[0].data_ptr(),
                                        g[1].data_ptr(), g[2].data_ptr(), g[3].data_ptr(), g[4].data_ptr(),
                                        g[5].data_ptr(), g[6].data_ptr(), None, None, None, 0, *sizes, None, 1, s),
                 lib.ss1d_conv_backward(c["x"].data_ptr(), c["conv_w"].data_ptr(), c["conv_b"].data_ptr(), None, None,
                                        c["dy"].data_ptr(), None, dx.data_ptr(), dw.data_ptr(), db.data_ptr(), None,
                                        None, 0, 1, 64, 1, 64, 4, None, 1, 1, s),
                 lib.ss2d_group_norm_backward(c["x"].data_ptr(), None, None, None, c["dy"].data_ptr(), dx.data_ptr(),
                                              None, None, None, 0, 1, 64, 64, 4, 1, 1e-5, 1, s)]
        x.add_(1)
    assert codes == [bnd.SS2D_ERR_SCRATCH] * 4
    graph.replay()
    torch.cuda.synchronize()
    assert (x == 1).all()


def test_c_calls_with_the_librarys_scratch():
    """The C entry points without scratch of the caller's: the same bits."""
    lib = bnd.load_library()
    t = gpu(su.make_inputs(1, 2048, 64, 1, 16, BF16, seed=1))
    p, s = [t[n].data_ptr() for n in su.NAMES], torch.cuda.current_stream().cuda_stream
    sizes = (1, 2048, 1, 64, 1, 16)
    y = torch.empty_like(t["u"])
    g = {n: torch.empty_like(t[n]) for n in su.NAMES}
    assert lib.ss1d_scan_forward(*p, None, None, None, y.data_ptr(), None, None, None, 0, *sizes, None, 1, s) == 0
    assert lib.ss1d_scan_backward(*p, None, None, None, None, t["dy"].data_ptr(), None,
                                  *[g[n].data_ptr() for n in su.NAMES], None, None, None, 0, *sizes, None, 1, s) == 0
    assert torch.equal(y, ss.ss1d_scan_forward(*args(t)))
    for n, x in ss.ss1d_scan_backward(*args(t), t["dy"]).items():
        assert torch.equal(g[n], x), n
    c = su.conv_inputs(1, 64, 64, 4, BF16, device="cuda")
    dx, dw, db = (torch.empty_like(c[n]) for n in ("x", "conv_w", "conv_b"))
    assert lib.ss1d_conv_backward(c["x"].data_ptr(), c["conv_w"].data_ptr(), c["conv_b"].data_ptr(), None, None,
                                  c["dy"].data_ptr(), None, dx.data_ptr(), dw.data_ptr(), db.data_ptr(), None, None, 0,
                                  1, 64, 1, 64, 4, None, 1, 1, s) == 0
    want = ss.ss1d_conv_backward(c["x"], c["conv_w"], c["dy"], c["conv_b"])
    assert torch.equal(dx, want["x"]) and torch.equal(dw, want["conv_w"]) and torch.equal(db, want["conv_b"])


def test_scan_past_32_bit_elements():
    """u, y and their gradients of 2.2e9 elements: the last sequences are those of a small call."""
    L, S, D, N, last = 600, 900, 4096, 4, 2
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=BF16)

    u, dt, dy = (normal(1, L * S, D) for _ in range(3))
    Bs, Cs = normal(1, L * S, 1, N), normal(1, L * S, 1, N)
    assert u.numel() > 1 << 31
    par = dict(A_log=torch.zeros(D, N, device="cuda"), Ds=torch.ones(D, device="cuda"),
               dt_bias=torch.full((D,), -2.0, device="cuda"))

    def run(u, dt, Bs, Cs, dy, count):
        cu = torch.arange(0, count * L + 1, L, dtype=torch.int32, device="cuda")
        a = (u, dt, par["A_log"], Bs, Cs, par["Ds"], par["dt_bias"])
        y, end, saved = ss.ss1d_scan_forward_save(*a, cu_seqlens=cu, final_state=True)
        d = ss.ss1d_scan_backward(*a, dy, cu_seqlens=cu, saved=saved)
        return [end, y, d["u"], d["dt_raw"], d["Bs"], d["Cs"]]

    with su.plan(0, 4):
        want = run(*[x[:, -last * L:].contiguous() for x in (u, dt, Bs, Cs, dy)], last)
        got = run(u, dt, Bs, Cs, dy, S)
    assert torch.equal(got[0][-last:], want[0])
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a[:, -last * L:], b)


def test_steps_past_32_bit_elements():
    D, N, slots, KW = 8192, 32, 8300, 8
    t = gpu(su.make_inputs(3, 1, D, 1, N, BF16, seed=4, h0=3))
    state = torch.zeros(slots, D, N, device="cuda")
    assert state.numel() > 1 << 31
    at = torch.tensor([slots - 1, 0, slots - 70], dtype=torch.int32, device="cuda")
    state[at.long()] = t["h0"]
    y = ss.ss1d_scan_step(*args(t), state, z=t["z"], slots=at)
    want = ss.ss1d_scan_step(*args(t), t["h0"], z=t["z"])
    assert torch.equal(y, want) and torch.equal(state[at.long()], t["h0"])
    assert not state[1:slots - 70].any()
    del state
    c = {n: x.cuda() for n, x in su.conv_inputs(3, 1, D, KW, BF16, seed=4, h0=3).items()}
    held = torch.zeros(40000, KW - 1, D, device="cuda", dtype=BF16)
    assert held.numel() > 1 << 31
    at = torch.tensor([39999, 0, 39000], dtype=torch.int32, device="cuda")
    held[at.long()] = c["h0"]
    y = ss.ss1d_conv_step(c["x"], c["conv_w"], held, c["conv_b"], slots=at)
    want = ss.ss1d_conv_step(c["x"], c["conv_w"], c["h0"], c["conv_b"])
    assert torch.equal(y, want) and torch.equal(held[at.long()], c["h0"])


def test_conv_past_32_bit_elements():
    L, B, D, last = 700, 800, 4096, 2
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.randn(B, L, D, generator=gen, device="cuda", dtype=BF16) for _ in range(2))
    assert x.numel() > 1 << 31
    w, b = torch.randn(D, 4, generator=gen, device="cuda"), torch.randn(D, generator=gen, device="cuda")

    def run(x, dy):
        y, end = ss.ss1d_conv_forward(x, w, b, final_state=True)
        return y, end, ss.ss1d_conv_backward(x, w, dy, b)["x"]

    for a, want in zip(run(x, dy), run(x[-last:].clone(), dy[-last:].clone())):
        assert torch.equal(a[-last:], want)


@pytest.mark.parametrize("shape, G", [((700, 800, 4096), 512), ((2, 70000, 16384), 16)])
def test_group_norm_past_32_bit_elements(shape, G):
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, dy = (torch.randn(shape, generator=gen, device="cuda", dtype=BF16) for _ in range(2))
    assert x.numel() > 1 << 31
    y = ss.ss2d_group_norm_forward(x, G)
    d = ss.ss2d_group_norm_backward(x, dy, G)["x"]
    few = [x[-1:].clone(), dy[-1:].clone()]
    want, dwant = ss.ss2d_group_norm_forward(few[0], G), ss.ss2d_group_norm_backward(*few, G)["x"]
    # one image may be cut otherwise than many: half a step of each, and some of the statistics' in fp32
    for a, b in ((y, want), (d, dwant)):
        err = (a[-1:].float() - b.float()).abs() - 2 * su.BF16_HALF * b.float().abs()
        assert float(err.max()) <= 1e-4


def test_steps_of_padding_alone():
    """A pool without a state: every row is padding."""
    t = gpu(su.make_inputs(3, 1, 40, 1, 16, BF16, seed=4))
    c = {n: x.cuda() for n, x in su.conv_inputs(3, 1, 40, 4, BF16, seed=4, h0=3).items()}
    slots = torch.tensor([0, -1, 5], dtype=torch.int32, device="cuda")
    y = torch.full_like(t["u"], 3.0)
    ss.ss1d_scan_step(*args(t), torch.empty(0, 40, 16, device="cuda"), slots=slots, y=y)
    ss.ss1d_conv_step(c["x"], c["conv_w"], torch.empty(0, 3, 40, device="cuda", dtype=BF16), c["conv_b"], slots=slots, y=y)
    torch.cuda.synchronize()
    assert (y == 3.0).all()


@pytest.mark.parametrize("B, L, C, G", [(400000, 1, 64, 4), (300000, 2, 24, 3), (5000, 33, 40, 40)])
def test_group_norm_of_many_images(B, L, C, G):
    """Each image's outputs and gradient are those of a call of few, up to the cut of its sums."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    x, dy = (torch.randn(B, L, C, generator=gen, device="cuda") for _ in range(2))
    w, b = torch.rand(C, generator=gen, device="cuda"), torch.rand(C, generator=gen, device="cuda")
    y = ss.ss2d_group_norm_forward(x, G, weight=w, bias=b)
    d = ss.ss2d_group_norm_backward(x, dy, G, weight=w, bias=b)
    few = [x[-7:].clone(), dy[-7:].clone()]
    want = ss.ss2d_group_norm_forward(few[0], G, weight=w, bias=b)
    dwant = ss.ss2d_group_norm_backward(*few, G, weight=w, bias=b)["x"]
    # sums of up to 64 values in another order; 1 / sqrt(var) of a group stays below 30
    for got, ref in ((y[-7:], want), (d["x"][-7:], dwant)):
        assert float((got - ref).abs().max()) <= 2e-4
    unit = ((x.double().view(B, L, G, -1) - x.double().view(B, L, G, -1).mean((1, 3), keepdim=True)))
    unit = (unit / (unit.square().mean((1, 3), keepdim=True) + 1e-5).sqrt()).view(B, L, C)
    pre = unit * w + b
    sg = torch.sigmoid(pre)
    e = dy * sg * (1 + pre * (1 - sg))
    for name, ref in (("weight", (e * unit).sum((0, 1))), ("bias", e.sum((0, 1)))):
        # pairs of sums over B images in fp32: sqrt of the count of roundings of terms of size about 1
        assert float((d[name] - ref).abs().max()) <= 4 * su.F32_HALF * B * L, name


def block(t, conv, scan):
    """The inner part of a block over tokens: the convolution, B, C and delta from its output, the scan."""
    x = conv(t["x"])
    low = x @ t["x_proj"].to(x.dtype)
    R, N = t["R"], t["N"]
    dt = low[..., :R] @ t["dt_proj"].to(x.dtype)
    Bs, Cs = (low[..., R + i * N:R + (i + 1) * N].unflatten(-1, (1, N)) for i in range(2))
    return scan(x, dt, Bs, Cs)


def block_inputs(L, D=48, N=16, R=6, seed=7):
    gen = torch.Generator().manual_seed(seed)
    t = dict(R=R, N=N, x=torch.randn(1, L, D, generator=gen), z=torch.randn(1, L, D, generator=gen),
             x_proj=torch.randn(D, R + 2 * N, generator=gen) * D ** -0.5, dt_proj=torch.randn(R, D, generator=gen) * 0.3,
             conv_w=torch.randn(D, 4, generator=gen) * 0.5, conv_b=torch.randn(D, generator=gen) * 0.1,
             A_log=torch.arange(1, N + 1).float().log().repeat(D, 1), Ds=torch.ones(D), dt_bias=torch.full((D,), -2.0))
    return t


def block_reference(t):
    d = {n: v.double().requires_grad_() if isinstance(v, torch.Tensor) else v for n, v in t.items()}

    def conv(x):
        whole = torch.cat([x.new_zeros(1, 3, x.shape[2]), x], 1)
        v = sum(whole[:, j:j + x.shape[1]] * d["conv_w"][:, j] for j in range(4)) + d["conv_b"]
        return v * torch.sigmoid(v)

    def scan(u, dt, Bs, Cs):
        delta = torch.nn.functional.softplus(dt + d["dt_bias"])
        y, _ = su.scan(u[0], delta[0], -d["A_log"].exp(), Bs[0], Cs[0], d["Ds"],
                       torch.zeros(u.shape[2], t["N"]).double())
        return y[None] * d["z"] * torch.sigmoid(d["z"])

    return block(d, conv, scan), d


def test_a_block_of_prompts_and_tokens():
    """Packed prompts through the convolution and the scan, their states handed on to steps token by
    token, against each whole sequence in 64 bits."""
    lengths, more, D, N = (20, 1, 0, 33), 3, 48, 16
    seqs = [block_inputs(n + more, seed=20) for n in lengths]
    for i, t in enumerate(seqs):
        t.update({n: v for n, v in seqs[0].items() if n not in ("x", "z")})  # one block's weights
        gen = torch.Generator().manual_seed(100 + i)
        t["x"], t["z"] = (torch.randn(t["x"].shape, generator=gen) for _ in range(2))
    ref = [block_reference(t)[0].detach() for t in seqs]
    g = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in seqs[0].items()}
    par = [g["A_log"], g["Ds"], g["dt_bias"]]
    cu = torch.tensor([0, 20, 21, 21, 54], dtype=torch.int32, device="cuda")
    g["x"], g["z"] = (torch.cat([t[n][:, :-more] for t in seqs], 1).cuda() for n in ("x", "z"))
    states = {}

    def conv(x):
        y, states["conv"] = ss.ss1d_conv_forward(x, g["conv_w"], g["conv_b"], cu_seqlens=cu, final_state=True)
        return y

    def scan(u, dt, Bs, Cs):
        y, states["scan"] = ss.ss1d_scan_forward(u, dt, par[0], Bs, Cs, par[1], par[2], z=g["z"], cu_seqlens=cu,
                                                 final_state=True)
        return y

    y = block(g, conv, scan)[0]
    outs = [[y[a:e]] for a, e in zip(cu.tolist()[:-1], cu.tolist()[1:])]
    pool, held = torch.zeros(7, D, N, device="cuda"), torch.zeros(7, 3, D, device="cuda")
    slots = torch.tensor([5, 2, 0, 6], dtype=torch.int32, device="cuda")
    pool[slots.long()], held[slots.long()] = states["scan"], states["conv"]
    for k in range(more):
        g["x"], z = (torch.cat([t[n][:, t[n].shape[1] - more + k][:, None] for t in seqs]).cuda() for n in ("x", "z"))
        y = block(g, lambda x: ss.ss1d_conv_step(x, g["conv_w"], held, g["conv_b"], slots=slots),
                  lambda u, dt, Bs, Cs: ss.ss1d_scan_step(u, dt, par[0], Bs, Cs, par[1], par[2], pool, z=z, slots=slots))
        for i in range(4):
            outs[i].append(y[i])
    for i in range(4):
        got, want = torch.cat(outs[i]).double().cpu(), ref[i][0]
        # fp32 throughout: sums of up to 48 products before the scan's own roundings
        assert float((got - want).norm() / want.norm()) <= 256 * su.F32_HALF, i


def test_gradients_of_a_block():
    """The chain of both backward passes with the projections between them, against autograd in 64 bits."""
    t = block_inputs(40)
    y64, leaves = block_reference(t)
    gen = torch.Generator().manual_seed(1)
    dy = torch.randn(y64.shape, generator=gen)
    names = ("x", "z", "conv_w", "conv_b", "x_proj", "dt_proj", "A_log", "Ds", "dt_bias")
    want = dict(zip(names, torch.autograd.grad(y64, [leaves[n] for n in names], dy.double())))
    g = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in t.items()}
    x = ss.ss1d_conv_forward(g["x"], g["conv_w"], g["conv_b"])
    low = x @ g["x_proj"]
    R, N = g["R"], g["N"]
    dt = (low[..., :R] @ g["dt_proj"]).contiguous()
    Bs, Cs = (low[..., R + i * N:R + (i + 1) * N].unflatten(-1, (1, N)) for i in range(2))
    a = (x, dt, g["A_log"], Bs, Cs, g["Ds"], g["dt_bias"])
    _, saved = ss.ss1d_scan_forward_save(*a, z=g["z"])
    d = ss.ss1d_scan_backward(*a, dy.cuda(), z=g["z"], saved=saved)
    got = {n: d[n] for n in ("z", "A_log", "Ds", "dt_bias")}
    got["dt_proj"] = low[0, :, :R].T @ d["dt_raw"][0]
    dlow = torch.cat([d["dt_raw"] @ g["dt_proj"].T, d["Bs"].flatten(2), d["Cs"].flatten(2)], -1)
    got["x_proj"] = x[0].T @ dlow[0]
    c = ss.ss1d_conv_backward(g["x"], g["conv_w"], (d["u"] + dlow @ g["x_proj"].T).contiguous(), g["conv_b"])
    got.update(x=c["x"], conv_w=c["conv_w"], conv_b=c["conv_b"])
    for n in names:
        err = float((got[n].double().cpu() - want[n]).norm() / want[n].norm())
        assert err <= 512 * su.F32_HALF, (n, err)
