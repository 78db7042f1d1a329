"""Measured cases of the token-order scan, its short causal convolution and the group norm.

``run`` computes either the plain form (elementary torch operations in 32 bits) or, with
``own`` set, the calls that a user makes of the package.

The scan keeps N states per channel d of a sequence; group g = d // (D / G) has its own B and C:
    delta = softplus(dt_raw + dt_bias),   h_n <- exp(-exp(A_log_n) delta) h_n + delta B_n u,
    y = (sum_n C_n h_n + Ds u) * SiLU(z).
The convolution, causal and per channel, with KW - 1 inputs carried from call to call:
    y_t = SiLU(conv_b + sum_j conv_w_j x_{t - KW + 1 + j}).
The group norm, over the positions and the C / G channels of a group, channels last:
    y = SiLU((x - mean) / sqrt(var + eps) * weight + bias).
"""
import math

import torch

own = False
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---- the cases ---------------------------------------------------------------------------
def listed():
    return [
        # one token of one sequence: the latency of a single reply
        dict(name="scan step, one sequence", op="scan_step", B=1, T=1, D=4096, N=16, G=1,
             slots=1, gate=True, views=True, dtype="bf16"),
        # a served batch: one token of each of 256 sequences, their states in a pool of slots
        dict(name="scan step, batch of 256", op="scan_step", B=256, T=1, D=4096, N=16, G=1,
             slots=300, gate=True, views=True, dtype="bf16"),
        # the prompt of one request, its final state handed on to the steps
        dict(name="scan prompt of 4096", op="scan", B=1, L=4096, D=4096, N=16, G=1, packed=0,
             h0=False, gate=True, views=True, dtype="bf16"),
        # prompts of odd lengths packed into one call, continuing from earlier states
        dict(name="scan packed prompts", op="scan", B=1, L=12007, D=1000, N=16, G=4, packed=25,
             h0=True, gate=True, views=True, dtype="bf16"),
        # one pass over two images of 256 x 256 positions in fp32
        dict(name="scan 256x256 image fp32", op="scan", B=2, L=65536, D=192, N=16, G=1, packed=0,
             h0=False, gate=False, views=False, dtype="f32"),
        # a training step over 8 sequences of 2048 tokens
        dict(name="scan training, 8 x 2048", op="scan_train", B=8, L=2048, D=2048, N=16, G=1,
             gate=True, views=True, dtype="bf16"),
        # the convolution of 5 drafted tokens of each of 64 sequences
        dict(name="conv step, 5 drafted tokens", op="conv_step", B=64, T=5, D=4096, KW=4,
             slots=80, views=True, dtype="bf16"),
        # the packed prompts' convolution, continuing from the inputs before them
        dict(name="conv packed prompts", op="conv", B=1, L=12007, D=4096, KW=4, packed=25,
             h0=True, views=True, dtype="bf16"),
        # the convolution of a training step over 14 * 14 + 1 tokens of 128 images, width 768
        dict(name="conv training, 197 tokens", op="conv_train", B=128, L=197, D=768, KW=4,
             views=False, dtype="bf16"),
        # one small map, where latency counts
        dict(name="group norm, 16x16 map", op="group", B=1, L=256, C=256, G=32, act=True,
             affine=True, dtype="bf16"),
        # the norm behind a convolution of the first stage: 56 x 56 maps of 192 channels
        dict(name="group norm, 56x56 maps", op="group", B=64, L=3136, C=192, G=32, act=True,
             affine=True, dtype="bf16"),
        # a training step of it on the second stage's maps, fp32
        dict(name="group norm training, 28x28", op="group_train", B=64, L=784, C=384, G=32,
             act=True, affine=True, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_step", "scan", "scan_train", "conv_step", "conv", "conv_train", "group",
                     "group_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("group", "group_train"):
        G = rng.choice([1, 2, 4, 8, 16, 32, 32])
        C = G * _log(rng, 1, max(1, 2048 // G))
        total = _log(rng, 4000, 20_000_000)
        L = max(1, min(_log(rng, 1, 70_000), total // C))
        return dict(op=op, B=max(1, min(256, total // C // L)), L=L, C=C, G=G,
                    act=rng.random() < 0.7, affine=rng.random() < 0.8, dtype=dtype)
    views = rng.random() < 0.5
    if op in ("conv_step", "conv", "conv_train"):
        D, KW = _log(rng, 32, 8192), rng.choice([2, 3, 4, 4, 4, 8])
        if op == "conv_step":
            B = _log(rng, 1, 400)
            return dict(op=op, B=B, T=rng.choice([1, 1, 2, 7]), D=D, KW=KW, views=views,
                        slots=rng.choice([0, B + rng.randint(0, 40)]), dtype=dtype)
        tokens = max(2, min(200_000, _log(rng, 2000, 19_000_000) // D))
        packed = rng.choice([0, rng.randint(1, 40)]) if op == "conv" else 0
        B = 1 if packed else min(128, _log(rng, 1, max(2, tokens // 20)))
        case = dict(op=op, B=B, L=tokens // B + 1, D=D, KW=KW, views=views, dtype=dtype)
        return case if op == "conv_train" else dict(case, packed=packed, h0=rng.random() < 0.5)
    G, N = rng.choice([1, 1, 1, 2, 4]), rng.choice([4, 8, 16, 16, 16, 32])
    D = G * max(1, _log(rng, 48, 6000) // G)
    gate = rng.random() < 0.7
    if op == "scan_step":
        B = _log(rng, 1, max(1, min(400, 16_000_000 // (D * N))))
        return dict(op=op, B=B, T=rng.choice([1, 1, 1, 2, 5]), D=D, N=N, G=G, gate=gate,
                    slots=rng.choice([0, B + rng.randint(0, 40)]), views=views, dtype=dtype)
    tokens = max(2, min(130_000, _log(rng, 100_000, 250_000_000) // (D * N)))
    packed = rng.choice([0, 0, rng.randint(1, 40)]) if op == "scan" else 0
    B = 1 if packed else min(64, _log(rng, 1, max(2, tokens // 50)))
    case = dict(op=op, B=B, L=tokens // B + 1, D=D, N=N, G=G, gate=gate, views=views, dtype=dtype)
    return case if op == "scan_train" else dict(case, packed=packed, h0=rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------------------
def _type(name):
    return BF16 if name == "bf16" else F32


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, op = _type(case["dtype"]), case["op"]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device="cuda")

    s = dict(case=case)
    if op in ("group", "group_train"):
        B, L, C = case["B"], case["L"], case["C"]
        s["x"] = normal(B, L, C, std=1.5) + normal(1, 1, C, std=0.5)
        s["weight"] = normal(C, std=0.2, dtype=F32) + 1 if case["affine"] else None
        s["bias"] = normal(C, std=0.2, dtype=F32) if case["affine"] else None
        s["eps"] = 1e-5
        if op == "group_train":
            s["dy"] = normal(B, L, C)
        return s

    B, D = case["B"], case["D"]
    L = case["T"] if op.endswith("step") else case["L"]
    s["slots"] = s["cu"] = s["h0"] = None
    rows = B
    if op.endswith("step"):
        rows = case["slots"] or B
        if case["slots"]:
            s["slots"] = torch.randperm(rows, generator=gen, device="cuda")[:B].to(torch.int32)
    elif case.get("packed"):
        S = rows = case["packed"]
        cuts = torch.randint(0, L + 1, (S - 1,), generator=gen, device="cuda").sort().values
        cuts[: S // 5] = cuts[: S // 5 + 1].min() if S > 5 else cuts[: S // 5]  # empty ones
        ends = torch.tensor([0, L], device="cuda")
        s["cu"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
        s["longest"] = int((s["cu"][1:] - s["cu"][:-1]).max())

    if op.startswith("conv"):
        KW = case["KW"]
        # the first half of one projection's output, or a tensor of its own
        s["x"] = normal(B, L, 2 * D)[..., :D] if case["views"] else normal(B, L, D)
        s["conv_w"], s["conv_b"] = normal(D, KW, std=KW ** -0.5, dtype=F32), normal(D, std=0.1, dtype=F32)
        if op == "conv_step":
            s["state"] = normal(rows, KW - 1, D)
        elif op == "conv_train":
            s["dy"] = normal(B, L, D)
        elif case["h0"]:
            s["h0"] = normal(rows, KW - 1, D)
        return s

    N, G = case["N"], case["G"]
    s["u"] = torch.nn.functional.silu(normal(B, L, D, dtype=F32)).to(dt)
    s["dt_raw"] = normal(B, L, D, std=0.5)
    low = max(1, D // 16)
    if case["views"]:  # z beside x in one projection's output, B and C in another's
        z = normal(B, L, 2 * D)[..., D:]
        bc = normal(B, L, low + 2 * G * N)
        s["Bs"], s["Cs"] = (bc[..., low + i * G * N:low + (i + 1) * G * N].unflatten(-1, (G, N))
                            for i in range(2))
    else:
        z = normal(B, L, D)
        s["Bs"], s["Cs"] = normal(B, L, G, N), normal(B, L, G, N)
    s["z"] = z if case["gate"] else None
    n = torch.arange(1, N + 1, device="cuda", dtype=F32)
    s["A_log"] = n.log() + normal(D, N, std=0.2, dtype=F32)
    s["Ds"] = normal(D, std=0.2, dtype=F32) + 1
    step = (uniform(D) * math.log(100.0) + math.log(1e-3)).exp()  # delta of 0.001 to 0.1
    s["dt_bias"] = step + (-(-step).expm1()).log()
    if op == "scan_step":
        s["state"] = normal(rows, D, N, std=0.3, dtype=F32)
    elif op == "scan_train":
        s["dy"] = normal(B, L, D)
    elif case["h0"]:
        s["h0"] = normal(rows, D, N, std=0.3, dtype=F32)
    return s


# ---- one pass ----------------------------------------------------------------------------
def run(s):
    return globals()[("_own_" if own else "_plain_") + s["case"]["op"]](s)


_SCAN = ("u", "dt_raw", "A_log", "Bs", "Cs", "Ds", "dt_bias")


def _own_scan_step(s):
    import selective_scan_ss2d_amd as ss
    y = ss.ss1d_scan_step(*[s[k] for k in _SCAN], s["state"], z=s["z"], slots=s["slots"])
    return dict(y=y, state=s["state"])


def _own_scan(s):
    import selective_scan_ss2d_amd as ss
    y, state = ss.ss1d_scan_forward(*[s[k] for k in _SCAN], z=s["z"], cu_seqlens=s["cu"],
                                    initial_state=s["h0"], final_state=True)
    return dict(y=y, state=state)


def _own_scan_train(s):
    import selective_scan_ss2d_amd as ss
    args = [s[k] for k in _SCAN]
    y, saved = ss.ss1d_scan_forward_save(*args, z=s["z"])
    d = ss.ss1d_scan_backward(*args, s["dy"], z=s["z"], saved=saved)
    return dict(y=y, **{"d" + k: d[k] for k in _SCAN + ("z",) if k in d})


def _own_conv_step(s):
    import selective_scan_ss2d_amd as ss
    y = ss.ss1d_conv_step(s["x"], s["conv_w"], s["state"], conv_b=s["conv_b"], slots=s["slots"])
    return dict(y=y, state=s["state"])


def _own_conv(s):
    import selective_scan_ss2d_amd as ss
    y, state = ss.ss1d_conv_forward(s["x"], s["conv_w"], conv_b=s["conv_b"], cu_seqlens=s["cu"],
                                    initial_state=s["h0"], final_state=True)
    return dict(y=y, state=state)


def _own_conv_train(s):
    import selective_scan_ss2d_amd as ss
    y = ss.ss1d_conv_forward(s["x"], s["conv_w"], conv_b=s["conv_b"])
    d = ss.ss1d_conv_backward(s["x"], s["conv_w"], s["dy"], conv_b=s["conv_b"])
    return dict(y=y, **{"d" + k: d[k] for k in ("x", "conv_w", "conv_b")})


def _group_args(s):
    return dict(weight=s["weight"], bias=s["bias"], silu=s["case"]["act"], eps=s["eps"])


def _own_group(s):
    import selective_scan_ss2d_amd as ss
    return dict(y=ss.ss2d_group_norm_forward(s["x"], s["case"]["G"], **_group_args(s)))


def _own_group_train(s):
    import selective_scan_ss2d_amd as ss
    y, stats = ss.ss2d_group_norm_forward(s["x"], s["case"]["G"], stats=True, **_group_args(s))
    d = ss.ss2d_group_norm_backward(s["x"], s["dy"], s["case"]["G"], stats=stats, **_group_args(s))
    return dict(y=y, **{"d" + k: v for k, v in d.items()})


# ---- the plain form of the scan --------------------------------------------------------------
def _softplus(x):
    return x.clamp(min=0) + (-x.abs()).exp().log1p()


def _silu(x):
    return x * torch.sigmoid(x)


def _spread(x, D):
    """(B, L, G, N) of the groups to (B, L, D, N) of the channels."""
    return x.float().repeat_interleave(D // x.shape[2], 2)


def _along_time(a, x, start):
    """h_t = a_t h_{t-1} + x_t along axis 1 of (B, L, D, N), from start (B, D, N): about sqrt(L)
    blocks at once, then their starts one after the other."""
    B, L = a.shape[:2]
    C = max(1, math.isqrt(L - 1) + 1) if L else 1
    pad = -L % C
    if pad:
        a = torch.cat([a, a.new_ones(B, pad, *a.shape[2:])], 1)
        x = torch.cat([x, x.new_zeros(B, pad, *x.shape[2:])], 1)
    a, x = (t.reshape(B, -1, C, *t.shape[2:]) for t in (a, x))
    h, p = torch.empty_like(x), torch.empty_like(a)
    for i in range(C):
        h[:, :, i] = x[:, :, i] + (a[:, :, i] * h[:, :, i - 1] if i else 0)
        p[:, :, i] = a[:, :, i] * p[:, :, i - 1] if i else a[:, :, i]
    for c in range(h.shape[1]):
        h[:, c] += p[:, c] * start[:, None]
        start = h[:, c, -1]
    return h.flatten(1, 2)[:, :L]


def _pad_rows(s, names):
    """Packed sequences as rows of the longest one's length: those of `names`, and which are tokens."""
    cu = s["cu"].long()
    at = torch.arange(s["longest"], device=cu.device)
    inside = at < (cu[1:] - cu[:-1])[:, None]
    index = torch.where(inside, cu[:-1, None] + at, 0)
    return [s[n][0][index] if s[n] is not None else None for n in names], inside


def _plain_scan_parts(s, inside=None, rows=None):
    u, dt_raw, Bs, Cs = rows or [s[n] for n in ("u", "dt_raw", "Bs", "Cs")]
    u, D = u.float(), u.shape[2]
    delta = _softplus(dt_raw.float() + s["dt_bias"])
    if inside is not None:
        delta = delta * inside[..., None]  # exp(0) h + 0: a token that leaves the state alone
    A = -s["A_log"].exp()
    a = (delta[..., None] * A).exp()
    Bs, Cs = _spread(Bs, D), _spread(Cs, D)
    return u, delta, A, a, Bs, Cs


def _plain_scan(s):
    z, inside = s["z"], None
    rows = None
    if s["cu"] is not None:
        (u, dt_raw, Bs, Cs, z), inside = _pad_rows(s, ("u", "dt_raw", "Bs", "Cs", "z"))
        rows = (u, dt_raw, Bs, Cs)
    u, delta, A, a, Bs, Cs = _plain_scan_parts(s, inside, rows)
    h0 = s["h0"] if s["h0"] is not None else u.new_zeros(u.shape[0], *A.shape)
    h = _along_time(a, (delta * u)[..., None] * Bs, h0)
    y = (h * Cs).sum(-1) + s["Ds"] * u
    if z is not None:
        y = y * _silu(z.float())
    y = y.to(s["u"].dtype)
    if inside is not None:
        y = y[inside][None]
    return dict(y=y, state=h[:, -1].clone())


def _plain_scan_step(s):
    at = s["slots"].long() if s["slots"] is not None else None
    u, delta, A, a, Bs, Cs = _plain_scan_parts(s)
    h, out = (s["state"] if at is None else s["state"][at]), []
    for t in range(u.shape[1]):
        h = a[:, t] * h + (delta[:, t] * u[:, t])[..., None] * Bs[:, t]
        out.append((h * Cs[:, t]).sum(-1))
    y = torch.stack(out, 1) + s["Ds"] * u
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    if at is None:
        s["state"].copy_(h)
    else:
        s["state"][at] = h
    return dict(y=y.to(s["u"].dtype), state=s["state"])


def _plain_scan_train(s):
    u, delta, A, a, Bs, Cs = _plain_scan_parts(s)
    B, L, D = u.shape
    G = s["Bs"].shape[2]
    h = _along_time(a, (delta * u)[..., None] * Bs, u.new_zeros(B, *A.shape))
    v = (h * Cs).sum(-1) + s["Ds"] * u
    dy, out = s["dy"].float(), {}
    y = v
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        y = v * (z * sg)
        out["dz"] = (dy * v * sg * (1 + z * (1 - sg))).to(s["z"].dtype)
        dy = dy * (z * sg)
    out["dCs"] = (dy[..., None] * h).unflatten(2, (G, -1)).sum(3).to(s["Cs"].dtype)
    # the adjoint, from the last token to the first: l_t = dy_t C_t + a_{t+1} l_{t+1}
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1).flip(1)
    lam = _along_time(after, (dy[..., None] * Cs).flip(1), u.new_zeros(B, *A.shape)).flip(1)
    out["dBs"] = (lam * (delta * u)[..., None]).unflatten(2, (G, -1)).sum(3).to(s["Bs"].dtype)
    q = (lam * Bs).sum(-1)
    before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
    w = lam * a * before
    out["dA_log"] = (w * delta[..., None]).sum((0, 1)) * A
    ddelta = (w * A).sum(-1) + u * q
    draw = ddelta * torch.sigmoid(s["dt_raw"].float() + s["dt_bias"])
    out["ddt_raw"], out["ddt_bias"] = draw.to(s["dt_raw"].dtype), draw.sum((0, 1))
    out["du"] = (delta * q + s["Ds"] * dy).to(s["u"].dtype)
    out["dDs"] = (dy * u).sum((0, 1))
    return dict(y=y.to(s["u"].dtype), **{k: out[k] for k in ["d" + n for n in _SCAN + ("z",)] if k in out})


# ---- the plain form of the convolution -----------------------------------------------------------
def _plain_taps(x, before, w, b):
    """x (B, L, D) and the KW - 1 inputs before it: the sum over the taps, and what it read."""
    KW, L = w.shape[1], x.shape[1]
    whole = torch.cat([before, x], 1).float()
    return sum(whole[:, j:j + L] * w[:, j] for j in range(KW)) + b, whole


def _plain_conv(s):
    x, inside = s["x"], None
    if s["cu"] is not None:
        (x,), inside = _pad_rows(s, ("x",))
    before = s["h0"] if s["h0"] is not None else x.new_zeros(x.shape[0], s["conv_w"].shape[1] - 1, x.shape[2])
    pre, _ = _plain_taps(x, before, s["conv_w"], s["conv_b"])
    y, whole = _silu(pre).to(x.dtype), torch.cat([before, x], 1)
    if inside is None:
        return dict(y=y, state=whole[:, x.shape[1]:].clone())
    at = inside.sum(1)[:, None] + torch.arange(before.shape[1], device=x.device)  # the last inputs
    state = whole.gather(1, at[..., None].expand(-1, -1, x.shape[2]))
    return dict(y=y[inside][None], state=state)


def _plain_conv_step(s):
    x, at = s["x"], s["slots"].long() if s["slots"] is not None else None
    before = s["state"] if at is None else s["state"][at]
    pre, _ = _plain_taps(x, before, s["conv_w"], s["conv_b"])
    end = torch.cat([before, x], 1)[:, x.shape[1]:]
    if at is None:
        s["state"].copy_(end)
    else:
        s["state"][at] = end
    return dict(y=_silu(pre).to(x.dtype), state=s["state"])


def _plain_conv_train(s):
    x, w = s["x"], s["conv_w"]
    KW, L = w.shape[1], x.shape[1]
    pre, whole = _plain_taps(x, x.new_zeros(x.shape[0], KW - 1, x.shape[2]), w, s["conv_b"])
    sg = torch.sigmoid(pre)
    d = s["dy"].float() * sg * (1 + pre * (1 - sg))
    dw = torch.stack([(d * whole[:, j:j + L]).sum((0, 1)) for j in range(KW)], 1)
    behind = torch.cat([d, d.new_zeros(d.shape[0], KW - 1, d.shape[2])], 1)
    dx = sum(behind[:, KW - 1 - j:KW - 1 - j + L] * w[:, j] for j in range(KW))
    return dict(y=(pre * sg).to(x.dtype), dx=dx.to(x.dtype), dconv_w=dw, dconv_b=d.sum((0, 1)))


# ---- the plain form of the group norm --------------------------------------------------------------
def _plain_unit(s):
    """x of every group with mean 0 and a mean square of one, (B, L, G, C / G), and the scale."""
    x = s["x"].float().unflatten(2, (s["case"]["G"], -1))
    x = x - x.mean((1, 3), keepdim=True)
    r = (x.square().mean((1, 3), keepdim=True) + s["eps"]).rsqrt()
    return x * r, r


def _plain_affine(s, x):
    x = x.flatten(2)
    return x * s["weight"] + s["bias"] if s["weight"] is not None else x


def _plain_group(s):
    y = _plain_affine(s, _plain_unit(s)[0])
    return dict(y=(_silu(y) if s["case"]["act"] else y).to(s["x"].dtype))


def _plain_group_train(s):
    x, r = _plain_unit(s)
    y, d = _plain_affine(s, x), s["dy"].float()
    if s["case"]["act"]:
        sg = torch.sigmoid(y)
        d = d * sg * (1 + y * (1 - sg))
        y = y * sg
    out = dict(y=y.to(s["x"].dtype))
    e = d if s["weight"] is None else d * s["weight"]
    e = e.unflatten(2, (s["case"]["G"], -1))
    e = e - e.mean((1, 3), keepdim=True) - x * (e * x).mean((1, 3), keepdim=True)
    out["dx"] = (e * r).flatten(2).to(s["x"].dtype)
    if s["weight"] is not None:
        out["dweight"], out["dbias"] = (d * x.flatten(2)).sum((0, 1)), d.sum((0, 1))
    return out


# ---- the work ----------------------------------------------------------------------------
def work(case):
    e, op = 2 if case["dtype"] == "bf16" else 4, case["op"]
    if op in ("group", "group_train"):
        n, v = case["B"] * case["L"] * case["C"], 8 * case["C"] * case["affine"]
        if op == "group":
            return {"bytes": 2 * n * e + v, "flops": 14 * n}
        return {"bytes": 4 * n * e + 2 * v, "flops": 40 * n}  # x, dy; y, dx
    B, D = case["B"], case["D"]
    rows = B * (case["T"] if op.endswith("step") else case["L"])
    if op.startswith("conv"):
        KW, seqs = case["KW"], case.get("packed") or B
        state, weights = seqs * (KW - 1) * D * e, D * (KW + 1) * 4
        if op == "conv_train":
            return {"bytes": 4 * rows * D * e + 2 * weights, "flops": rows * D * (6 * KW + 16)}
        states = 2 if op == "conv_step" else 1 + case["h0"]
        return {"bytes": 2 * rows * D * e + weights + states * state, "flops": rows * D * (2 * KW + 6)}
    N, G = case["N"], case["G"]
    params, state = D * (N + 2) * 4, D * N * 4
    wide, bc = rows * D * e, 2 * rows * G * N * e
    once = (3 + case["gate"]) * wide + bc + params
    if op == "scan_step":
        return {"bytes": once + 2 * B * state, "flops": 8 * rows * D * N}
    if op == "scan":
        return {"bytes": once + (1 + case["h0"]) * (case["packed"] or B) * state, "flops": 8 * rows * D * N}
    # forward: u, dt_raw, z, B, C; y.  backward: dy; and every input's gradient
    return {"bytes": once + wide + (2 + case["gate"]) * wide + bc + params, "flops": 26 * rows * D * N}


# ---- the definition in 64 bits -------------------------------------------------------------
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("group", "group_train"):
        return _exact_group(s)
    if op.startswith("conv"):
        return _exact_conv(s)
    if op == "scan_train":
        return _exact_scan_train(s) if case["L"] <= 20_000 else None
    if op == "scan" and case["L"] > 140_000:
        return None
    if op == "scan_step":
        at = torch.arange(case["B"], device="cuda") if s["slots"] is None else s["slots"].long()
        state = s["state"].double()
        y, state[at], _ = _exact_rows(s, slice(None), state[at])
        return dict(y=y, state=state)
    start = s["h0"].double() if s["h0"] is not None else None
    zero = torch.zeros(case["B"], case["D"], case["N"], dtype=F64, device="cuda")
    if s["cu"] is None:
        y, end, _ = _exact_rows(s, slice(None), zero if start is None else start)
        return dict(y=y, state=end)
    cu, parts = s["cu"].tolist(), []
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        parts.append(_exact_rows(s, slice(a, b), zero if start is None else start[i:i + 1])[:2])
    return dict(y=torch.cat([y for y, _ in parts], 1), state=torch.cat([h for _, h in parts]))


def _exact_rows(s, tokens, h, every=0):
    """The recurrence token by token over `tokens`; with `every`, the states before each
    every-th token."""
    u, raw, Bs, Cs = (s[n][:, tokens].double() for n in ("u", "dt_raw", "Bs", "Cs"))
    rep = u.shape[2] // Bs.shape[2]
    A = -s["A_log"].double().exp()
    delta = (1 + (raw + s["dt_bias"].double()).exp()).log()
    y, marks = torch.empty_like(u), []
    for t in range(u.shape[1]):
        if every and t % every == 0:
            marks.append(h)
        Bt, Ct = (x[:, t].repeat_interleave(rep, 1) for x in (Bs, Cs))
        h = (delta[:, t, :, None] * A).exp() * h + (delta[:, t] * u[:, t])[..., None] * Bt
        y[:, t] = (h * Ct).sum(-1)
    y = y + s["Ds"].double() * u
    if s["z"] is not None:
        z = s["z"][:, tokens].double()
        y = y * z / (1 + (-z).exp())
    return y, h, marks


def _exact_scan_train(s):
    u, raw, Bs, Cs, g = (s[n].double() for n in ("u", "dt_raw", "Bs", "Cs", "dy"))
    B, L, D = u.shape
    G, N = Bs.shape[2:]
    A = -s["A_log"].double().exp()
    v = raw + s["dt_bias"].double()
    delta, slope = (1 + v.exp()).log(), 1 / (1 + (-v).exp())
    every = max(1, math.isqrt(L))  # states kept every so many tokens, the others made again
    y, _, marks = _exact_rows(s, slice(None), torch.zeros(B, D, N, dtype=F64, device="cuda"), every)
    d = {n: torch.zeros_like(s[n], dtype=F64) for n in _SCAN}
    if s["z"] is not None:
        z = s["z"].double()
        sg = 1 / (1 + (-z).exp())
        plain = torch.empty_like(u)
    gated = g if s["z"] is None else g * z * sg
    lam = torch.zeros(B, D, N, dtype=F64, device="cuda")
    for c in range(len(marks) - 1, -1, -1):
        t0, t1 = c * every, min(L, (c + 1) * every)
        states = [marks[c]]
        for t in range(t0, t1):
            Bt = Bs[:, t].repeat_interleave(D // G, 1)
            a = (delta[:, t, :, None] * A).exp()
            states.append(a * states[-1] + (delta[:, t] * u[:, t])[..., None] * Bt)
        for t in range(t1 - 1, t0 - 1, -1):
            Bt, Ct = (x[:, t].repeat_interleave(D // G, 1) for x in (Bs, Cs))
            before, h = states[t - t0], states[t - t0 + 1]
            if s["z"] is not None:
                plain[:, t] = (h * Ct).sum(-1) + s["Ds"].double() * u[:, t]
            dy = gated[:, t]
            lam = lam + dy[..., None] * Ct
            a = (delta[:, t, :, None] * A).exp()
            d["Cs"][:, t] = (dy[..., None] * h).reshape(B, G, -1, N).sum(2)
            d["Bs"][:, t] = (lam * (delta[:, t] * u[:, t])[..., None]).reshape(B, G, -1, N).sum(2)
            through = lam * a * before
            d["A_log"] += (through * delta[:, t, :, None]).sum(0) * A
            back = (lam * Bt).sum(-1)
            raw_t = ((through * A).sum(-1) + back * u[:, t]) * slope[:, t]
            d["dt_raw"][:, t] = raw_t
            d["dt_bias"] += raw_t.sum(0)
            d["u"][:, t] = back * delta[:, t] + s["Ds"].double() * dy
            d["Ds"] += (dy * u[:, t]).sum(0)
            lam = lam * a
    out = {"d" + n: d[n] for n in _SCAN}
    if s["z"] is not None:
        out["dz"] = g * plain * sg * (1 + z * (1 - sg))
    return dict(y=y, **out)


def _exact_conv(s):
    op, KW = s["case"]["op"], s["conv_w"].shape[1]
    train = op == "conv_train"
    x = s["x"].double().requires_grad_(train)
    w, b = (s[n].double().requires_grad_(train) for n in ("conv_w", "conv_b"))

    def sequence(x, before):  # (L, D) behind (KW - 1, D)
        whole = torch.cat([before, x])
        v = torch.stack([whole[j:j + x.shape[0]] for j in range(KW)], -1)
        v = (v * w).sum(-1) + b
        return v / (1 + (-v).exp()), whole[x.shape[0]:]

    none = torch.zeros(KW - 1, x.shape[2], dtype=F64, device="cuda")
    if op == "conv_step":
        at = list(range(x.shape[0])) if s["slots"] is None else s["slots"].tolist()
        state, ys = s["state"].double(), []
        for i, slot in enumerate(at):
            y, state[slot] = sequence(x[i], state[slot].clone())
            ys.append(y)
        return dict(y=torch.stack(ys), state=state)
    if s["cu"] is None:
        parts = [sequence(x[i], s["h0"][i].double() if s["h0"] is not None else none)
                 for i in range(x.shape[0])]
        y = torch.stack([p for p, _ in parts])
    else:
        cu = s["cu"].tolist()
        parts = [sequence(x[0, a:e], s["h0"][i].double() if s["h0"] is not None else none)
                 for i, (a, e) in enumerate(zip(cu[:-1], cu[1:]))]
        y = torch.cat([p for p, _ in parts])[None]
    if not train:
        return dict(y=y, state=torch.stack([e for _, e in parts]))
    dx, dw, db = torch.autograd.grad(y, [x, w, b], s["dy"].double())
    return dict(y=y.detach(), dx=dx, dconv_w=dw, dconv_b=db)


def _exact_group(s):
    train = s["case"]["op"] == "group_train"
    x = s["x"].double().requires_grad_(train)
    wb = [s[n].double().requires_grad_(train) for n in ("weight", "bias") if s[n] is not None]
    B, L, C = x.shape
    G = s["case"]["G"]
    v = x.reshape(B, L, G, C // G).transpose(1, 2).reshape(B, G, -1)
    var, mean = torch.var_mean(v, -1, keepdim=True, unbiased=False)
    v = ((v - mean) / (var + s["eps"]).sqrt()).reshape(B, G, L, C // G).transpose(1, 2).reshape(B, L, C)
    if wb:
        v = v * wb[0] + wb[1]
    y = v / (1 + (-v).exp()) if s["case"]["act"] else v
    if not train:
        return dict(y=y)
    d = torch.autograd.grad(y, [x] + wb, s["dy"].double())
    return dict(y=y.detach(), **dict(zip(("dx", "dweight", "dbias"), d)))
