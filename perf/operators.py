"""Measured cases of the sequence operators: the gated delta rule and the block norm.

``run`` computes either the plain form (elementary torch operations in 32 bits) or, with
``own`` set, the calls that a user makes of the package.

The gated delta rule keeps one (DK, DV) state S per sequence and value head:
    S <- exp(g_t) S,   u_t = beta_t (v_t - S^T k_t),   S <- S + k_t u_t^T,
    o_t = scale S^T q_t.

The block norm joins the two norms around a residual connection:
    p = Norm(h; w_post, b_post) (p = h without w_post),   p <- p * SiLU(z),
    y = residual + res_scale * p,   n = Norm(y; w_pre, b_pre).
"""
import math

import torch

own = False
CHUNK = 64
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---- the cases ---------------------------------------------------------------------------
def listed():
    return [
        # one token of one sequence: the latency of a single reply, 32 heads of 128
        dict(name="delta step, one sequence", op="step", B=1, T=1, HK=16, H=32, DK=128, DV=128,
             slots=1, dtype="bf16"),
        # a served batch: one token of each of 256 sequences, their states in a pool of slots
        dict(name="delta step, batch of 256", op="step", B=256, T=1, HK=16, H=32, DK=128,
             DV=128, slots=300, dtype="bf16"),
        # drafted tokens: 5 tokens of each of 64 sequences, 12 heads of 64 (a width of 768)
        dict(name="delta step, 5 drafted fp32", op="step", B=64, T=5, HK=12, H=12, DK=64, DV=64,
             slots=0, dtype="f32"),
        # the prompt of one request, its final state handed on to the steps
        dict(name="delta prompt of 4096", op="forward", B=1, L=4096, HK=16, H=32, DK=128,
             DV=128, packed=0, h0=False, dtype="bf16"),
        # prompts of odd lengths packed into one call, continuing from earlier states
        dict(name="delta packed prompts", op="forward", B=1, L=12007, HK=4, H=8, DK=128, DV=96,
             packed=25, h0=True, dtype="bf16"),
        # one pass over two images of 256 x 256 positions in fp32 (3 heads of 64: width 192)
        dict(name="delta 256x256 image fp32", op="forward", B=2, L=65536, HK=3, H=3, DK=64,
             DV=64, packed=0, h0=False, dtype="f32"),
        # a training step over 14 * 14 + 1 tokens of 128 images, width 768
        dict(name="delta training, 197 tokens", op="train", B=128, L=197, HK=12, H=12, DK=64,
             DV=64, dtype="bf16"),
        # a training step over 56 * 56 positions of 64 images, width 192
        dict(name="delta training, 56x56", op="train", B=64, L=3136, HK=3, H=3, DK=64, DV=64,
             dtype="bf16"),
        # the residual connection and the next block's norm for the tokens of one step
        dict(name="norm, 8 tokens", op="norm", R=8, D=768, L=0, post=True, gate=False,
             residual=True, groups=1, pre=True, layer=False, ytype="bf16", dtype="bf16"),
        # the gated norm of every head's output (the delta rule's o) over 64 images
        dict(name="norm, gated heads", op="norm", R=602112, D=64, L=0, post=True, gate=True,
             residual=False, groups=0, pre=False, layer=False, ytype="bf16", dtype="bf16"),
        # around the image operator: channels first (64, 192, 56, 56), fp32 residual stream
        dict(name="norm, 56x56 maps", op="norm", R=64 * 3136, D=192, L=3136, post=True,
             gate=False, residual=True, groups=64, pre=True, layer=True, ytype="f32",
             dtype="bf16"),
        # the backward of gate, residual scale and both norms over 197 tokens of 128 images
        dict(name="norm backward, 197 tokens", op="norm_grad", R=25216, D=768, L=0, post=True,
             gate=True, residual=True, groups=1, pre=True, layer=False, ytype="bf16",
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "forward", "train", "norm", "norm_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("norm", "norm_grad"):
        first = rng.random() < 0.35
        D = _log(rng, 16, 1024 if first else 4096)
        total = _log(rng, 2000, 30_000_000)
        residual, pre = rng.random() < 0.7, rng.random() < 0.6
        post = rng.random() < 0.7 or not pre
        gate = rng.random() < 0.4
        B = rng.randint(1, 48)
        L = max(1, total // D // B)
        return dict(op=kind, R=B * L, D=D, L=L if first else 0, post=post, gate=gate,
                    residual=residual, groups=rng.choice([0, 1, B]), pre=pre,
                    layer=rng.random() < 0.5, ytype=dtype if not residual else
                    rng.choice([dtype, "f32"]), dtype=dtype)
    HK = rng.choice([1, 2, 3, 4, 8, 12, 16])
    H = HK * rng.choice([1, 1, 2, 3])
    DK, DV = rng.choice([32, 64, 80, 96, 128]), rng.choice([32, 48, 64, 100, 128, 192])
    if kind == "step":
        B = max(1, min(512, _log(rng, 1, 512) * 16 // H))
        return dict(op="step", B=B, T=rng.choice([1, 1, 2, 3, 7]), HK=HK, H=H, DK=DK, DV=DV,
                    slots=rng.choice([0, B + rng.randint(0, 40)]), dtype=dtype)
    tokens = min(60_000, _log(rng, 20, 300_000 if kind == "forward" else 100_000) // H + 1)
    if kind == "forward":
        packed = rng.choice([0, 0, rng.randint(1, 40)])
        B = 1 if packed else min(64, _log(rng, 1, max(2, tokens // 50)))
        return dict(op="forward", B=B, L=tokens // B + 1, HK=HK, H=H, DK=DK, DV=DV,
                    packed=packed, h0=rng.random() < 0.5, dtype=dtype)
    B = min(64, _log(rng, 1, max(2, tokens // 50)))
    return dict(op="train", B=B, L=tokens // B + 1, HK=HK, H=H, DK=DK, DV=DV, dtype=dtype)


# ---- inputs ------------------------------------------------------------------------------
def _type(name):
    return BF16 if name == "bf16" else F32


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _type(case["dtype"])

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    if case["op"] in ("norm", "norm_grad"):
        R, D, L = case["R"], case["D"], case["L"]
        shape = (R // L, D, L) if L else (R, D)
        yt = _type(case["ytype"])
        s = dict(case=case, h=normal(*shape, std=1.5))
        s["w_post"] = normal(D, std=0.2, dtype=F32) + 1 if case["post"] else None
        s["b_post"] = normal(D, std=0.2, dtype=F32) if case["post"] and case["layer"] else None
        s["z"] = normal(*shape) if case["gate"] else None
        s["residual"] = normal(*shape, std=3.0, dtype=yt) if case["residual"] else None
        g = case["groups"]
        s["res_scale"] = normal(g, D, std=0.3, dtype=F32) + 0.5 if g else None
        s["w_pre"] = normal(D, std=0.2, dtype=F32) + 1 if case["pre"] else None
        s["b_pre"] = normal(D, std=0.2, dtype=F32) if case["pre"] and case["layer"] else None
        s["layer"], s["eps"] = case["layer"], 1e-6
        if case["op"] == "norm_grad":  # what the forward left, and what the next layers send
            s["y"] = normal(*shape, std=3.0, dtype=yt)
            s["dy"] = normal(*shape, dtype=yt)
            s["dn"] = normal(*shape) if case["pre"] else None
        return s

    B, HK, H, DK, DV = (case[k] for k in ("B", "HK", "H", "DK", "DV"))
    L = case["T"] if case["op"] == "step" else case["L"]

    def unit(*shape):
        x = torch.nn.functional.silu(torch.randn(shape, generator=gen, device="cuda"))
        return (x / (x.square().sum(-1, keepdim=True) + 1e-6).sqrt()).to(dt)

    s = dict(case=case, q=unit(B, L, HK, DK), k=unit(B, L, HK, DK), v=normal(B, L, H, DV))
    rate = torch.rand(H, generator=gen, device="cuda") * 15 + 1  # decay rates of 1 to 16
    step = torch.nn.functional.softplus(normal(B, L, H, dtype=F32) - 4)
    s["g"] = -rate * step
    s["beta"] = torch.sigmoid(normal(B, L, H, dtype=F32))
    s["scale"] = DK ** -0.5
    s["cu"] = s["h0"] = s["slots"] = None
    if case["op"] == "step":
        n = case["slots"] or B
        s["state"] = normal(n, H, DK, DV, std=0.3, dtype=F32)
        if case["slots"]:
            s["slots"] = torch.randperm(n, generator=gen, device="cuda")[:B].to(torch.int32)
    if case["op"] == "forward":
        S = case["packed"]
        if S:
            cuts = torch.randint(0, L + 1, (S - 1,), generator=gen, device="cuda").sort().values
            cuts[: S // 5] = cuts[: S // 5 + 1].min() if S > 5 else cuts[: S // 5]  # empty ones
            ends = torch.tensor([0, L], device="cuda")
            s["cu"] = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
            s["longest"] = int((s["cu"][1:] - s["cu"][:-1]).max())
        if case["h0"]:
            s["h0"] = normal(S or B, H, DK, DV, std=0.3, dtype=F32)
    if case["op"] == "train":
        s["do"] = normal(B, L, H, DV)
    return s


# ---- one pass ----------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"step": _own_step, "forward": _own_forward, "train": _own_train,
                "norm": _own_norm, "norm_grad": _own_norm_grad}[op](s)
    return {"step": _plain_step, "forward": _plain_forward, "train": _plain_train,
            "norm": _plain_norm, "norm_grad": _plain_norm_grad}[op](s)


_SEQ = ("q", "k", "v", "g", "beta")
_NORM = ("w_post", "b_post", "z", "res_scale", "w_pre", "b_pre", "layer", "eps")


def _own_step(s):
    import selective_scan_ss2d_amd as ss
    o = ss.ss1d_delta_step(*[s[k] for k in _SEQ], s["state"], slots=s["slots"],
                           scale=s["scale"])
    return dict(o=o, state=s["state"])


def _own_forward(s):
    import selective_scan_ss2d_amd as ss
    o, state = ss.ss1d_delta_forward(*[s[k] for k in _SEQ], scale=s["scale"],
                                     cu_seqlens=s["cu"], initial_state=s["h0"],
                                     final_state=True)
    return dict(o=o, state=state)


def _own_train(s):
    import selective_scan_ss2d_amd as ss
    args = [s[k] for k in _SEQ]
    o, saved = ss.ss1d_delta_forward_save(*args, scale=s["scale"])
    d = ss.ss1d_delta_backward(*args, s["do"], scale=s["scale"], saved=saved)
    return dict(o=o, **{"d" + k: d[k] for k in _SEQ})


def _own_norm(s):
    import selective_scan_ss2d_amd as ss
    y, n = ss.ss2d_norm_forward(s["h"], residual=s["residual"],
                                channels_first=s["case"]["L"] > 0, **{k: s[k] for k in _NORM})
    return dict(y=y, n=n)


def _own_norm_grad(s):
    import selective_scan_ss2d_amd as ss
    d = ss.ss2d_norm_backward(s["h"], s["y"], s["dy"], s["dn"],
                              residual=s["residual"] is not None,
                              channels_first=s["case"]["L"] > 0, **{k: s[k] for k in _NORM})
    return {"d" + k: v for k, v in d.items()}


# ---- the plain form of the delta rule --------------------------------------------------------
def _plain_step(s):
    q, k, v = (s[n].float() for n in ("q", "k", "v"))
    rep = v.shape[2] // q.shape[2]
    q, k = (x.repeat_interleave(rep, 2) for x in (q, k))
    at = s["slots"].long() if s["slots"] is not None else None
    S = s["state"] if at is None else s["state"][at]
    outs = []
    for t in range(q.shape[1]):
        S = S * s["g"][:, t, :, None, None].exp()
        kt = k[:, t, :, :, None]
        u = s["beta"][:, t, :, None] * (v[:, t] - (S * kt).sum(-2))
        S = S + kt * u[:, :, None, :]
        outs.append(s["scale"] * (S * q[:, t, :, :, None]).sum(-2))
    if at is None:
        s["state"].copy_(S)
    else:
        s["state"][at] = S
    return dict(o=torch.stack(outs, 1).to(s["v"].dtype), state=s["state"])


def _inverse(A):
    """(I + A)^-1 of strictly lower triangular A: inverses of diagonal blocks of 1, 2, 4, ...
    joined in pairs, [[P, 0], [X, Q]]^-1 = [[P', 0], [-Q' X P', Q']]."""
    C = A.shape[-1]
    i = torch.arange(C, device=A.device)
    T = torch.eye(C, device=A.device).expand_as(A)
    size = 1
    while size < C:
        pair = (i[:, None] // (2 * size) == i // (2 * size)) & (i[:, None] // size
                                                               != i // size)
        T = T - T @ (A * pair) @ T
        size *= 2
    return T


def _plain_chunks(q, k, v, g, beta, scale, S):
    """(N, L, DK) q, k, (N, L, DV) v, (N, L) g and beta, S (N, DK, DV): o and the end state."""
    N, L, DK = q.shape
    C = min(CHUNK, 1 << max(0, (L - 1).bit_length()))
    pad = -L % C
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, pad)) for x in (q, k, v))
    g, beta = (torch.nn.functional.pad(x, (0, pad)) for x in (g, beta))
    q, k, v = (x.reshape(N, -1, C, x.shape[-1]) for x in (q, k, v))
    g, beta = (x.reshape(N, -1, C) for x in (g, beta))
    G = g.cumsum(-1)
    low = torch.ones(C, C, device=q.device).tril().bool()
    M = (G[..., :, None] - G[..., None, :]).masked_fill(~low, -math.inf).exp()
    kt = k.transpose(-1, -2)
    A = ((k @ kt) * M).tril(-1)
    T = _inverse(A * beta[..., None, :])
    P = (q @ kt) * M
    decay = G.exp()[..., None]
    kin, qin = k * decay, q * decay
    kout = (k * (G[..., -1:] - G).exp()[..., None]).transpose(-1, -2)
    whole = decay[:, :, -1:]
    outs = []
    for c in range(q.shape[1]):
        u = beta[:, c, :, None] * (T[:, c] @ (v[:, c] - kin[:, c] @ S))
        outs.append(scale * (qin[:, c] @ S + P[:, c] @ u))
        S = whole[:, c] * S + kout[:, c] @ u
    return torch.cat(outs, 1)[:, :L], S


def _heads(q, k, v, g, beta):
    """Every sequence and value head a row: the key heads repeated, in 32 bits."""
    B, L, H, DV = v.shape
    rep = H // q.shape[2]
    q, k = (x.float().repeat_interleave(rep, 2) for x in (q, k))
    rows = [x.transpose(1, 2).reshape(B * H, L, -1) for x in (q, k, v.float())]
    return rows + [x.transpose(1, 2).reshape(B * H, L) for x in (g, beta)]


def _plain_forward(s):
    q, k, v, g, beta = (s[n] for n in _SEQ)
    H, DV, DK = v.shape[2], v.shape[3], q.shape[3]
    cu = s["cu"]
    if cu is not None:  # one row a sequence, padded with tokens that leave the state alone
        at = torch.arange(s["longest"], device=v.device)
        cu = cu.long()
        inside = at < (cu[1:] - cu[:-1])[:, None]
        index = torch.where(inside, cu[:-1, None] + at, 0)
        q, k, v, g, beta = (x[0][index] * inside.reshape(inside.shape + (1,) * (x.dim() - 2))
                            for x in (q, k, v, g, beta))
    N, L = v.shape[:2]
    S = torch.zeros(N * H, DK, DV, device=v.device)
    if s["h0"] is not None:
        S = s["h0"].reshape(N * H, DK, DV)
    o, S = _plain_chunks(*_heads(q, k, v, g, beta), s["scale"], S)
    o = o.reshape(N, H, L, DV).transpose(1, 2).to(v.dtype)
    if cu is not None:
        o = o[inside][None]
    return dict(o=o.contiguous(), state=S.reshape(N, H, DK, DV))


def _plain_train(s):
    leaves = [s[n].detach().float().requires_grad_() for n in _SEQ]
    q, k, v, g, beta = leaves
    B, L, H, DV = v.shape
    S = torch.zeros(B * H, q.shape[3], DV, device=v.device)
    o, _ = _plain_chunks(*_heads(q, k, v, g, beta), s["scale"], S)
    o = o.reshape(B, H, L, DV).transpose(1, 2)
    grads = torch.autograd.grad(o, leaves, s["do"].float())
    out = {"d" + n: d.to(s[n].dtype) for n, d in zip(_SEQ, grads)}
    return dict(o=o.detach().to(s["v"].dtype).contiguous(), **out)


# ---- the plain form of the norm ----------------------------------------------------------
def _unit(x, layer, eps, dim):
    """x centred (layer) and scaled to a mean square of one, and the scale."""
    if layer:
        x = x - x.mean(dim, keepdim=True)
    r = (x.square().mean(dim, keepdim=True) + eps).rsqrt()
    return x * r, r


def _along(w, s):
    """A channel vector (D) or (G, D) against the rows, (R, D) or (B, D, L)."""
    if w is None:
        return None
    h, first = s["h"], s["case"]["L"] > 0
    if w.dim() == 1:
        return w[:, None] if first else w
    if first:
        return w[..., None]
    return w if w.shape[0] == 1 else w.repeat_interleave(h.shape[0] // w.shape[0], 0)


def _plain_branch(s, dim):
    p = s["h"].float()
    x, r = _unit(p, s["layer"], s["eps"], dim) if s["w_post"] is not None else (p, None)
    p = x
    if s["w_post"] is not None:
        p = p * _along(s["w_post"], s)
        p = p if s["b_post"] is None else p + _along(s["b_post"], s)
    return x, r, p


def _plain_norm(s):
    dim = 1
    _, _, y = _plain_branch(s, dim)
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z * torch.sigmoid(z))
    if s["res_scale"] is not None:
        y = y * _along(s["res_scale"], s)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    n = None
    if s["w_pre"] is not None:
        n = _unit(y, s["layer"], s["eps"], dim)[0] * _along(s["w_pre"], s)
        n = (n if s["b_pre"] is None else n + _along(s["b_pre"], s)).to(s["h"].dtype)
    return dict(y=y.to(_type(s["case"]["ytype"])), n=n)


def _through(d, x, r, layer, dim):
    """The gradient at a norm's input from that at its unit output x = (input - mean) r."""
    d = d - x * (d * x).mean(dim, keepdim=True)
    if layer:
        d = d - d.mean(dim, keepdim=True)
    return d * r


def _plain_norm_grad(s):
    dim, first = 1, s["case"]["L"] > 0
    rows = (0, 2) if first else (0,)
    out = {}
    d = s["dy"].float()
    if s["w_pre"] is not None:
        x, r = _unit(s["y"].float(), s["layer"], s["eps"], dim)
        dn = s["dn"].float()
        out["dw_pre"] = (dn * x).sum(rows)
        if s["b_pre"] is not None:
            out["db_pre"] = dn.sum(rows)
        d = d + _through(dn * _along(s["w_pre"], s), x, r, s["layer"], dim)
    if s["residual"] is not None:
        out["dresidual"] = d.to(s["y"].dtype)
    x, r, p = _plain_branch(s, dim)
    if s["z"] is not None:
        z = s["z"].float()
        sg = torch.sigmoid(z)
        gated = p * (z * sg)
    else:
        gated = p
    if s["res_scale"] is not None:
        g = s["res_scale"].shape[0]
        ds = d * gated
        if g == 1:
            ds = ds.sum(rows)[None]
        else:
            ds = ds.sum(2) if first else ds.reshape(g, -1, ds.shape[-1]).sum(1)
            ds = ds.reshape(g, -1, ds.shape[-1]).sum(1) if first else ds
        out["dres_scale"] = ds
        d = d * _along(s["res_scale"], s)
    if s["z"] is not None:
        out["dz"] = (d * p * sg * (1 + z * (1 - sg))).to(s["h"].dtype)
        d = d * (z * sg)
    if s["w_post"] is not None:
        out["dw_post"] = (d * x).sum(rows)
        if s["b_post"] is not None:
            out["db_post"] = d.sum(rows)
        d = _through(d * _along(s["w_post"], s), x, r, s["layer"], dim)
    out["dh"] = d.to(s["h"].dtype)
    return out


# ---- the work ----------------------------------------------------------------------------
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_grad"):
        n, D, ye = case["R"] * case["D"], case["D"], 2 if case["ytype"] == "bf16" else 4
        vectors = (case["post"] + case["pre"]) * (1 + case["layer"]) + case["groups"]
        if case["op"] == "norm":
            per = e + e * case["gate"] + ye * case["residual"] + ye + e * case["pre"]
            return {"bytes": n * per + vectors * D * 4, "flops": n * 10}
        per = e + ye + e * case["gate"] + (ye + e) * case["pre"]
        per += e + e * case["gate"] + ye * case["residual"]
        return {"bytes": n * per + 2 * vectors * D * 4, "flops": n * 25}
    B, HK, H, DK, DV = (case[k] for k in ("B", "HK", "H", "DK", "DV"))
    L = case["T"] if case["op"] == "step" else case["L"]
    rows, state = B * L, H * DK * DV * 4
    qk, vo, gates = rows * HK * DK * e, rows * H * DV * e, rows * H * 4
    moved, flops = 2 * qk + 2 * vo + 2 * gates, 6 * rows * H * DK * DV
    if case["op"] == "step":
        return {"bytes": moved + 2 * B * state, "flops": flops}
    if case["op"] == "forward":
        seqs = case["packed"] or B
        return {"bytes": moved + (1 + case["h0"]) * seqs * state, "flops": flops}
    return {"bytes": moved + vo + 2 * qk + vo + 2 * gates, "flops": 3 * flops}


# ---- the definition in 64 bits -------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(s)
    q, k, v, g, beta = (s[n].double() for n in _SEQ)
    rep = v.shape[2] // q.shape[2]
    if case["op"] == "step":
        S = s["state"].double()
        rows = torch.arange(q.shape[0], device="cuda") if s["slots"] is None else s["slots"].long()
        o, end, _ = _exact_rule(q, k, v, g, beta, s["scale"], S[rows], rep)
        S[rows] = end
        return dict(o=o, state=S)
    if case["op"] == "forward":
        B, L, H, DV = v.shape
        S = s["h0"].double() if s["h0"] is not None else None
        if s["cu"] is None:
            if S is None:
                S = torch.zeros(B, H, q.shape[3], DV, dtype=F64, device="cuda")
            if L > 70_000:
                return None
            o, end, _ = _exact_rule(q, k, v, g, beta, s["scale"], S, rep)
            return dict(o=o, state=end)
        cu = s["cu"].tolist()
        if S is None:
            S = torch.zeros(len(cu) - 1, H, q.shape[3], DV, dtype=F64, device="cuda")
        if L > 70_000:
            return None
        os, ends = [], []
        for i in range(len(cu) - 1):
            part = [x[:, cu[i]:cu[i + 1]] for x in (q, k, v, g, beta)]
            o, end, _ = _exact_rule(*part, s["scale"], S[i:i + 1], rep)
            os.append(o)
            ends.append(end)
        return dict(o=torch.cat(os, 1), state=torch.cat(ends))
    B, L, H, DV = v.shape
    DK = q.shape[3]
    if L > 25_000:
        return None
    every = max(1, math.isqrt(L))  # states kept every so many tokens, the others made again
    S = torch.zeros(B, H, DK, DV, dtype=F64, device="cuda")
    o, _, marks = _exact_rule(q, k, v, g, beta, s["scale"], S, rep, every)
    do, dS = s["do"].double(), torch.zeros_like(S)
    d = {n: torch.zeros_like(x) for n, x in zip(_SEQ, (q, k, v, g, beta))}
    for c in range(len(marks) - 1, -1, -1):
        t0, t1 = c * every, min(L, (c + 1) * every)
        part = [x[:, t0:t1] for x in (q, k, v, g, beta)]
        _, _, states = _exact_rule(*part, s["scale"], marks[c], rep, 1)
        for t in range(t1 - 1, t0 - 1, -1):
            qt, kt = (x[:, t].repeat_interleave(rep, 1)[..., None] for x in (q, k))
            a = g[:, t].exp()[..., None, None]
            before = a * states[t - t0]
            r = v[:, t] - (before * kt).sum(-2)
            u = beta[:, t][..., None] * r
            dot = s["scale"] * do[:, t][:, :, None]
            fold = (B, H // rep, rep, DK)
            d["q"][:, t] = ((before + kt * u[:, :, None]) * dot).sum(-1).reshape(fold).sum(2)
            dS = dS + qt * dot
            du = (dS * kt).sum(-2)
            d["beta"][:, t] = (du * r).sum(-1)
            dr = beta[:, t][..., None] * du
            d["v"][:, t] = dr
            dk = (dS * u[:, :, None]).sum(-1) - (before * dr[:, :, None]).sum(-1)
            d["k"][:, t] = dk.reshape(fold).sum(2)
            dS = dS - kt * dr[:, :, None]
            d["g"][:, t] = (dS * before).sum((-1, -2))
            dS = dS * a
    return dict(o=o, **{"d" + n: x for n, x in d.items()})


def _exact_rule(q, k, v, g, beta, scale, S, rep, every=0):
    """The recurrence token by token; with `every`, the states before tokens 0, every, ..."""
    out, marks = torch.empty_like(v), []
    decay = g.exp()
    for t in range(q.shape[1]):
        if every and t % every == 0:
            marks.append(S)
        qt, kt = (x[:, t].repeat_interleave(rep, 1)[..., None] for x in (q, k))
        S = S * decay[:, t, :, None, None]
        u = beta[:, t, :, None] * (v[:, t] - (S * kt).sum(-2))
        S = S + kt * u[:, :, None]
        out[:, t] = scale * (S * qt).sum(-2)
    return out, S, marks


def _exact_norm(s):
    grad = s["case"]["op"] == "norm_grad"
    names = ("h", "z", "residual", "res_scale", "w_post", "b_post", "w_pre", "b_pre")
    t = {n: s[n].double().requires_grad_(grad) if s[n] is not None else None for n in names}

    def move(x):  # channels last
        return x.transpose(1, 2) if s["case"]["L"] else x

    def norm(x, w, b):
        if s["layer"]:
            x = x - x.mean(-1, keepdim=True)
        x = x / (x.square().mean(-1, keepdim=True) + s["eps"]).sqrt() * w
        return x if b is None else x + b

    p = move(t["h"])
    if t["w_post"] is not None:
        p = norm(p, t["w_post"], t["b_post"])
    if t["z"] is not None:
        z = move(t["z"])
        p = p * z / (1 + (-z).exp())
    if t["res_scale"] is not None:
        G, D = t["res_scale"].shape
        p = (p.reshape(G, -1, D) * t["res_scale"][:, None]).reshape(p.shape)
    y = p if t["residual"] is None else p + move(t["residual"])
    if not grad:
        n = norm(y, t["w_pre"], t["b_pre"]) if t["w_pre"] is not None else None
        return dict(y=move(y), n=move(n) if n is not None else None)
    # the second norm reads y as it was stored; what it sends back joins dy
    d, out = move(s["dy"].double()), {}
    if t["w_pre"] is not None:
        stored = move(s["y"].double()).requires_grad_()
        wb = [x for x in (t["w_pre"], t["b_pre"]) if x is not None]
        n = norm(stored, t["w_pre"], t["b_pre"])
        got = torch.autograd.grad(n, [stored] + wb, move(s["dn"].double()))
        d = d + got[0]
        out["dw_pre"] = got[1]
        if t["b_pre"] is not None:
            out["db_pre"] = got[2]
    left = [n for n in names[:6] if t[n] is not None]
    got = torch.autograd.grad(y, [t[n] for n in left], d)
    out.update({"d" + n: x for n, x in zip(left, got)})
    return out
