"""The gated delta rule's forward and single-token forms against the definition in 64 bits."""
import pytest
import torch

import selective_scan_ss2d_amd as ss
from tests import delta_util as du

pytestmark = pytest.mark.gpu

SHAPES = [  # B, L, HK, H, DK, DV
    (1, 1, 1, 1, 1, 1), (1, 1, 2, 4, 64, 64), (2, 31, 1, 2, 32, 32), (3, 32, 2, 2, 16, 40),
    (1, 33, 1, 3, 64, 31), (2, 100, 2, 4, 128, 96), (1, 197, 3, 3, 64, 64),
    (2, 130, 1, 1, 80, 100), (1, 257, 2, 2, 127, 33), (1, 1030, 1, 2, 128, 128),
]
TYPES = [torch.float32, torch.bfloat16]


def run(t, scale=None, **kw):
    d = du.to_gpu(t)
    return ss.ss1d_delta_forward(*[d[n] for n in du.NAMES], scale=scale,
                                 initial_state=d["h0"], **kw)


def check_forward(t, dtype, o, ht, scale, cu=None):
    ref_o, ref_s = du.reference(t, scale, cu)
    DK = t["q"].shape[3]
    du.check(o, ref_o, "o", *du.o_bounds(DK, ref_o, dtype))
    du.check(ht, ref_s, "end states", du.f32_bound(DK, ref_s))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(shape, dtype):
    B, L, HK, H, DK, DV = shape
    t = du.make_inputs(*shape, dtype, seed=L, h0=B if L % 2 else 0)
    o, ht = run(t, final_state=True)
    check_forward(t, dtype, o, ht, DK ** -0.5)
    only = run(t)
    assert torch.equal(only, o)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("decay", [0.0, 3.0, 40.0])
def test_decays_from_none_to_strong(dtype, decay):
    t = du.make_inputs(2, 150, 2, 2, 64, 48, dtype, seed=5, decay=decay, h0=2)
    o, ht = run(t, scale=0.7, final_state=True)
    check_forward(t, dtype, o, ht, 0.7)


@pytest.mark.parametrize("dtype", TYPES)
def test_forgetting_everything_and_writing_nothing(dtype):
    t = du.make_inputs(1, 140, 1, 2, 64, 64, dtype, seed=6, h0=1)
    t["g"][0, 70, 0] = -float("inf")     # the state is dropped before token 70
    t["g"][0, 3, 1] = torch.finfo(torch.float32).min
    t["beta"][0, :, 1] = 0.0             # head 1 only ever decays its initial state
    t["beta"][0, 40:60, 0] = 1.0
    o, ht = run(t, scale=1.0, final_state=True)
    check_forward(t, dtype, o, ht, 1.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_repeated_keys(dtype):
    """The triangular solve at its worst: one key for all tokens, beta = 1."""
    t = du.make_inputs(1, 100, 1, 1, 64, 64, dtype, seed=7, decay=0.0)
    t["k"][:] = t["k"][:, :1]
    t["beta"][:] = 1.0
    o, ht = run(t, scale=1.0, final_state=True)
    ref_o, ref_s = du.reference(t, 1.0)
    big = torch.cat([ref_o.flatten(), t["v"].double().flatten()])
    # the solution u cancels v against S^T k: its terms have v's magnitude
    du.check(o, ref_o, "o", du.o_bounds(64, big, dtype)[0] * 4, du.BF16_HALF)
    du.check(ht, ref_s, "end states", du.f32_bound(64, big) * 4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("with_h0", [False, True])
def test_packed_sequences(dtype, with_h0):
    """Sequences of 0, 1, 31, 32, 33, 64, 65 and 100 tokens, none at both ends, and rows that
    belong to no sequence, which stay as they were."""
    lens = [0, 1, 31, 32, 0, 33, 64, 65, 100, 0]
    cu = torch.tensor([5] + [0] * len(lens), dtype=torch.int32)
    for i, n in enumerate(lens):
        cu[i + 1] = cu[i] + n
    L = int(cu[-1]) + 9
    t = du.make_inputs(1, L, 2, 4, 64, 48, dtype, seed=8, h0=len(lens) if with_h0 else 0)
    d = du.to_gpu(t)
    o = torch.full((1, L, 4, 48), 7.0, dtype=dtype, device="cuda")
    o, ht = ss.ss1d_delta_forward(*[d[n] for n in du.NAMES], scale=0.5, cu_seqlens=cu.cuda(),
                                  initial_state=d["h0"], final_state=True, o=o)
    assert (o[0, :5] == 7).all() and (o[0, L - 9:] == 7).all()
    ref_o, _ = du.reference(t, 0.5, cu)
    o[0, :5] = 0
    o[0, L - 9:] = 0
    check_forward(t, dtype, o, ht, 0.5, cu)
    if not with_h0:
        assert (ht[0] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_packed_equals_dense(dtype):
    """The same sequences as rows and packed: bit for bit."""
    B, L = 5, 77
    t = du.make_inputs(B, L, 1, 2, 64, 64, dtype, seed=9)
    o, ht = run(t, final_state=True)
    p = {n: t[n].reshape(1, B * L, *t[n].shape[2:]) for n in du.NAMES}
    p["h0"] = None
    cu = torch.arange(0, B * L + 1, L, dtype=torch.int32, device="cuda")
    po, pht = run(p, cu_seqlens=cu, final_state=True)
    assert torch.equal(po.view_as(o), o) and torch.equal(pht, ht)


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_views_of_one_projection(dtype):
    """q, k and v as slices of a fused projection, at offsets that break 16-byte alignment."""
    B, L, H, D = 2, 70, 2, 64
    t = du.make_inputs(B, L, H, H, D, D, dtype, seed=10)
    whole, _ = run(t, final_state=True)
    for pad in (0, 1, 8):
        fused = torch.zeros(B, L, 3 * H * D + pad + 8, dtype=dtype, device="cuda")
        parts = []
        for i, n in enumerate(("q", "k", "v")):
            at = pad + i * H * D
            fused[:, :, at:at + H * D] = t[n].cuda().reshape(B, L, H * D)
            parts.append(fused[:, :, at:at + H * D].unflatten(2, (H, D)))
        o = ss.ss1d_delta_forward(*parts, t["g"].cuda(), t["beta"].cuda())
        assert torch.equal(o, whole), pad


@pytest.mark.parametrize("dtype", TYPES)
def test_continuing_from_a_state(dtype):
    """Two parts, the second from the first's end state (in place): the whole's values, to the
    rounding of where the sums and the states' factors are cut."""
    t = du.make_inputs(2, 160, 1, 2, 64, 64, dtype, seed=11, h0=2)
    d = du.to_gpu(t)
    for cut in (1, 50, 96):
        first = [d[n][:, :cut].contiguous() for n in du.NAMES]
        second = [d[n][:, cut:].contiguous() for n in du.NAMES]
        state = d["h0"].clone()
        oa, back = ss.ss1d_delta_forward(*first, initial_state=state, final_state=state)
        assert back is state
        ob, _ = ss.ss1d_delta_forward(*second, initial_state=state, final_state=state)
        check_forward(t, dtype, torch.cat([oa, ob], 1), state, 64 ** -0.5)


SEGMENTED = [(1, 1, 1, 1, 8, 8), (2, 130, 1, 2, 64, 48), (1, 257, 2, 2, 127, 33),
             (1, 400, 1, 2, 128, 128), (3, 192, 1, 1, 32, 64), (1, 129, 1, 1, 30, 100)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("chunks", [2, 4])
@pytest.mark.parametrize("shape", SEGMENTED)
def test_segments(shape, chunks, dtype):
    """Sequences cut into segments that run at once, joined by their matrices."""
    B, L, HK, H, DK, DV = shape
    t = du.make_inputs(*shape, dtype, seed=L, h0=B if L % 2 else 0)
    with du.segments(chunks):
        o, ht = run(t, final_state=True)
        check_forward(t, dtype, o, ht, DK ** -0.5)
        state = t["h0"].cuda() if t["h0"] is not None else None
        if state is not None:  # in place
            d = du.to_gpu(t)
            p, _ = ss.ss1d_delta_forward(*[d[n] for n in du.NAMES], initial_state=state,
                                         final_state=state)
            assert torch.equal(p, o) and torch.equal(state, ht)


def test_end_states_over_initial_states_of_many_segments():
    """In place, the last segment's waves write where the first one's start is kept."""
    t = du.make_inputs(12, 1500, 2, 8, 64, 64, torch.bfloat16, seed=5, h0=12)
    d = du.to_gpu(t)
    with du.segments(2):
        o, ht = run(t, final_state=True)
        for _ in range(5):
            state = t["h0"].cuda()
            p, _ = ss.ss1d_delta_forward(*[d[n] for n in du.NAMES], initial_state=state,
                                         final_state=state)
            assert torch.equal(p, o) and torch.equal(state, ht)


@pytest.mark.parametrize("dtype", TYPES)
def test_segments_of_packed_sequences(dtype):
    lens = [0, 1, 31, 300, 0, 33, 64, 65, 128, 129, 0]
    cu = torch.tensor([5] + [0] * len(lens), dtype=torch.int32)
    for i, n in enumerate(lens):
        cu[i + 1] = cu[i] + n
    t = du.make_inputs(1, int(cu[-1]) + 9, 2, 4, 64, 48, dtype, seed=8, h0=len(lens))
    d = du.to_gpu(t)
    o = torch.zeros_like(d["v"])
    with du.segments(2):
        o, ht = ss.ss1d_delta_forward(*[d[n] for n in du.NAMES], scale=0.5, cu_seqlens=cu.cuda(),
                                      initial_state=d["h0"], final_state=True, o=o)
    check_forward(t, dtype, o, ht, 0.5, cu)
    assert torch.equal(ht[0], d["h0"][0])


@pytest.mark.parametrize("dtype", TYPES)
def test_a_long_sequence_cuts_itself(dtype):
    """One head and 2,100 tokens: the rule's own segments, against the uncut run."""
    t = du.make_inputs(1, 2100, 1, 1, 64, 64, dtype, seed=3, decay=0.02)
    o, ht = run(t, final_state=True)
    with du.segments(0):
        p, pht = run(t, final_state=True)
    assert not torch.equal(ht, pht)
    big = p.double().cpu()
    du.check(o, big, "o", *[2 * x for x in du.o_bounds(64, big, dtype)])
    du.check(ht, pht.double().cpu(), "end state", 2 * du.f32_bound(64, pht.double().cpu()))


def test_values_in_masked_places():
    """NaN and infinities in tokens that belong to no sequence reach nothing."""
    t = du.make_inputs(1, 100, 1, 1, 64, 64, torch.bfloat16, seed=12)
    cu = torch.tensor([10, 45, 77], dtype=torch.int32)
    o, ht = run(t, cu_seqlens=cu.cuda(), final_state=True)
    for n in du.NAMES:
        t[n][0, :10] = float("nan")
        t[n][0, 77:] = float("inf")
    o2, ht2 = run(t, cu_seqlens=cu.cuda(), final_state=True)
    assert torch.equal(o2[0, 10:77], o[0, 10:77]) and torch.equal(ht2, ht)


# ---- the form for single tokens -----------------------------------------------------------
STEPS = [  # B, T, HK, H, DK, DV, slots
    (1, 1, 1, 1, 1, 1, 0), (1, 1, 2, 4, 128, 128, 0), (3, 1, 1, 3, 64, 31, 0),
    (5, 4, 2, 2, 32, 64, 9), (2, 7, 1, 2, 80, 100, 2), (4, 2, 1, 1, 127, 6, 6),
    (70, 1, 1, 2, 64, 64, 90),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", STEPS)
def test_step(shape, dtype):
    B, T, HK, H, DK, DV, slots = shape
    t = du.make_inputs(B, T, HK, H, DK, DV, dtype, seed=B + T, h0=slots or B)
    d = du.to_gpu(t)
    at = torch.randperm(slots, generator=torch.Generator().manual_seed(1))[:B] if slots else None
    state = d["h0"].clone()
    o = ss.ss1d_delta_step(*[d[n] for n in du.NAMES], state,
                           slots=at.to(torch.int32).cuda() if slots else None)
    ref_state = t["h0"].double()
    rows = at if slots else torch.arange(B)
    t["h0"] = t["h0"][rows]
    ref_o, ends = du.reference(t, DK ** -0.5)
    ref_state[rows] = ends
    du.check(o, ref_o, "o", du.f32_bound(DK, ref_o),
             du.BF16_HALF if dtype == torch.bfloat16 else 0.0)
    du.check(state, ref_state, "state", du.f32_bound(DK, ref_state))
    untouched = torch.ones(state.shape[0], dtype=torch.bool)
    untouched[rows] = False
    assert torch.equal(state[untouched.cuda()], d["h0"][untouched.cuda()])


def test_step_with_padding_and_repeated_slots():
    """Padded rows leave o and every state alone; rows of one slot are successive tokens."""
    dtype = torch.float32
    t = du.make_inputs(8, 2, 1, 2, 64, 64, dtype, seed=3, h0=4)
    slots = torch.tensor([2, -1, 0, 2, 4, 2, 0, 9], dtype=torch.int32)
    d = du.to_gpu(t)
    state, o = d["h0"].clone(), torch.full((8, 2, 2, 64), 5.0, device="cuda")
    ss.ss1d_delta_step(*[d[n] for n in du.NAMES], state, slots=slots.cuda(), o=o)
    ref = t["h0"].double()
    for b in range(8):
        s = int(slots[b])
        if not 0 <= s < 4:
            assert (o[b] == 5).all()
            continue
        x = [t[n][b].double() for n in du.NAMES]
        ro, ref[s], _ = du.rule(*x, 64 ** -0.5, ref[s])
        du.check(o[b], ro, f"o of row {b}", du.f32_bound(64, ro))
    du.check(state, ref, "state", du.f32_bound(64, ref))
    assert torch.equal(state[1], d["h0"][1]) and torch.equal(state[3], d["h0"][3])


@pytest.mark.parametrize("dtype", TYPES)
def test_prompt_then_steps(dtype):
    """A run as serving makes it: packed prompts, then tokens one by one on the pooled states."""
    cu = torch.tensor([0, 40, 73], dtype=torch.int32)
    t = du.make_inputs(1, 73 + 2 * 6, 2, 4, 64, 64, dtype, seed=4)
    d = du.to_gpu(t)
    o, state = ss.ss1d_delta_forward(*[d[n] for n in du.NAMES], cu_seqlens=cu.cuda(),
                                     final_state=True)
    for i in range(6):
        rows = [d[n][0, 73 + 2 * i:75 + 2 * i].unsqueeze(1) for n in du.NAMES]
        o[0, 73 + 2 * i:75 + 2 * i] = ss.ss1d_delta_step(
            *rows, state, slots=torch.tensor([0, 1], dtype=torch.int32, device="cuda"))[:, 0]
    for s, (a, e) in enumerate(((0, 40), (40, 73))):
        idx = list(range(a, e)) + [73 + 2 * i + s for i in range(6)]
        x = [t[n][0][idx].double() for n in du.NAMES]
        ref_o, ref_s, _ = du.rule(*x, 64 ** -0.5, torch.zeros(4, 64, 64).double())
        du.check(o[0][idx], ref_o, "o", *du.o_bounds(64, ref_o, dtype))
        du.check(state[s], ref_s, "state", du.f32_bound(64, ref_s))


# ---- streams, graphs ----------------------------------------------------------------------
def test_graph_replays():
    """Forward and step in one captured graph, replayed on new inputs with eager work between."""
    t = du.to_gpu(du.make_inputs(2, 90, 1, 2, 64, 64, torch.bfloat16, seed=13, h0=2))
    tok = du.to_gpu(du.make_inputs(2, 1, 1, 2, 64, 64, torch.bfloat16, seed=14))
    seq, one = [t[n] for n in du.NAMES], [tok[n] for n in du.NAMES]

    def work():
        o, state = ss.ss1d_delta_forward(*seq, initial_state=t["h0"], final_state=True)
        return o, ss.ss1d_delta_step(*one, state), state

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = work()
    for i in range(3):
        t["v"].copy_(torch.randn_like(t["v"]))
        t["h0"].copy_(torch.randn_like(t["h0"]))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        for x, y in zip(got, work()):
            assert torch.equal(x, y), i
        torch.cuda.synchronize()


def test_two_streams_at_once():
    ts = [du.to_gpu(du.make_inputs(2, 300, 1, 2, 64, 64, torch.bfloat16, seed=20 + i)) for i in (0, 1)]
    want = [ss.ss1d_delta_forward(*[t[n] for n in du.NAMES]) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(3):
        got = [ss.ss1d_delta_forward(*[t[n] for n in du.NAMES], stream=s)
               for t, s in zip(ts, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
