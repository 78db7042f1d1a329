"""Refusals and sizes of the C entry points of the token-order scan, its convolution and the group
norm (no GPU: nothing is launched), and of their bindings."""
import ctypes

import pytest
import torch

import selective_scan_ss2d_amd as ss
from selective_scan_ss2d_amd import _binding as bnd
from selective_scan_ss2d_amd import _call


@pytest.fixture(scope="module")
def lib():
    if not bnd.LIBRARY_PATH.exists():
        from selective_scan_ss2d_amd import build
        build.build()
    return bnd.load_library()


def ptrs(n, without=()):  # fake device addresses, never dereferenced
    return [None if i in without else (1 << 40) + i * (1 << 36) for i in range(n)]


def aligned(x):
    return (x + 255) // 256 * 256


PLENTY = 1 << 34

# u dt A B C D bias z h0 cu | y ht saved scratch
def scan(lib, p, nbytes=PLENTY, B=2, L=300, S=2, D=64, G=2, N=16, strides=None, dtype=1):
    return lib.ss1d_scan_forward(*p, nbytes, B, L, S, D, G, N, strides, dtype, None)


# u dt A B C D bias z h0 cu saved dy dht | du ddt dA dB dC dD dbias dz dh0 scratch
def scan_bwd(lib, p, nbytes=PLENTY, B=2, L=300, S=2, D=64, G=2, N=16, strides=None, dtype=1):
    return lib.ss1d_scan_backward(*p, nbytes, B, L, S, D, G, N, strides, dtype, None)


# u dt A B C D bias z | state slots y
def scan_step(lib, p, B=2, T=1, S=2, D=64, G=2, N=16, strides=None, dtype=1):
    return lib.ss1d_scan_step(*p[:8], p[8], p[9], p[10], B, T, S, D, G, N, strides, dtype, None)


# x w b h0 cu | y ht
def conv(lib, p, B=2, L=300, S=2, D=64, KW=4, strides=None, dtype=1):
    return lib.ss1d_conv_forward(*p, B, L, S, D, KW, strides, 1, dtype, None)


# x w b h0 cu dy dht | dx dw db dh0 scratch
def conv_bwd(lib, p, nbytes=PLENTY, B=2, L=300, S=2, D=64, KW=4, strides=None, dtype=1):
    return lib.ss1d_conv_backward(*p, nbytes, B, L, S, D, KW, strides, 1, dtype, None)


# x w b state slots y
def conv_step(lib, p, B=2, T=1, S=2, D=64, KW=4, strides=None, dtype=1):
    return lib.ss1d_conv_step(*p, B, T, S, D, KW, strides, 1, dtype, None)


# x w b | y stats scratch
def group(lib, p, nbytes=PLENTY, B=2, L=300, C=64, G=4, eps=1e-5, dtype=1):
    return lib.ss2d_group_norm_forward(*p, nbytes, B, L, C, G, 1, eps, dtype, None)


# x w b stats dy | dx dw db scratch
def group_bwd(lib, p, nbytes=PLENTY, B=2, L=300, C=64, G=4, eps=1e-5, dtype=1):
    return lib.ss2d_group_norm_backward(*p, nbytes, B, L, C, G, 1, eps, dtype, None)


# call, pointers without cu, optional pointers, outputs, inputs that an output may be
CALLS = {
    "scan": (scan, ptrs(14, (9,)), (7, 8, 11, 12, 13), (10, 11, 12, 13), {(11, 8)}),
    "scan_bwd": (scan_bwd, ptrs(23, (9,)), (8, 10, 12, 21, 22), tuple(range(13, 23)), set()),
    "scan_step": (scan_step, ptrs(11), (7, 9), (8, 10), set()),
    "conv": (conv, ptrs(7, (4,)), (2, 3, 6), (5, 6), {(6, 3)}),
    "conv_bwd": (conv_bwd, ptrs(12, (4,)), (3, 6, 10, 11), tuple(range(7, 12)), set()),
    "conv_step": (conv_step, ptrs(6), (2, 4), (3, 5), set()),
    "group": (group, ptrs(6), (1, 2, 4, 5), (3, 4, 5), set()),
    "group_bwd": (group_bwd, ptrs(9), (3, 8), (5, 6, 7, 8), set()),
}


@pytest.mark.parametrize("name", CALLS)
def test_null_pointers(lib, name):
    call, p, optional, _, _ = CALLS[name]
    for i in range(len(p)):
        if p[i] is None or i in optional:
            continue
        q = list(p)
        q[i] = None
        assert call(lib, q) == bnd.SS2D_ERR_NULL, i


@pytest.mark.parametrize("name", CALLS)
def test_misaligned(lib, name):
    call, p, *_ = CALLS[name]
    for i in range(len(p)):
        if p[i] is not None:
            q = list(p)
            q[i] += 1
            assert call(lib, q) == bnd.SS2D_ERR_ALIGN, i


@pytest.mark.parametrize("name", CALLS)
def test_outputs_over_other_arguments(lib, name):
    call, p, _, outs, allowed = CALLS[name]
    scratch = name == "group"  # a forward in one launch needs none: nothing to overlap
    for out in outs:
        for i in range(len(p)):
            if i == out or p[i] is None or (out, i) in allowed or (i, out) in allowed:
                continue
            if scratch and 5 in (out, i):
                continue
            q = list(p)
            q[out] = p[i]
            assert call(lib, q) == bnd.SS2D_ERR_ALIAS, (out, i)


def test_states_in_place_wholly_or_not_at_all(lib):
    for call, p, ht, h0 in ((scan, ptrs(14, (9,)), 11, 8), (conv, ptrs(7, (4,)), 6, 3)):
        p[ht] = p[h0] + 256
        assert call(lib, p) == bnd.SS2D_ERR_ALIAS
    p = ptrs(14, (9,))
    p[11] = p[8]
    p[10] = p[8] + 256
    assert scan(lib, p) == bnd.SS2D_ERR_ALIAS


@pytest.mark.parametrize("change, code", [
    (dict(dtype=2), "UNSUPPORTED"), (dict(N=33), "UNSUPPORTED"), (dict(N=0), "SHAPE"), (dict(G=0), "SHAPE"),
    (dict(G=3), "SHAPE"), (dict(B=-1), "SHAPE"), (dict(D=-2), "SHAPE"), (dict(D=(1 << 24) + 2), "SHAPE"),
    (dict(D=1 << 24, B=1 << 38, S=1 << 38), "SHAPE")])
def test_scan_sizes(lib, change, code):
    want = getattr(bnd, "SS2D_ERR_" + code)
    assert scan(lib, ptrs(14, (9,)), **change) == want
    assert scan_bwd(lib, ptrs(23, (9,)), **change) == want
    assert scan_step(lib, ptrs(11), **change) == want
    sizes = dict(B=2, L=300, S=2, D=64, G=2, N=16, dtype=1)
    sizes.update(change)
    assert lib.ss1d_scan_scratch_bytes(0, 0, *sizes.values(), 0) == -1


@pytest.mark.parametrize("change, code", [
    (dict(dtype=2), "UNSUPPORTED"), (dict(KW=9), "UNSUPPORTED"), (dict(KW=0), "SHAPE"), (dict(B=-1), "SHAPE"),
    (dict(D=-2), "SHAPE"), (dict(D=(1 << 24) + 2), "SHAPE"), (dict(D=1 << 24, B=1 << 38, S=1 << 38), "SHAPE")])
def test_conv_sizes(lib, change, code):
    want = getattr(bnd, "SS2D_ERR_" + code)
    assert conv(lib, ptrs(7, (4,)), **change) == want
    assert conv_bwd(lib, ptrs(12, (4,)), **change) == want
    assert conv_step(lib, ptrs(6), **change) == want


@pytest.mark.parametrize("change, code", [
    (dict(dtype=2), "UNSUPPORTED"), (dict(C=0), "SHAPE"), (dict(G=0), "SHAPE"), (dict(G=3), "SHAPE"),
    (dict(B=-1), "SHAPE"), (dict(L=-1), "SHAPE"), (dict(eps=-1.0), "UNSUPPORTED"),
    (dict(eps=float("nan")), "UNSUPPORTED"), (dict(eps=float("inf")), "UNSUPPORTED"),
    (dict(C=(1 << 20) + 4), "SHAPE"), (dict(L=1 << 31), "SHAPE"), (dict(B=1 << 40, L=1 << 30), "SHAPE"),
    (dict(B=1 << 24), "SHAPE")])
def test_group_sizes(lib, change, code):
    want = getattr(bnd, "SS2D_ERR_" + code)
    assert group(lib, ptrs(6), **change) == want
    assert group_bwd(lib, ptrs(9), **change) == want


def test_sequences(lib):
    dense, packed = ptrs(14, (9,)), ptrs(14)
    assert scan(lib, dense, S=3) == bnd.SS2D_ERR_SHAPE            # dense: S is B
    assert scan(lib, packed, B=2, S=3) == bnd.SS2D_ERR_SHAPE      # packed: B is 1
    assert conv(lib, ptrs(7, (4,)), S=3) == bnd.SS2D_ERR_SHAPE
    assert conv(lib, ptrs(7), B=2, S=3) == bnd.SS2D_ERR_SHAPE
    assert scan_step(lib, ptrs(11, (9,)), B=3, S=2) == bnd.SS2D_ERR_SHAPE  # no slots: row b needs state b
    assert conv_step(lib, ptrs(6, (4,)), B=3, S=2) == bnd.SS2D_ERR_SHAPE


def test_scan_strides(lib):
    # (batch, token) of u, dt_raw, z; (batch, token, group) of Bs, Cs
    base = [300 * 64, 64] * 3 + [300 * 32, 32, 16] * 2

    def call(values, p=None):
        st = (ctypes.c_int64 * 12)(*values)
        return scan(lib, p or ptrs(14, (9,)), strides=st), scan_bwd(lib, ptrs(23, (9,)), strides=st)

    for i in range(12):
        for bad in (-64, 1 << 61):
            values = list(base)
            values[i] = bad
            assert call(values) == (bnd.SS2D_ERR_SHAPE, bnd.SS2D_ERR_SHAPE), i
        if i not in (0, 2, 4, 6, 9):  # token and group strides keep to 32-bit offsets
            values = list(base)
            values[i] = (1 << 24) + 1
            assert call(values)[0] == bnd.SS2D_ERR_SHAPE, i
    p = ptrs(14, (9,))
    p[10] = p[0] + 299 * 100000 * 2  # the extent of a strided input counts for the overlap checks
    wide = list(base)
    wide[1] = 100000
    assert call(wide, p)[0] == bnd.SS2D_ERR_ALIAS


def test_conv_strides(lib):
    for values in ((-64, 64), (300 * 64, -64), (1 << 61, 64), (300 * 64, 1 << 61)):
        st = (ctypes.c_int64 * 2)(*values)
        assert conv(lib, ptrs(7, (4,)), strides=st) == bnd.SS2D_ERR_SHAPE
        assert conv_bwd(lib, ptrs(12, (4,)), strides=st) == bnd.SS2D_ERR_SHAPE


def test_nothing_to_do(lib):
    assert scan(lib, [None] * 14, B=0, S=0) == bnd.SS2D_OK
    assert scan(lib, [None] * 14, D=0) == bnd.SS2D_OK
    assert scan(lib, [None] * 14, L=0) == bnd.SS2D_OK
    assert scan_step(lib, [None] * 11, B=0, S=0) == bnd.SS2D_OK
    assert scan_step(lib, [None] * 11, T=0) == bnd.SS2D_OK
    assert conv(lib, [None] * 7, B=0, S=0) == bnd.SS2D_OK
    assert conv(lib, [None] * 7, L=0) == bnd.SS2D_OK
    assert conv_step(lib, [None] * 6, T=0) == bnd.SS2D_OK
    assert group(lib, [None] * 6, B=0) == bnd.SS2D_OK
    assert group(lib, [None] * 6, L=0) == bnd.SS2D_OK


@pytest.mark.parametrize("dtype", [0, 1])
def test_too_little_scratch(lib, dtype):
    sizes = (1, 4096, 1, 256, 1, 16)  # long and narrow: cut into segments
    need = lib.ss1d_scan_scratch_bytes(0, 0, *sizes, dtype, 0)
    kw = dict(zip(("B", "L", "S", "D", "G", "N"), sizes), dtype=dtype)
    assert need > 0 and scan(lib, ptrs(14, (9, 12)), need - 1, **kw) == bnd.SS2D_ERR_SCRATCH
    assert scan(lib, ptrs(14, (9, 12)), -1, **kw) == bnd.SS2D_ERR_SCRATCH
    kept, again = (lib.ss1d_scan_scratch_bytes(1, k, *sizes, dtype, 0) for k in (1, 0))
    assert scan_bwd(lib, ptrs(23, (9,)), kept - 1, **kw) == bnd.SS2D_ERR_SCRATCH
    assert again > kept and scan_bwd(lib, ptrs(23, (9, 10)), again - 1, **kw) == bnd.SS2D_ERR_SCRATCH
    need = lib.ss1d_conv_scratch_bytes(2, 300, 2, 64, 4, dtype, 0)
    assert need >= 5 * 64 * 4 and conv_bwd(lib, ptrs(12, (4,)), need - 1, dtype=dtype) == bnd.SS2D_ERR_SCRATCH
    for kept in (0, 1):
        need = lib.ss2d_group_norm_scratch_bytes(1, kept, 2, 300, 64, 4, dtype)
        assert need > 0 and group_bwd(lib, ptrs(9, () if kept else (3,)), 0, dtype=dtype) == bnd.SS2D_ERR_SCRATCH
    need = lib.ss2d_group_norm_scratch_bytes(0, 0, 1, 1 << 20, 8, 1, dtype)
    assert need > 0 and group(lib, ptrs(6, (4,)), need - 1, B=1, L=1 << 20, C=8, G=1, dtype=dtype) == bnd.SS2D_ERR_SCRATCH


def test_saved_bytes(lib):
    assert lib.ss1d_scan_saved_bytes(3, 130, 3, 40, 16, 0) == aligned(3 * 9 * 40 * 16 * 4)
    assert lib.ss1d_scan_saved_bytes(1, 130, 5, 40, 16, 1) == aligned((8 + 5) * 40 * 16 * 4)
    assert lib.ss1d_scan_saved_bytes(1, 130, 1, 40, 32, 0) == aligned(17 * 40 * 32 * 4)
    assert lib.ss1d_scan_saved_bytes(1, 130, 2, 40, 16, 0) == -1
    assert lib.ss1d_scan_saved_bytes(1, 130, 1, 40, 33, 0) == -1


def test_plans(lib):
    assert lib.ss1d_scan_set_plan(5, 0) == bnd.SS2D_ERR_UNSUPPORTED
    assert lib.ss1d_scan_set_plan(0, -2) == bnd.SS2D_ERR_SHAPE
    assert lib.ss1d_scan_set_plan(0, -1) == bnd.SS2D_OK


def test_launches_past_32_bits_refused(lib):
    assert scan(lib, ptrs(14, (9,)), B=1 << 30, S=1 << 30, L=1, D=64) == bnd.SS2D_ERR_SHAPE
    assert scan_step(lib, ptrs(11), B=1 << 30, T=1, D=64) == bnd.SS2D_ERR_SHAPE
    assert conv(lib, ptrs(7, (4,)), B=1 << 34, S=1 << 34, L=1, D=64) == bnd.SS2D_ERR_SHAPE
    assert conv_step(lib, ptrs(6), B=1 << 34, T=1, D=64) == bnd.SS2D_ERR_SHAPE


def test_bindings_refuse():
    t, f = torch.zeros(1, 4, 8), torch.zeros(8, 4)
    bc = torch.zeros(1, 4, 1, 4)
    with pytest.raises(ValueError, match="GPU"):
        ss.ss1d_scan_forward(t, t, f, bc, bc, t[0, 0], t[0, 0])
    with pytest.raises(TypeError):
        ss.ss1d_scan_step(None, t, f, bc, bc, t, t, t)
    with pytest.raises(ValueError):
        ss.ss1d_scan_backward(t[0], t, f, bc, bc, t, t, t)
    with pytest.raises(ValueError, match="GPU"):
        ss.ss1d_conv_forward(t, f)
    with pytest.raises(TypeError):
        ss.ss1d_conv_step(t, None, t)
    with pytest.raises(ValueError, match="GPU"):
        ss.ss2d_group_norm_forward(t, 2)
    with pytest.raises(TypeError, match="cu_seqlens"):
        _call.packed_sequences([0, 4], 1, torch.device("cuda", 0))


def test_rows():
    cpu, f32 = torch.device("cpu"), torch.float32
    wide = torch.zeros(2, 3, 10)
    assert _call.rows("x", torch.zeros(2, 3, 4), (2, 3, 4), f32, cpu) is True
    assert _call.rows("x", wide[..., 2:6], (2, 3, 4), f32, cpu) is False
    for bad, error in ((wide[..., ::2], ValueError), (wide.double()[..., :5], TypeError), (None, TypeError),
                       (wide[..., :4], ValueError)):
        with pytest.raises(error):
            _call.rows("x", bad, (2, 3, 5), f32, cpu)
