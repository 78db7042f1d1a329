"""Refusals of the gated delta rule's C entry points (no GPU: nothing is launched)."""
import ctypes

import pytest

from selective_scan_ss2d_amd import _binding as bnd


@pytest.fixture(scope="module")
def lib():
    if not bnd.LIBRARY_PATH.exists():
        from selective_scan_ss2d_amd import build
        build.build()
    return bnd.load_library()


def ptrs(n):  # fake device addresses, never dereferenced
    return [(1 << 40) + i * (1 << 36) for i in range(n)]


def forward(lib, p, B=1, L=64, S=1, HK=2, H=4, DK=64, DV=64, strides=None, scale=1.0, dtype=1):
    return lib.ss1d_delta_forward(*p, B, L, S, HK, H, DK, DV, strides, scale, dtype, None)


def args(h0=False, cu=False, ht=False, saved=False):
    p = ptrs(10)
    for i, on in ((5, h0), (6, cu), (8, ht), (9, saved)):
        if not on:
            p[i] = None
    return p


def step(lib, p, B=2, T=1, S=2, HK=2, H=4, DK=64, DV=64, strides=None, scale=1.0, dtype=1):
    return lib.ss1d_delta_step(*p, B, T, S, HK, H, DK, DV, strides, scale, dtype, None)


BAD = [
    (dict(dtype=2), "UNSUPPORTED"), (dict(DK=129), "UNSUPPORTED"), (dict(DK=0), "SHAPE"),
    (dict(DV=0), "SHAPE"), (dict(HK=0), "SHAPE"), (dict(HK=3), "SHAPE"), (dict(B=-1), "SHAPE"),
    (dict(scale=float("nan")), "UNSUPPORTED"), (dict(scale=float("inf")), "UNSUPPORTED"),
    (dict(DV=1 << 20), "SHAPE"),
]


@pytest.mark.parametrize("change, code", BAD)
def test_sizes_refused(lib, change, code):
    want = getattr(bnd, "SS2D_ERR_" + code)
    assert forward(lib, args(), **change) == want
    assert step(lib, ptrs(8), **change) == want


def test_rows_past_32_bit_offsets_refused(lib):
    wide = dict(L=1, HK=1 << 18, H=1 << 18, DK=128, DV=1)
    assert forward(lib, args(), **wide) == bnd.SS2D_ERR_UNSUPPORTED
    assert forward(lib, args(), L=1, HK=1, H=1 << 18, DK=8, DV=128) == bnd.SS2D_ERR_UNSUPPORTED


def test_sequences_refused(lib):
    assert forward(lib, args(), S=2) == bnd.SS2D_ERR_SHAPE                # dense: S is B
    assert forward(lib, args(cu=True), B=2, S=3) == bnd.SS2D_ERR_SHAPE    # packed: B is 1
    assert forward(lib, args(), L=-1) == bnd.SS2D_ERR_SHAPE
    assert forward(lib, args(), L=1 << 39, H=4096, HK=1) == bnd.SS2D_ERR_SHAPE  # a launch too large
    p = ptrs(8)
    p[6] = None
    assert step(lib, p, B=3, S=2) == bnd.SS2D_ERR_SHAPE  # no slots: row b needs state b


@pytest.mark.parametrize("i", [0, 1, 2, 3, 4, 7])
def test_null_pointers(lib, i):
    p = args()
    p[i] = None
    assert forward(lib, p) == bnd.SS2D_ERR_NULL


@pytest.mark.parametrize("i", [0, 1, 2, 3, 4, 5, 7])
def test_null_pointers_step(lib, i):
    p = ptrs(8)
    p[i] = None
    assert step(lib, p) == bnd.SS2D_ERR_NULL


def test_misaligned(lib):
    for i in range(10):
        p = args(True, True, True, True)
        p[i] += 1
        assert forward(lib, p) == bnd.SS2D_ERR_ALIGN, i
    p = args(saved=True)
    p[9] += 128
    assert forward(lib, p) == bnd.SS2D_ERR_ALIGN
    for i in range(8):
        p = ptrs(8)
        p[i] += 1
        assert step(lib, p) == bnd.SS2D_ERR_ALIGN, i


def test_outputs_over_inputs(lib):
    for out in (7, 8, 9):
        for i in range(10):
            if i == out or (out == 8 and i == 5):
                continue
            p = args(True, True, True, True)
            p[out] = p[i]
            assert forward(lib, p) == bnd.SS2D_ERR_ALIAS, (out, i)
    p = args(h0=True, ht=True)
    p[8] = p[5] + 256  # over the initial states, but not in place
    assert forward(lib, p) == bnd.SS2D_ERR_ALIAS
    for out in (5, 7):
        for i in range(8):
            if i != out:
                p = ptrs(8)
                p[out] = p[i]
                assert step(lib, p) == bnd.SS2D_ERR_ALIAS, (out, i)


def backward(lib, p, B=1, L=64, S=1, HK=2, H=4, DK=64, DV=64, strides=None, scale=1.0, dtype=1):
    return lib.ss1d_delta_backward(*p, B, L, S, HK, H, DK, DV, strides, scale, dtype, None)


def test_backward_refusals(lib):
    for change, code in BAD:
        assert backward(lib, ptrs(16), S=1, **dict(change)) != bnd.SS2D_OK
    optional = (5, 6, 7, 9, 15)
    dense = ptrs(16)
    dense[6] = None
    for i in range(16):
        if i not in optional:
            p = list(dense)
            p[i] = None
            assert backward(lib, p) == bnd.SS2D_ERR_NULL, i
        p = ptrs(16)
        p[i] += 1
        assert backward(lib, p) == bnd.SS2D_ERR_ALIGN, i
    for out in range(10, 16):
        for i in range(16):
            if i != out:
                p = ptrs(16)
                p[out] = p[i]
                assert backward(lib, p) == bnd.SS2D_ERR_ALIAS, (out, i)


def test_strides(lib):
    def st(*v):
        return (ctypes.c_int64 * 9)(*v)
    base = [64 * 2 * 64, 128, 64] * 2 + [64 * 4 * 64, 256, 64]
    for i in range(9):
        bad = list(base)
        bad[i] = -64
        assert forward(lib, args(), B=2, S=2, strides=st(*bad)) == bnd.SS2D_ERR_SHAPE, i
        bad[i] = 1 << 61
        assert forward(lib, args(), B=2, S=2, strides=st(*bad)) == bnd.SS2D_ERR_SHAPE, i
    # the extent of a strided input counts for the overlap checks
    p = args()
    p[7] = p[0] + 63 * 100000 * 2
    wide = list(base)
    wide[1] = 100000
    assert forward(lib, p, strides=st(*wide)) == bnd.SS2D_ERR_ALIAS


def test_nothing_to_do(lib):
    none = [None] * 10
    assert forward(lib, none, B=0, S=0) == bnd.SS2D_OK
    assert forward(lib, none, H=0) == bnd.SS2D_OK
    assert forward(lib, none, L=0) == bnd.SS2D_OK
    assert step(lib, [None] * 8, B=0, S=0) == bnd.SS2D_OK
    assert step(lib, [None] * 8, T=0) == bnd.SS2D_OK


def test_saved_bytes(lib):
    def aligned(x):
        return (x + 255) // 256 * 256
    n = lib.ss1d_delta_saved_bytes(3, 130, 3, 4, 64, 32, 0)
    assert n == aligned(3 * 3 * 4 * 64 * 32 * 4) + aligned(3 * 4 * 64 * 32 * 4) + 2 * aligned(3 * 130 * 4 * 32 * 4)
    n = lib.ss1d_delta_saved_bytes(1, 130, 5, 4, 64, 32, 1)
    assert n == aligned((2 + 5) * 4 * 64 * 32 * 4) + aligned(5 * 4 * 64 * 32 * 4) + 2 * aligned(130 * 4 * 32 * 4)
    assert lib.ss1d_delta_saved_bytes(1, 130, 2, 4, 64, 32, 0) == -1
    assert lib.ss1d_delta_saved_bytes(1, 130, 1, 4, 200, 32, 0) == -1


def test_binding_refuses():
    import torch
    import selective_scan_ss2d_amd as ss
    t = torch.zeros(1, 4, 1, 8)
    with pytest.raises(ValueError, match="GPU"):
        ss.ss1d_delta_forward(t, t, t, t[..., 0], t[..., 0])
    with pytest.raises(TypeError):
        ss.ss1d_delta_forward(None, t, t, t, t)
    with pytest.raises(ValueError):
        ss.ss1d_delta_step(t[0], t, t, t, t, t)


def test_launches_past_64_bits_refused(lib):
    """The threads of a launch are counted without passing 64 bits themselves: 64 * 9 of each
    sequence and head here, 2^64 and a few million in all."""
    H = 30000
    S = -(-(1 << 64) // (576 * H))
    assert forward(lib, args(ht=True), B=S, S=S, L=0, HK=1, H=H, DK=1, DV=1) == bnd.SS2D_ERR_SHAPE
