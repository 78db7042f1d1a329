"""Refusals of the block norm's C entry points (no GPU: nothing is launched)."""
import pytest

from selective_scan_ss2d_amd import _binding as bnd


@pytest.fixture(scope="module")
def lib():
    if not bnd.LIBRARY_PATH.exists():
        from selective_scan_ss2d_amd import build
        build.build()
    return bnd.load_library()


def ptrs(n):
    return [(1 << 40) + i * (1 << 36) for i in range(n)]


def forward(lib, p, B=4, L=16, D=64, G=2, first=0, layer=1, eps=1e-6, dtype=1, ytype=0):
    return lib.ss2d_norm_forward(*p, B, L, D, G, first, layer, eps, dtype, ytype, None)


def backward(lib, p, B=4, L=16, D=64, G=2, first=0, layer=1, eps=1e-6, dtype=1, ytype=0):
    return lib.ss2d_norm_backward(*p, B, L, D, G, first, layer, eps, dtype, ytype, None)


@pytest.mark.parametrize("change, code", [
    (dict(dtype=2), "UNSUPPORTED"), (dict(dtype=0, ytype=1), "UNSUPPORTED"),
    (dict(D=8193), "UNSUPPORTED"), (dict(D=1025, first=1), "UNSUPPORTED"), (dict(D=0), "SHAPE"),
    (dict(B=2, L=(1 << 24) + 1, D=4, first=1), "UNSUPPORTED"),
    (dict(B=-1), "SHAPE"), (dict(L=-1), "SHAPE"), (dict(G=-1), "SHAPE"), (dict(G=3), "SHAPE"),
    (dict(G=8, first=1), "SHAPE"), (dict(eps=-1.0), "UNSUPPORTED"),
    (dict(eps=float("nan")), "UNSUPPORTED"), (dict(B=1 << 40, L=1 << 30), "SHAPE")])
def test_sizes_refused(lib, change, code):
    want = getattr(bnd, "SS2D_ERR_" + code)
    assert forward(lib, ptrs(10), **change) == want
    assert backward(lib, ptrs(17), **change) == want


def test_forward_combinations(lib):
    def without(*idx):
        p = ptrs(10)
        for i in idx:
            p[i] = None
        return p
    for bad in ((0,), (8, 9), (6,), (9,), (3,), (4,), (6, 9)):
        assert forward(lib, without(*bad)) == bnd.SS2D_ERR_NULL, bad
    assert forward(lib, ptrs(10), G=0) == bnd.SS2D_ERR_NULL  # a scale without groups


def test_backward_combinations(lib):
    # h z scale w_post b_post w_pre y dy dn | dh dz dres dscale dw_post db_post dw_pre db_pre
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9, 10, 12, 13, 14, 15):
        p = ptrs(17)
        p[i] = None
        assert backward(lib, p) == bnd.SS2D_ERR_NULL, i


def test_alignment_and_overlap(lib):
    for i in range(10):
        p = ptrs(10)
        p[i] += 1
        assert forward(lib, p) == bnd.SS2D_ERR_ALIGN, i
    for i in range(17):
        p = ptrs(17)
        p[i] += 1
        assert backward(lib, p) == bnd.SS2D_ERR_ALIGN, i
    for out in (8, 9):
        for i in range(10):
            if i != out and (out, i) != (8, 2):
                p = ptrs(10)
                p[out] = p[i]
                assert forward(lib, p) == bnd.SS2D_ERR_ALIAS, (out, i)
    p = ptrs(10)
    p[8] = p[2] + 256  # over the residual, but not in place
    assert forward(lib, p) == bnd.SS2D_ERR_ALIAS
    for out in range(9, 17):
        for i in range(17):
            if i != out:
                p = ptrs(17)
                p[out] = p[i]
                assert backward(lib, p) == bnd.SS2D_ERR_ALIAS, (out, i)


def test_nothing_to_do(lib):
    assert forward(lib, [None] * 10, B=0) == bnd.SS2D_OK
    assert forward(lib, [None] * 10, L=0) == bnd.SS2D_OK


def test_binding_refuses():
    import torch
    import selective_scan_ss2d_amd as ss
    with pytest.raises(ValueError, match="GPU"):
        ss.ss2d_norm_forward(torch.zeros(2, 8), w_post=torch.ones(8))
    with pytest.raises(TypeError):
        ss.ss2d_norm_backward(None)
