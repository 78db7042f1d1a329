"""The caller's scratch of the gated delta rule and the block norm: sizes and refusals (no GPU:
nothing is launched)."""
import pytest

from selective_scan_ss2d_amd import _binding as bnd

SIZES = [(1, 64, 1, 2, 4, 64, 64), (2, 300, 2, 1, 3, 128, 96), (3, 1, 3, 1, 1, 8, 8), (1, 5000, 1, 1, 1, 64, 32)]


@pytest.fixture(scope="module")
def lib():
    if not bnd.LIBRARY_PATH.exists():
        from selective_scan_ss2d_amd import build
        build.build()
    return bnd.load_library()


def ptrs(n):  # fake device addresses, never dereferenced
    return [(1 << 40) + i * (1 << 36) for i in range(n)]


def forward(lib, p, nbytes, size, dtype=1):
    return lib.ss1d_delta_forward_ws(*p, nbytes, *size, None, 1.0, dtype, None)


def backward(lib, p, nbytes, size, dtype=1):
    return lib.ss1d_delta_backward_ws(*p, nbytes, *size, None, 1.0, dtype, None)


def norm(lib, p, nbytes, B=4, L=16, D=64, G=2, first=0):
    return lib.ss2d_norm_backward_ws(*p, nbytes, B, L, D, G, first, 1, 1e-6, 1, 0, None)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("size", SIZES)
def test_too_little(lib, size, dtype):
    for kept in (0, 1):
        f = ptrs(11)
        f[6] = None
        f[9] = f[9] if kept else None
        need = lib.ss1d_delta_scratch_bytes(0, kept, *size, dtype, 0)
        assert need > 0 and forward(lib, f, need - 1, size, dtype) == bnd.SS2D_ERR_SCRATCH
        assert forward(lib, f, -1, size, dtype) == bnd.SS2D_ERR_SCRATCH
        b = ptrs(17)
        b[6] = None
        b[7] = b[7] if kept else None
        more = lib.ss1d_delta_scratch_bytes(1, kept, *size, dtype, 0)
        assert more > need and backward(lib, b, more - 1, size, dtype) == bnd.SS2D_ERR_SCRATCH
    assert lib.ss1d_delta_scratch_bytes(1, 0, *size, dtype, 0) > lib.ss1d_delta_scratch_bytes(1, 1, *size, dtype, 0)


def test_too_little_for_the_norm(lib):
    for shape in (dict(), dict(G=1), dict(B=64, L=300, D=100, G=1), dict(B=8, L=50, D=96, G=4, first=1)):
        s = dict(dict(B=4, L=16, D=64, G=2, first=0), **shape)
        need = lib.ss2d_norm_scratch_bytes(s["B"], s["L"], s["D"], s["G"], s["first"])
        assert need >= 4 * s["D"] * 4
        assert norm(lib, ptrs(18), need - 1, **s) == bnd.SS2D_ERR_SCRATCH


def test_sizes_of_refused_calls(lib):
    assert lib.ss1d_delta_scratch_bytes(0, 0, 1, 64, 1, 2, 4, 200, 64, 1, 0) == -1
    assert lib.ss1d_delta_scratch_bytes(1, 0, 2, 64, 3, 2, 4, 64, 64, 1, 1) == -1
    assert lib.ss2d_norm_scratch_bytes(4, 16, 9000, 0, 0) == -1
    assert lib.ss2d_norm_scratch_bytes(4, 16, 64, 3, 0) == -1
    assert lib.ss2d_norm_scratch_bytes(0, 16, 64, 0, 0) == 0


def test_misaligned_or_overlapping(lib):
    size = (1, 64, 1, 2, 4, 64, 64)
    plenty = 1 << 30
    for make, n, at in ((lambda p: forward(lib, p, plenty, size), 11, 10),
                        (lambda p: backward(lib, p, plenty, size), 17, 16),
                        (lambda p: norm(lib, p, plenty), 18, 17)):
        p = ptrs(n)
        p[at] += 128
        assert make(p) == bnd.SS2D_ERR_ALIGN
        for i in range(n):
            if i != at:
                p = ptrs(n)
                p[at] = p[i]
                assert make(p) == bnd.SS2D_ERR_ALIAS, (n, i)
