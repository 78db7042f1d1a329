"""Which sizes and strides the C entry points of the token-order scan refuse (no GPU: every call here is
refused before anything is launched; one whose sizes pass is refused for an output over an input)."""
import ctypes

from selective_scan_ss2d_amd import _binding as bnd
from tests.test_token_ops_cpu import lib, ptrs, scan, scan_bwd, scan_step  # noqa: F401 (lib: the fixture)


def overlapping(n, out, over, without=()):
    p = ptrs(n, without)
    p[out] = p[over]
    return p


def calls(lib, **kw):  # noqa: F811
    """The codes of a forward, a backward and a step."""
    L = kw.pop("L")
    return (scan(lib, overlapping(14, 10, 0, (9,)), L=L, **kw), scan_bwd(lib, overlapping(23, 13, 0, (9,)), L=L, **kw),
            scan_step(lib, overlapping(11, 10, 0), T=L, **kw))


def test_strides_of_one_token_or_group_are_free(lib):  # noqa: F811
    shape, alias = (bnd.SS2D_ERR_SHAPE,) * 3, (bnd.SS2D_ERR_ALIAS,) * 3

    def strides(L, G, token=None, group=None):
        t, w = token or 64, token or G * 16
        return (ctypes.c_int64 * 12)(*[L * 64, t] * 3, *[L * G * 16, w, group or 16] * 2)

    wide = (1 << 24) + 64
    assert calls(lib, L=1, strides=strides(1, 2)) == alias
    assert calls(lib, L=1, strides=strides(1, 2, token=wide)) == alias
    assert calls(lib, L=2, strides=strides(2, 2, token=wide)) == shape
    assert calls(lib, L=3, G=1, strides=strides(3, 1, group=wide)) == alias
    assert calls(lib, L=3, G=2, strides=strides(3, 2, group=wide)) == shape
    assert calls(lib, L=1, G=1, strides=strides(1, 1, token=1 << 61, group=1 << 61)) == alias
    assert calls(lib, L=1, strides=strides(1, 2, token=-64)) == shape
    assert calls(lib, L=3, G=1, strides=strides(3, 1, group=-16)) == shape


def test_launches_are_limited_by_the_threads_that_they_take(lib):  # noqa: F811
    ALIAS, SHAPE = bnd.SS2D_ERR_ALIAS, bnd.SS2D_ERR_SHAPE

    def both(packed=False, **kw):
        cu = () if packed else (9,)
        return scan(lib, overlapping(14, 10, 0, cu), **kw), scan_bwd(lib, overlapping(23, 13, 0, cu), **kw)

    # S D N past 2^32 where nothing is joined, and up to 2^24 blocks of 64 channels
    assert both(B=70000, S=70000, L=2, D=4096, G=1) == (ALIAS, ALIAS)
    assert both(B=1 << 17, S=1 << 17, L=2, D=8128, G=1) == (ALIAS, ALIAS)  # 127 blocks each
    assert both(B=1 << 17, S=1 << 17, L=2, D=8192, G=1) == (SHAPE, SHAPE)
    # 2^29 tokens; their sums of dB and dC take 2^25 blocks
    assert both(True, B=1, S=4, L=1 << 29, D=64, G=1) == (ALIAS, SHAPE)
    assert both(True, B=1, S=4, L=1 << 27, D=64, G=1) == (ALIAS, ALIAS)
    # columns of the parameters' sums
    assert both(B=1, S=1, L=1, D=1 << 23, N=32) == (ALIAS, SHAPE)
    assert both(B=1, S=1, L=1, D=7 << 20, N=32) == (ALIAS, ALIAS)
