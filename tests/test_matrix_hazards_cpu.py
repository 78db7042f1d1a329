"""No kernel of the built library touches a matrix instruction's result too early."""
import concurrent.futures

import pytest

from selective_scan_ss2d_amd import _binding as bnd
from tests import matrix_hazards as mh


def check(text):
    """(kernels with matrix instructions, what they touch too early)."""
    kernels, bad = 0, []
    for name, body in mh.functions(text):
        if any(code.startswith("v_mfma") for _, code, _ in body):
            kernels += 1
            bad += [(name, *x) for x in mh.early_uses(body)]
    return kernels, bad


def test_the_librarys_kernels():
    if not bnd.LIBRARY_PATH.exists():
        from selective_scan_ss2d_amd import build
        build.build()
    texts = [t for t in mh.disassembly(bnd.LIBRARY_PATH) if "v_mfma" in t]
    with concurrent.futures.ProcessPoolExecutor(max_workers=4) as pool:
        results = list(pool.map(check, texts))
    assert sum(k for k, _ in results) > 100
    assert not [b for _, bad in results for b in bad]


def lines(*codes):
    """A disassembly of one function, 4 bytes an instruction."""
    out = ["0000000000001000 <k>:"]
    for i, code in enumerate(codes):
        note = ""
        if "branch" in code:
            code, target = code.split("->")
            note = f" <k+0x{4 * int(target):x}>" if int(target) else " <k>"
        out.append(f"\t{code.strip()}    // {0x1000 + 4 * i:012X}: 00000000{note}")
    return "\n".join(out)


P = "v_mfma_f32_32x32x16_bf16 v[0:15], v[20:23], v[24:27], 0"
F = "v_mfma_f32_32x32x2_f32 a[0:15], v20, v24, a[0:15]"


@pytest.mark.parametrize("codes, early", [
    ((P, "s_nop 11", "v_add_f32_e32 v30, 1.0, v3", "s_endpgm"), False),
    ((P, "s_nop 10", "v_add_f32_e32 v30, 1.0, v3", "s_endpgm"), True),
    ((P, "s_nop 10", "global_store_dwordx4 v40, v[12:15], s[0:1]", "s_endpgm"), True),
    ((P, "s_nop 10", "v_add_f32_e32 v30, 1.0, v16", "s_endpgm"), False),
    ((F, F, "s_nop 15", "s_nop 1", "v_accvgpr_read_b32 v1, a7", "s_endpgm"), False),
    ((F, F, "s_nop 15", "s_nop 0", "v_accvgpr_read_b32 v1, a7", "s_endpgm"), True),
    # operands of another product are uses as well
    ((P, P.replace("v[0:15], v[20:23]", "v[32:47], v[8:11]"), "s_endpgm"), True),
    # a short block that one path jumps over: its instructions do not count there
    ((P, "s_cbranch_scc1 2 -> 4", "s_nop 5", "s_nop 5", "v_add_f32_e32 v30, 1.0, v3", "s_endpgm"), True),
    ((P, "s_cbranch_scc1 2 -> 4", "s_nop 5", "s_nop 5", "s_nop 10", "v_add_f32_e32 v30, 1.0, v3", "s_endpgm"), False),
    # around a loop
    (("s_nop 0", "v_add_f32_e32 v30, 1.0, v3", P, "s_cbranch_scc1 65533 -> 0", "s_endpgm"), True),
    (("s_nop 10", "v_add_f32_e32 v30, 1.0, v3", P, "s_cbranch_scc1 65533 -> 0", "s_endpgm"), False),
])
def test_the_check_itself(codes, early):
    kernels, bad = check(lines(*codes))
    assert kernels == 1 and bool(bad) == early
