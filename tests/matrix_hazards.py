"""Wait states between matrix instructions and the first use of their results, in the code that
the compiler made for the library's kernels.

A matrix instruction writes its registers some wait states after it is issued, and nothing in the
hardware holds back an instruction that touches them earlier: the compiler has to count the
instructions in between, on every path.  This walks every path of a kernel and reports registers
that are touched too early.
"""
from __future__ import annotations

import pathlib
import re
import shutil
import struct
import subprocess
import tempfile

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
# Wait states that the compiler itself puts between the instruction and a use of its result in
# straight-line code (one per instruction, s_nop n counts n + 1).
NEEDED = {"v_mfma_f32_32x32x16_bf16": 12, "v_mfma_f32_32x32x2_f32": 18,
          "v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10}
_REGISTERS = re.compile(r"([va])(?:(\d+)|\[(\d+):(\d+)\])(?!\w)")
_TARGET = re.compile(r"<([^>]+)\+0x([0-9a-f]+)>")


def tool(name):
    return shutil.which(name) or f"/opt/rocm/llvm/bin/{name}"


def disassembly(library):
    """The text of every gfx950 code object in the library."""
    with tempfile.TemporaryDirectory() as d:
        d = pathlib.Path(d)
        subprocess.run([tool("llvm-objcopy"), "--dump-section", f".hip_fatbin={d}/fat", str(library),
                        "/dev/null"], check=True)
        data, at = (d / "fat").read_bytes(), 0
        while (at := data.find(MAGIC, at)) >= 0:
            count, = struct.unpack_from("<Q", data, at + len(MAGIC))
            p = at + len(MAGIC) + 8
            for _ in range(count):
                offset, size, length = struct.unpack_from("<QQQ", data, p)
                name = data[p + 24:p + 24 + length].decode()
                p += 24 + length
                if "gfx950" in name and size:
                    (d / "object").write_bytes(data[at + offset:at + offset + size])
                    yield subprocess.run([tool("llvm-objdump"), "-d", "--no-show-raw-insn", str(d / "object")],
                                         check=True, capture_output=True, text=True).stdout
            at += len(MAGIC)


def functions(text):
    """(name, instructions) of a disassembly: (offset in the function, text, branch target)."""
    name, start, body = None, None, []
    for line in text.splitlines():
        if line.endswith(">:"):
            if name:
                yield name, body
            name, start, body = line[line.index("<") + 1:-2], None, []
        elif name and "//" in line:
            code, note = line.split("//", 1)
            where = int(note.split(":")[0], 16)
            start = where if start is None else start
            target = _TARGET.search(note) if "branch" in code else None
            body.append((where - start, code.strip(), int(target.group(2), 16) if target else
                         (0 if "branch" in code else None)))
    if name:
        yield name, body


def registers(operand):
    out = []
    for kind, one, first, last in _REGISTERS.findall(operand):
        out += [(kind, i) for i in (range(int(first), int(last) + 1) if first else [int(one)])]
    return out


def touched(code):
    """An instruction's operands as lists of registers, the result first."""
    op, _, rest = code.partition(" ")
    return op, [registers(x) for x in rest.split(",")]


def early_uses(body):
    """Uses of a matrix instruction's result that some path reaches too early: (instruction,
    the matrix instruction, wait states short)."""
    index = {offset: i for i, (offset, _, _) in enumerate(body)}
    leaders = {0} | {index[t] for _, _, t in body if t is not None} \
        | {i + 1 for i, (_, _, t) in enumerate(body) if t is not None and i + 1 < len(body)}
    parsed = [touched(code) for _, code, _ in body]
    entry, work, found = {0: {}}, [0], {}
    while work:
        i = work.pop()
        waiting = dict(entry[i])  # register -> (wait states still needed, the instruction)
        while True:
            offset, code, target = body[i]
            op, operands = parsed[i]
            matrix = op.startswith("v_mfma")
            if waiting:
                use = operands
                if matrix:  # the matrix core itself keeps the order of sums and results
                    whole = touched(waiting[operands[3][0]][1])[1][0] if operands[3] and \
                        operands[3][0] in waiting else operands[3]
                    use = operands[1:3] + ([] if operands[3] == whole else operands[3:4])
                for r in (r for x in use for r in x):
                    if r in waiting:
                        found[code] = (offset, code, waiting[r][1], waiting[r][0])
                step = int(code.split()[1]) + 1 if op == "s_nop" else 1
                waiting = {r: (n - step, w) for r, (n, w) in waiting.items() if n > step}
            if matrix:
                waiting.update({r: (NEEDED[op], code) for r in operands[0]})
            nexts = []
            if target is not None:
                nexts.append(index[target])
            last = op in ("s_endpgm", "s_branch", "s_setpc_b64") or i + 1 == len(body)
            if not last and i + 1 in leaders:
                nexts.append(i + 1)
            for n in nexts:
                old = entry.get(n)
                new = dict(old or {})
                for r, v in waiting.items():
                    if r not in new or new[r][0] < v[0]:
                        new[r] = v
                if old is None or new != old:
                    entry[n] = new
                    if n not in work:
                        work.append(n)
            if last or i + 1 in leaders:
                break
            i += 1
    return list(found.values())
