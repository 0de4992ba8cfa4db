"""No kernel of the built library uses a matrix instruction's result before it is
there.

The hardware does not wait for it: between the instruction and one that is no
matrix instruction and reads or overwrites its result have to lie 8 wait states
(bfloat16, 16x16x32) or 10 (float32, 16x16x4), as many before a matrix instruction
takes it as an operand that is multiplied; for others 19, the most there is.  The
compiler counts them where control falls through, not everywhere along a branch
that is taken at once.  So this follows every path from every matrix instruction
through the disassembled library."""
import os
import re
import shutil
import struct
import subprocess

import pytest

from nonlinear_rnn_amd import build
from nonlinear_rnn_amd import pararnn as pr

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"
OBJDUMP = shutil.which("llvm-objdump") or "/opt/rocm/llvm/bin/llvm-objdump"
REGISTERS = re.compile(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b")
WAITS = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_16x16x4_f32": 10}


def device_code(path):
    """The code objects for the device in a shared library."""
    data = open(path, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        (entries,) = struct.unpack_from("<Q", data, at + 24)
        p = at + 32
        for _ in range(entries):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + length]
            p += 24 + length
            if build.ARCH.encode() in name and size:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, at + 24)


def registers(text):
    out = set()
    for m in REGISTERS.finditer(text):
        if m.group(1):
            out |= {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
        else:
            out.add((m.group(4), int(m.group(5))))
    return out


def functions(text):
    """(name, [(instruction, index of its branch's target or None)]) of those with
    matrix instructions."""
    for part in re.split(r"\n(?=[0-9a-f]{16} <)", text):
        head = re.match(r"\s*([0-9a-f]{16}) <(\S+)>:\n", part)
        if not head or "v_mfma" not in part:
            continue
        found, at = [], {}
        for m in re.finditer(r"^\t(\S.*?)\s*// ([0-9A-F]+):(.*)$", part, re.M):
            at[int(m.group(2), 16)] = len(found)
            target = re.search(r"<[^>+]*(?:\+0x([0-9a-f]+))?>", m.group(3))
            found.append((m.group(1), int(target.group(1) or "0", 16) if target else None))
        start = int(head.group(1), 16)
        yield head.group(2), [(i, None if t is None else at[start + t]) for i, t in found]


def early_uses(code):
    """(matrix instructions, [(one of them, what uses its result, wait states between)])."""
    count, found = 0, []
    for first, (text, _) in enumerate(code):
        if not text.startswith("v_mfma"):
            continue
        count += 1
        op, args = text.split(None, 1)
        result, need = registers(args.split(",")[0]), WAITS.get(op, 19)
        paths, seen = [(first + 1, 0)], {}
        while paths:
            i, waits = paths.pop()
            while i < len(code) and waits < need and seen.get(i, need) > waits:
                seen[i] = waits
                text, target = code[i]
                op, _, args = text.partition(" ")
                if op == "s_endpgm":
                    break
                if op.startswith("v_mfma"):
                    parts = args.split(",")
                    if registers(",".join(parts[1:3])) & result:
                        found.append((code[first][0], text, waits))
                    if registers(parts[0]) & result:
                        break  # adds to it or replaces it, in the matrix cores' own order
                elif not op.startswith("s_"):
                    if registers(args) & result:
                        found.append((code[first][0], text, waits))
                        break
                if op == "s_branch":
                    i, waits = target, waits + 1
                    continue
                if op.startswith("s_cbranch"):
                    paths.append((target, waits + 1))
                waits += int(args, 0) + 1 if op == "s_nop" else 1
                i += 1
    return count, found


def listing(*lines):
    """Instructions of 4 bytes, as they are printed; (text, target)."""
    out = "0000000000001000 <f>:\n"
    for i, line in enumerate(lines):
        text, target = line if isinstance(line, tuple) else (line, None)
        out += f"\t{text}   // {0x1000 + 4 * i:012X}: 00000000" + ("" if target is None else f" <f+0x{4 * target:x}>") + "\n"
    return out


@pytest.mark.parametrize("lines,wrong", [
    (["s_nop 7", "v_add_f32_e32 v9, v1, v9", "s_endpgm"], 0),
    (["s_nop 6", "v_add_f32_e32 v9, v1, v9", "s_endpgm"], 1),
    (["s_nop 6", "v_add_f32_e32 v9, v8, v9", "s_endpgm"], 0),
    (["s_nop 6", "v_mov_b32_e32 v0, v9", "s_endpgm"], 1),  # overwrites it
    (["ds_write_b128 v20, v[0:3]", "s_endpgm"], 1),
    ([("s_cbranch_scc1", 4), "s_nop 9", "s_endpgm", "v_add_f32_e32 v9, v1, v9", "s_endpgm"], 1),  # the branch alone
    ([("s_cbranch_scc1", 4), "s_nop 9", "s_endpgm", "s_nop 6", "v_add_f32_e32 v9, v1, v9", "s_endpgm"], 0),
    (["v_mfma_f32_16x16x32_bf16 v[0:3], v[30:33], v[34:37], v[0:3]", "s_nop 7", "v_add_f32_e32 v9, v1, v9", "s_endpgm"], 0),
    (["v_mfma_f32_16x16x32_bf16 v[40:43], v[0:3], v[34:37], v[40:43]", "s_nop 7", "s_endpgm"], 1),  # as a factor
    ([("s_branch", 0), "s_endpgm"], 0),
])
def test_the_search_itself(lines, wrong):
    code = list(functions(listing("v_mfma_f32_16x16x32_bf16 v[0:3], v[10:13], v[14:17], v[0:3]", *lines)))[0][1]
    assert len(early_uses(code)[1]) == wrong


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no disassembler")
def test_no_result_is_used_early(tmp_path):
    count = 0
    for n, code in enumerate(device_code(pr.LIB_PATH)):
        path = tmp_path / f"{n}.elf"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", str(path)], stdout=subprocess.PIPE, check=True, text=True).stdout
        for name, instructions in functions(text):
            matrix, wrong = early_uses(instructions)
            count += matrix
            assert not wrong, (name, wrong[:3])
    assert count > 1000
