"""Every reader of a matrix instruction's result stands far enough behind it in
the 4-bit and expert kernels of the built library (no GPU).

The compiler counts the distance along the straight path only: where a branch
skips the next matrix instructions, the reader behind the branch's target came
1 instruction after the result's own, on the other side, and the GPU gave wrong
sums.  The sources keep such branches out; this looks at what was built.  A
16x16x32 product of 16-bit numbers takes 4 passes, its result may be read by
anything but a matrix instruction that adds to it 8 wait states later."""
import os
import re
import struct
import subprocess

import pytest

import dense_gemm_tiled_amd as tg

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
WAIT = 8


def registers(operand):
    m = re.match(r"^([va])\[(\d+):(\d+)\]$", operand)
    if m:
        return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)}
    m = re.match(r"^([va])(\d+)$", operand)
    return {(m.group(1), int(m.group(2)))} if m else set()


def parse(text):
    """[(name, [(op, operands, target index or None)])] of objdump's listing."""
    out = []
    for m in re.finditer(r"^([0-9a-f]+) <(\S+)>:\n(.*?)(?=\n\n|\Z)", text, re.S | re.M):
        base, lines, at = int(m.group(1), 16), [], {}
        for line in m.group(3).split("\n"):
            p = line.split("//")
            code = p[0].strip()
            a = re.match(r"\s*([0-9A-F]+):", p[1]) if len(p) > 1 else None
            if not code or not a:
                continue
            at[int(a.group(1), 16)] = len(lines)
            op, _, rest = code.partition(" ")
            t = re.search(r"<\S+\+0x([0-9a-f]+)>\s*$", line) if op.startswith(("s_branch", "s_cbranch")) else None
            lines.append((op, [o.strip().split()[0] for o in rest.split(",") if o.strip()],
                          base + int(t.group(1), 16) if t else None))
        out.append((m.group(2), [(op, o, at.get(t)) for op, o, t in lines]))
    return out


def early_readers(code, need=WAIT):
    """(matrix instruction, reader, wait states between them) of every pair
    that is too close on some path."""
    found = []
    for i, (op, operands, _) in enumerate(code):
        if not op.startswith("v_mfma"):
            continue
        result, todo, seen = registers(operands[0]), [(i + 1, 0)], {}
        while todo:
            j, states = todo.pop()
            while j < len(code) and states < need:
                if seen.get(j, need) <= states:
                    break
                seen[j] = states
                o, args, target = code[j]
                if o == "s_endpgm":
                    break
                if o.startswith("v_mfma"):
                    if any(registers(a) & result for a in args[1:3]):
                        found.append((i, j, states))
                    if registers(args[0]) & result or registers(args[3]) & result:
                        break          # (adds to it, in the matrix units' own order)
                elif o.startswith(("v_", "ds_", "buffer_", "global_", "flat_", "scratch_")):
                    if any(registers(a) & result for a in args):
                        found.append((i, j, states))
                        break
                if o.startswith("s_branch"):
                    j = target if target is not None else len(code)
                    states += 1
                    continue
                if o.startswith("s_cbranch") and target is not None:
                    todo.append((target, states + 1))
                states += int(args[0], 0) + 1 if o == "s_nop" else 1
                j += 1
    return found


def device_code(library):
    """The gfx950 code objects of a shared library."""
    data = open(library, "rb").read()
    for m in re.finditer(b"__CLANG_OFFLOAD_BUNDLE__", data):
        n, = struct.unpack_from("<Q", data, m.start() + 24)
        p = m.start() + 32
        for _ in range(n):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + length]:
                yield data[m.start() + offset:m.start() + offset + size]
            p += 24 + length


LISTING = """
0000000000001900 <kernel>:
	v_mfma_f32_16x16x32_f16 v[88:91], v[92:95], v[96:99], v[88:91] // 000000001900: 00000000 00000000
	s_cbranch_vccnz 4                                          // 000000001908: BF870004 <kernel+0x1c>
	v_mfma_f32_16x16x32_f16 v[92:95], v[120:123], v[132:135], v[124:127] // 00000000190C: 00000000 00000000
	s_nop 7                                                    // 000000001914: BF800007
	v_fmac_f32_e32 v87, v2, v95                                // 000000001918: 00000000
	v_fmac_f32_e32 v209, v2, v88                               // 00000000191C: 00000000
	s_endpgm                                                   // 000000001920: BF810000
"""


def test_the_branch_that_was_wrong_is_seen():
    (name, code), = parse(LISTING)
    assert name == "kernel" and len(code) == 7 and code[1][2] == 5
    assert early_readers(code) == [(0, 5, 1)]
    assert early_readers(code[:1] + [("s_nop", ["7"], None)] + code[5:]) == []
    assert early_readers(code[:1] + [("s_nop", ["6"], None)] + code[5:]) == [(0, 2, 7)]


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
@pytest.mark.parametrize("kernel", ["w4_rows_kernel", "moe_down_kernel"])
def test_readers_wait_in_the_built_library(kernel, tmp_path):
    objects = [c for c in device_code(tg.library_path()) if kernel.encode() in c]
    assert len(objects) == 2                                   # f16 and bf16
    for i, c in enumerate(objects):
        path = tmp_path / ("code%d.o" % i)
        path.write_bytes(c)
        text = subprocess.run([OBJDUMP, "-d", str(path)], capture_output=True, text=True, check=True).stdout
        kernels = parse(text)
        products = 0
        for name, code in kernels:
            products += sum(op.startswith("v_mfma_f32_16x16x32") for op, _, _ in code)
            assert all("16x16x32" in op for op, _, _ in code if op.startswith("v_mfma"))
            for a, b, states in early_readers(code):
                raise AssertionError("%s: %s %s is read %d wait states later by %s %s" % (
                    name, code[a][0], code[a][1], states, code[b][0], code[b][1]))
        assert any(kernel in name for name, _ in kernels) and products > 1000
