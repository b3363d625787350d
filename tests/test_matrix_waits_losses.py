"""Every reader of a matrix instruction's result stands far enough behind it in
the cross entropy's own kernels of the built library, on every path (no GPU)."""
import os
import subprocess

import pytest

import dense_gemm_tiled_amd as tg
import test_matrix_waits as waits


@pytest.mark.skipif(not os.path.exists(waits.OBJDUMP), reason="no llvm-objdump")
def test_readers_wait_in_the_built_library(tmp_path):
    objects = [c for c in waits.device_code(tg.library_path()) if b"ce_outer_kernel" in c]
    assert len(objects) == 1
    path = tmp_path / "code.o"
    path.write_bytes(objects[0])
    text = subprocess.run([waits.OBJDUMP, "-d", str(path)], capture_output=True, text=True, check=True).stdout
    products = {"ce_rows_kernel": 0, "ce_outer_kernel": 0}
    for name, code in waits.parse(text):
        assert all("16x16x32" in op for op, _, _ in code if op.startswith("v_mfma")), name
        for kernel in products:
            if kernel in name:
                products[kernel] += sum(op.startswith("v_mfma_f32_16x16x32") for op, _, _ in code)
        for a, b, states in waits.early_readers(code):
            raise AssertionError("%s: %s %s is read %d wait states later by %s %s" % (
                name, code[a][0], code[a][1], states, code[b][0], code[b][1]))
    assert all(n > 64 for n in products.values()), products


@pytest.mark.skipif(not os.path.exists(waits.OBJDUMP), reason="no llvm-objdump")
@pytest.mark.parametrize("dtype", [1, 2])
def test_readers_wait_in_the_tiles_epilogues(dtype, tmp_path):
    """The tiles of x W^T whose epilogues take the softmax (6) or write the
    gradient (7): 3 tile classes, with and without a masked end of K."""
    marks = ["gemm_dma_kernelILi%dELb0ELb1ELi%dE" % (dtype, out) for out in (6, 7)]
    objects = [c for c in waits.device_code(tg.library_path()) if marks[0].encode() in c]
    assert len(objects) == 1
    path = tmp_path / "code.o"
    path.write_bytes(objects[0])
    text = subprocess.run([waits.OBJDUMP, "-d", str(path)], capture_output=True, text=True, check=True).stdout
    kernels = [(name, code) for name, code in waits.parse(text) if any(m in name for m in marks)]
    assert len(kernels) == 12
    for name, code in kernels:
        assert sum(op.startswith("v_mfma_f32_16x16x32") for op, _, _ in code) >= 32, name
        assert waits.early_readers(code) == [], name
