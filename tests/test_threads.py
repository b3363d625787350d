"""Threads that share a context (no GPU): the host code of the 4-bit and
expert entry points under a thread sanitizer, kernels and HIP calls stood in
for (threads_main.cpp), and the dense entry points' refusals."""
import ctypes
import os
import shutil
import subprocess
import threading

import pytest

import dense_gemm_tiled_amd as tg

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "dense_gemm_tiled_amd", "csrc")


def build_and_run(tmp_path, source, flags):
    exe = str(tmp_path / "main")
    cmd = ["g++", "-std=c++17", "-O1", "-g", *flags, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, source, os.path.join(CSRC, "qweight.cpp"),
           os.path.join(CSRC, "moe.cpp"), "-o", exe, "-pthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        return None, r.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=100), ""


@pytest.mark.skipif(not shutil.which("g++") or not os.path.exists("/opt/rocm/include/hip"), reason="no g++ or HIP headers")
def test_threads_share_a_context(tmp_path):
    (tmp_path / "one.cpp").write_text("int main() { return 0; }\n")
    flag = ["-fsanitize=thread"]
    probe = subprocess.run(["g++", *flag, str(tmp_path / "one.cpp"), "-o", str(tmp_path / "one"), "-pthread"],
                           capture_output=True)
    if probe.returncode or subprocess.run([str(tmp_path / "one")], capture_output=True).returncode:
        flag = []          # no sanitizer for this compiler or kernel: the counts alone
    run, err = build_and_run(tmp_path, os.path.join(HERE, "threads_main.cpp"), flag)
    assert run is not None, err
    assert run.returncode == 0 and "data race" not in run.stderr, run.stderr[:3000] + run.stdout


def test_refused_calls_on_one_context():
    """Every thread's calls return their own status, and what is read after
    them is a whole text."""
    lib, out = tg.load_library(), ctypes.c_void_p()
    assert lib.tc_context_create(ctypes.byref(out)) == 0
    texts, failed = {b"M must be >= 1 (got 0)", b"descriptor is NULL", b"A, B and C must be non-NULL"}, []
    P = [0x10000000000 * (i + 1) for i in range(5)]

    def run(kind):
        d, w = tg.QWeightDescT(1, 64, 256, 128, tg.BF16, False), tg.QWeightT(P[0], P[1], None)
        g, b = tg.QGemmDescT(0, tg.BF16, tg.BF16, 1.0, 0.0, 0, 0), tg.BatchedDescT()
        for _ in range(3000):
            if kind == 0:
                st = lib.tc_qgemm_async(out, ctypes.byref(g), ctypes.byref(d), P[2], ctypes.byref(w), P[3], None, P[4])
            elif kind == 1:
                st = lib.tc_gemm_async(out, None, P[0], P[1], P[2], P[4])
            else:
                st = lib.tc_gemm_batched_async(out, ctypes.byref(b), None, P[1], P[2], P[4])
            if st != 1 or lib.tc_last_error(out) not in texts | {b""}:
                failed.append((kind, st, lib.tc_last_error(out)))

    threads = [threading.Thread(target=run, args=(k,)) for k in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed[:3]
    assert lib.tc_dispatch_count(out) == 0
    lib.tc_context_destroy(out)
