"""What the host code of the block-scaled FP8 calls and the group norm hands to its
kernels, checked on the CPU: ``tests/fp8_host_check.hip`` is the library's host code
compiled with the HIP runtime's queries and launches replaced by recorders."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_launches_and_arguments(tmp_path):
    if not (os.path.exists(HIPCC) or shutil.which("hipcc")):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "fp8_host_check")
    cmd = [HIPCC, "--offload-host-only", "-std=c++17", "-O1", "-Wno-unused-function",
           # the other calls' launches and the device code are not linked
           "-Wl,--unresolved-symbols=ignore-all",
           "-I" + os.path.join(ROOT, "include"),
           "-I" + os.path.join(ROOT, "gemm_rwkv_decode_amd", "csrc"),
           os.path.join(ROOT, "tests", "fp8_host_check.hip"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and "wrong=0" in r.stdout, r.stdout[-3000:]
