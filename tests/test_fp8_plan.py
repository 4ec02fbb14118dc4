"""Which kernel a call of rq_gemm_fp8 runs, on the CPU: ``tests/fp8_plan_check.hip``
is the library's own choice, compiled for the host.  What include/rq.h says about
the FP8 matrix instructions is held to it."""
import os
import re
import shutil
import subprocess

import pytest

import gemm_rwkv_decode_amd as rq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
OUT = {"f32": rq.RQ_TYPE_F32, "f16": rq.RQ_TYPE_F16, "e4m3": rq.RQ_TYPE_E4M3}


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    """(kernel, ranges of K) of calls (M, out, workspace, [(N, K), ...])."""
    if not (os.path.exists(HIPCC) or shutil.which("hipcc")):
        pytest.skip("hipcc not available")
    exe = str(tmp_path_factory.mktemp("plan") / "fp8_plan_check")
    r = subprocess.run([HIPCC, "--offload-host-only", "-std=c++17", "-O1", "-Wno-unused-function",
                        "-Wl,--unresolved-symbols=ignore-all", "-I" + os.path.join(ROOT, "include"),
                        "-I" + os.path.join(ROOT, "gemm_rwkv_decode_amd", "csrc"),
                        os.path.join(ROOT, "tests", "fp8_plan_check.hip"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]

    def ask(calls):
        text = "\n".join(f"{M} {OUT[out]} {int(ws)} {len(shapes)} " +
                         " ".join(f"{n} {k}" for n, k in shapes) for M, out, ws, shapes in calls)
        r = subprocess.run([exe], input=text, capture_output=True, text=True)
        assert r.returncode == 0
        got = [(line.split()[0], int(line.split()[1])) for line in r.stdout.splitlines()]
        assert len(got) == len(calls)
        return got
    return ask


def tiles(M, shapes):
    return sum(-(-M // 128) * -(-n // 128) for n, _ in shapes)


def test_when_the_fp8_instructions_are_taken(plans):
    """More than 16 rows and more than 64 tiles of 128 x 128 over the call, more than
    128 of up to 64 rows: as the header says."""
    calls = []
    for M in (1, 4, 16, 17, 40, 64, 65, 128, 129, 203, 300, 513, 1000, 2047, 4001):
        for N in (1, 128, 768, 1000, 2560, 4096, 8192, 8320, 16384, 16512, 65529):
            for K in (128, 2048, 4096, 16384):
                for count in (1, 3, 8):
                    for out in OUT:
                        if out != "e4m3" or N % 128 == 0:
                            calls += [(M, out, ws, [(N, K)] * count) for ws in (0, 1)]
    # the borders themselves
    for M, border in ((64, 128), (65, 64), (128, 64), (17, 128)):
        rows = -(-M // 128)
        for t in (border, border + 1):
            calls += [(M, out, ws, [(128 * t // rows, 256)]) for out in OUT for ws in (0, 1)]
    for (M, out, ws, shapes), (kind, _) in zip(calls, plans(calls)):
        fp8 = out != "f32" and M > 16 and tiles(M, shapes) > (128 if M <= 64 else 64)
        assert kind.startswith("FP") == fp8, (M, out, ws, shapes, kind)
    text = " ".join(re.sub(r"\n \*", " ", open(os.path.join(ROOT, "include", "rq.h")).read()).split())
    assert "more than 16 rows whose outputs make more than 64 tiles of 128 x 128 over all products " \
           "(more than 128 with up to 64 rows) take the FP8 matrix instructions" in text
