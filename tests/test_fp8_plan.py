"""Which kernel a call of rq_gemm_fp8 runs, on the CPU: ``tests/fp8_plan_check.hip``
is the library's own choice, compiled for the host.  What include/rq.h says about
the FP8 matrix instructions is held to it, and the sizes of test_gpu_fp8_sums.py are
those of the kernels that they are there for."""
import os
import re
import shutil
import subprocess

import numpy as np
import pytest

import gemm_rwkv_decode_amd as rq
from tests import test_gpu_fp8_sums as G

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


def test_sizes_of_the_gpu_tests(plans):
    calls = [(c.M, c.out, c.ws, c.shapes) for c in G.CASES]
    for c, got in zip(G.CASES, plans(calls)):
        assert got == (c.kind, c.ranges), (c, got)
    assert {c.kind for c in G.CASES} >= {"ROWS16", "ROWS64", "RING1X2", "RING2X2", "RING4X2", "RING4X3",
                                         "RING4X4", "RING8X1", "RING8X2", "WIDE64", "WIDE128", "FP64",
                                         "FP128", "FP256"}
    # products that test_gpu_fp8_sums.py expects by themselves to the bit: kernels that
    # add a block after the other too
    one = [(c.M, c.out, False, [s]) for c in G.CASES if c.alone for s in c.shapes]
    assert one and all(k.startswith(("FP", "WIDE")) and r == 1 for k, r in plans(one))


def test_the_measure_of_sums_shows_a_scale_that_is_off():
    """The oracle with one block's scale 5% off at K = 4096: far past the limit."""
    g = np.random.default_rng(1)
    x, w = g.standard_normal((200, 32, 128)), g.standard_normal((300, 32, 128))
    y = np.einsum("mbk,nbk->mn", x, w)
    off = y + 0.05 * x[:, 3] @ w[:, 3].T
    assert G.difference(y.astype(np.float16), y) == 0
    assert G.difference(off.astype(np.float16), y) > 20 * G.FP8_LIMIT
