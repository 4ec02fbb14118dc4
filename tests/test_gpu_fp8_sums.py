"""Sums of rq_gemm_fp8 in every kernel that it has, of one product and of several in
a call.  (test_fp8_plan.py checks on the CPU that a case takes the kernel named.)

How far sums are off shows in the binary16 outputs that are not the number nearest
the sum in 64 bits.  An error e moves a sum over a border between two numbers, u
apart, with probability |e| / u, and the output then differs by u: on average a square
of u |e|, with u <= 2^-10 |y|.  For errors of a 2-norm of d times that of y,
independent of y, and normal y, whose mean |y| is 0.8 of its root mean square, the
outputs' difference is at most sqrt(2^-10 * 0.8 * d) of the 2-norm of y:
  FP8 instructions, d = 4e-5:      1.8e-4
  binary16 instructions, 16 units: 2.8e-5   (as test_gpu_gemm_fp8.py has binary32 outputs)
"""
import dataclasses

import numpy as np
import pytest
import torch

import gemm_rwkv_decode_amd as rq
from tests import aroundtest as R
from tests import fp8test as F

WIDE_SUMS, FP8_SUMS = 16 * F.U, 4e-5
FP8_LIMIT = (2.0 ** -10 * 0.8 * FP8_SUMS) ** 0.5
WIDE_LIMIT = (2.0 ** -10 * 0.8 * WIDE_SUMS) ** 0.5


@dataclasses.dataclass(frozen=True)
class Case:
    kind: str
    M: int
    shapes: tuple
    out: str = "f16"
    ranges: int = 1
    ws: bool = True
    alone: bool = False  # each product as by itself, to the bit

    def __str__(self):
        return f"{self.kind} {self.out} {self.M}x" + "+".join(f"{n}x{k}" for n, k in self.shapes)


CASES = [
    Case("ROWS16", 3, ((4096, 4096),)),
    Case("ROWS16", 16, ((2050, 768), (129, 1152))),
    Case("ROWS64", 4, ((16640, 640),)),
    Case("ROWS64", 13, ((9000, 384), (7000, 2560), (517, 128))),
    Case("RING1X2", 32, ((2048, 4096),)),
    Case("RING2X2", 100, ((2500, 1024), (1030, 384))),
    Case("RING4X2", 20, ((12000, 2048),)),
    Case("RING4X3", 203, ((2560, 2560),)),
    Case("RING4X4", 250, ((4095, 1280),)),
    Case("RING8X1", 33, ((1024, 1024), (256, 4096)), "e4m3"),
    Case("RING8X2", 96, ((7936, 640), (256, 256)), "e4m3"),
    Case("WIDE64", 61, ((32765, 640),), "f32"),
    Case("WIDE64", 1500, ((1025, 640), (2050, 1152)), "f32", alone=True),
    Case("WIDE128", 2047, ((4096, 640),), "f32"),
    Case("WIDE128", 2047, ((2049, 1152), (3157, 1152), (1024, 640)), "f32"),
    Case("FP64", 1100, ((1152, 1024),)),
    Case("FP64", 50, ((9000, 640), (8001, 384))),
    Case("FP64", 300, ((130, 640), (257, 128), (384, 2560), (1, 256), (500, 384), (640, 1152), (77, 512),
                       (768, 896))),
    Case("FP128", 1300, ((3500, 640),)),
    Case("FP128", 1300, ((1030, 384), (2049, 640), (777, 1152)), alone=True),
    Case("FP128", 1300, ((1024, 384), (2048, 640), (768, 1152)), "e4m3", alone=True),
    Case("FP256", 2561, ((3900, 640),)),
    Case("FP256", 2561, ((1500, 384), (2049, 640), (1000, 1152)), alone=True),
    Case("FP256", 2561, ((1536, 384), (2048, 640), (1024, 1152)), "e4m3", alone=True),
    Case("FP128", 1100, ((1152, 4224),), ranges=2),
    Case("FP128", 1025, ((1024, 6272),), ranges=3),
    Case("FP128", 700, ((640, 4224), (1025, 6400)), ranges=2),
    Case("FP128", 1100, ((300, 6272), (385, 6400), (129, 12800)), ranges=3),
    Case("FP128", 300, ((130, 4096), (257, 4224), (384, 6400), (1, 4480), (500, 5120), (640, 4352),
                        (77, 8192), (768, 10240)), ranges=2),
    Case("FP128", 700, ((640, 4224), (1024, 6400)), "e4m3", ranges=2),
    Case("FP128", 1100, ((256, 6272), (384, 6400), (384, 12800)), "e4m3", ranges=3),
]


def difference(y, exact):
    """2-norm of what binary16 outputs differ by from the nearest of the exact ones,
    beside the exact ones'."""
    near = np.asarray(exact).astype(np.float16).astype(np.float64)
    return float(np.linalg.norm(np.asarray(y).astype(np.float64) - near) / np.linalg.norm(exact))


def operands(M, N, K, e8m0, seed):
    g = torch.Generator().manual_seed(seed)
    w, x = F.random_codes(g, N, K), F.random_codes(g, M, K)
    return (w, F.random_scales(g, (N + 127) // 128, K // 128, e8m0), x,
            F.random_scales(g, M, K // 128, e8m0))


def call(ops, out, shapes, e8m0, workspace):
    """Outputs of a call (pairs for E4M3), checked for writes around them."""
    ys, whole = [], []
    for o, (n, _) in zip(ops, shapes):
        M = o[2].shape[0]
        if out == "e4m3":
            q, c1 = R.guarded((M, n), torch.uint8, 0x55)
            s, c2 = R.guarded((M, n // 128), torch.uint8 if e8m0 else torch.float32, 0x55)
            ys.append((q, s))
            whole += [c1, c2]
        else:
            y, c = R.guarded((M, n), torch.float16 if out == "f16" else torch.float32, -3.0)
            ys.append(y)
            whole.append(c)
    rq.rq_gemm_fp8([(*o, None, y, n, k) for o, y, (n, k) in zip(ops, ys, shapes)],
                   act=rq.RQ_ACT_RELU2 if out == "e4m3" else rq.RQ_ACT_NONE, workspace=workspace)
    assert all(c() for c in whole)
    return ys


def same(a, b):
    if isinstance(a, tuple):
        return all(torch.equal(x, y) for x, y in zip(a, b))
    return torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("e8m0", [True, False])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_sums(case, e8m0):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    print(f"[fp8 sums] {case} e8m0 {e8m0}", flush=True)
    ops = [operands(case.M, n, k, e8m0, 1000 * i + n + k) for i, (n, k) in enumerate(case.shapes)]
    ws = rq.AUTO if case.ws else None
    size = rq.rq_gemm_fp8_workspace_size(case.shapes, case.M, int(e8m0),
                                         {"f32": 0, "f16": 1, "e4m3": 2}[case.out])
    tiles = sum(-(-case.M // 128) * -(-n // 128) for n, _ in case.shapes)
    assert size == (65536 + tiles * case.ranges * 65536 if case.ranges > 1 else 0)
    ys = call(ops, case.out, case.shapes, e8m0, ws)
    for _ in range(3 if case.ranges > 1 else 1):  # ranges are joined in one order
        assert all(same(a, b) for a, b in zip(ys, call(ops, case.out, case.shapes, e8m0, ws)))
    if case.alone:
        for o, y, s in zip(ops, ys, case.shapes):
            assert same(y, call([o], case.out, [s], e8m0, None)[0]), s
    halves = ys if case.out != "e4m3" else call(ops, "f16", case.shapes, e8m0, ws)
    fp8 = case.kind.startswith("FP")
    err = norm = 0.0
    for o, y, h, (n, k) in zip(ops, ys, halves, case.shapes):
        if case.out == "e4m3":
            q, s = torch.empty_like(y[0]), torch.empty_like(y[1])
            rq.rq_quant_fp8(h, q, s, act=rq.RQ_ACT_RELU2)
            assert same(y, (q, s))
        want, mag = F.gemm_ref(*o)
        bound = F.gemm_bound(want, mag, k, "f32")
        if case.out != "f32":
            if fp8:
                bound = F.gemm_bound(want, mag, k, "f16")
            else:  # binary32 sums, rounded once
                bound = bound + F.HALF * (want.abs() + bound) + 2.0 ** -25
        assert bool(((h.double() - want).abs() <= bound).all()), (n, k)
        near = want.half().double() if case.out != "f32" else want
        err += float((h.double() - near).square().sum())
        norm += float(want.square().sum())
    limit = FP8_LIMIT if fp8 else (WIDE_LIMIT if case.out != "f32" else WIDE_SUMS)
    print(f"[fp8 sums] {(err / norm) ** 0.5:.3g} of {limit:.3g}", flush=True)
    assert (err / norm) ** 0.5 <= limit
