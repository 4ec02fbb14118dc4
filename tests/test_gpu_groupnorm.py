"""rq_groupnorm against its formula in 64 bits."""
import numpy as np
import pytest
import torch

import gemm_rwkv_decode_amd as rq
from tests import aroundtest as R
from tests import fp8test as F

pytestmark = pytest.mark.gpu
EPS = 64e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def make(T, C, seed, half=False, offset=0.0):
    g = np.random.default_rng(seed)
    dt = np.float16 if half else np.float32

    def n(*shape, scale=1.0):
        return (g.standard_normal(shape) * scale).astype(np.float32)
    y = n(T, C) * np.exp(n(T, 1)) + np.float32(offset)
    bonus = (n(T, C).astype(dt), n(T, C).astype(dt), n(C, scale=0.3), n(T, C).astype(dt))
    return dict(y=y, weight=1 + n(C, scale=0.1), bias=n(C, scale=0.1), bonus=bonus,
                gate=n(T, C, scale=2.0).astype(dt))


def cuda(t):
    if isinstance(t, tuple):
        return tuple(cuda(a) for a in t)
    return None if t is None else torch.from_numpy(np.ascontiguousarray(t)).cuda()


def run(a, groups, out="f32", act=rq.RQ_ACT_NONE, eps=EPS, e8m0=True):
    T, C = a["y"].shape
    d = {k: cuda(v) for k, v in a.items()}
    if out == "e4m3":
        q, c1 = R.guarded((T, C), torch.uint8, 0x55)
        s, c2 = R.guarded((T, C // 128), torch.uint8 if e8m0 else torch.float32, 0x55)
        o = (q, s)
    else:
        o, c1 = R.guarded((T, C), torch.float16 if out == "f16" else torch.float32, -3.0)
        c2 = c1
    rq.rq_groupnorm(d["y"], groups, d["weight"], d["bias"], eps, o, bonus=d["bonus"],
                    gate=d["gate"], act=act)
    assert c1() and c2()
    return o


def check(a, groups, act=rq.RQ_ACT_NONE, eps=EPS, out="f32"):
    got = run(a, groups, out, act, eps).cpu().double().numpy()
    want, bound = F.norm_ref(a["y"], groups, a["weight"], a["bias"], eps, a["bonus"], a["gate"],
                             act == rq.RQ_ACT_SILU)
    if out == "f16":
        bound = bound + F.HALF * (np.abs(want) + bound) + 2.0 ** -25
    worst = np.max(np.abs(got - want) / np.maximum(bound, 1e-300))
    assert worst <= 1, worst


@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("T,C,groups", [(1, 768, 12), (1, 64, 1), (2, 128, 2), (3, 64, 2),
                                        (5, 320, 5), (33, 4096, 64), (7, 2560, 40), (4, 1152, 18),
                                        (9, 1024, 8), (6, 768, 3), (130, 192, 6), (3, 96, 3),
                                        (1, 256, 1), (2, 5120, 40)])
def test_sizes(T, C, groups, half, out):
    check(make(T, C, T * 31 + C, half), groups, out=out)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("without", [("bonus",), ("gate",), ("weight", "bias"), ("bias", "gate"),
                                     ("bonus", "gate"), ("weight", "bias", "bonus", "gate")])
def test_parts_left_out(without, half):
    a = make(11, 640, 5, half)
    for k in without:
        a[k] = None
    check(a, 10)
    check(a, 10, rq.RQ_ACT_SILU)


@pytest.mark.parametrize("half", [False, True])
def test_silu_gates_of_every_size(half):
    a = make(8, 512, 6, half)
    a["gate"] = np.linspace(-200, 200, 8 * 512).reshape(8, 512).astype(a["gate"].dtype)
    check(a, 8, rq.RQ_ACT_SILU)
    check(a, 8, rq.RQ_ACT_SILU, out="f16")


def test_groups_far_from_zero_and_of_one_value():
    check(make(16, 512, 7, offset=1000.0), 8)
    a = make(4, 256, 8)
    a["y"][:] = 5.0
    a["y"][1] = 0.0
    a["y"][2] = 1e-20
    check(a, 4)
    check(a, 4, eps=1e-12)


@pytest.mark.parametrize("e8m0", [True, False])
@pytest.mark.parametrize("T,C,groups", [(1, 768, 12), (3, 128, 2), (21, 2560, 40), (5, 4096, 64),
                                        (6, 384, 12), (4, 1024, 4)])
def test_quantized_outputs_are_those_of_the_two_calls(T, C, groups, e8m0):
    a = make(T, C, 9 + T, half=T % 2 == 0)
    q, s = run(a, groups, "e4m3", e8m0=e8m0)
    h = run(a, groups, "f16")
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    rq.rq_quant_fp8(h, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_non_finite_inputs_stay_in_their_group():
    a = make(4, 512, 10)
    clean = run(a, 8).cpu().numpy()
    b = {k: v if v is None else (tuple(t.copy() for t in v) if isinstance(v, tuple) else v.copy())
         for k, v in a.items()}
    b["y"][0, 70] = np.inf
    b["y"][1, 130] = np.nan
    b["bonus"][0][2, 200] = np.nan
    b["bonus"][3][3, 300] = np.inf
    got = run(b, 8).cpu().numpy()
    hit = np.zeros((4, 512), bool)
    hit[0, 64:128] = hit[1, 128:192] = hit[2, 192:256] = hit[3, 300] = True
    assert np.array_equal(got[~hit], clean[~hit])
    assert not np.isfinite(got[hit]).any()
    q, s = run(b, 8, "e4m3")
    h = run(b, 8, "f16")
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    rq.rq_quant_fp8(h, q2, s2)
    assert F.same(F.values(q.view(F.E4M3)), F.values(q2.view(F.E4M3))) and torch.equal(s, s2)


def test_in_place_and_many_tokens():
    T, C = 5000, 448
    a = make(T, C, 11)
    want = run(a, 7)
    d = {k: cuda(v) for k, v in a.items()}
    rq.rq_groupnorm(d["y"], 7, d["weight"], d["bias"], EPS, d["y"], bonus=d["bonus"],
                    gate=d["gate"])
    assert torch.equal(d["y"], want)
    rows = slice(4990, 5000)
    b = {k: (v if k in ("weight", "bias") else
             (tuple(t[rows] if t.ndim == 2 else t for t in v) if isinstance(v, tuple) else v[rows]))
         for k, v in a.items()}
    check(b, 7)
    assert torch.equal(run(b, 7), want[rows])


@pytest.mark.parametrize("out", ["f32", "e4m3"])
def test_graph_replays_on_a_stream_of_its_own(out):
    T, C, H = 37, 768, 12
    a = make(T, C, 3)
    d = {k: cuda(v) for k, v in a.items()}
    o = torch.empty((T, C), device="cuda") if out == "f32" else \
        (torch.empty((T, C), dtype=torch.uint8, device="cuda"),
         torch.empty((T, C // 128), dtype=torch.uint8, device="cuda"))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = rq.prepare("rq_groupnorm", d["y"], H, d["weight"], d["bias"], EPS, o, stream=st,
                      bonus=d["bonus"], gate=d["gate"], act=rq.RQ_ACT_SILU)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for k in range(3):
        d["gate"].mul_(-1.5)
        d["y"].add_(0.25)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        b = dict(a, y=d["y"].cpu().numpy(), gate=d["gate"].cpu().numpy())
        want = run(b, H, out, rq.RQ_ACT_SILU)
        for x, y in zip((o,) if out == "f32" else o, (want,) if out == "f32" else want):
            assert torch.equal(x, y)
