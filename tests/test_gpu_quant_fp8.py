"""rq_quant_fp8 against the definition in 64 bits: there is one right answer, so
values and scales are equal to it."""
import numpy as np
import pytest
import torch

import gemm_rwkv_decode_amd as rq
from tests import aroundtest as R
from tests import fp8test as F

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def run(x, act=rq.RQ_ACT_NONE, e8m0=True):
    """Values and scales of float16 or float32 numpy rows."""
    M, K = x.shape
    q, whole = R.guarded((M, K), torch.uint8, 0x55)
    if e8m0:
        s, swhole = R.guarded((M, K // 128), torch.uint8, 0x55)
    else:
        s, swhole = R.guarded((M, K // 128), torch.float32, -7.0)
    rq.rq_quant_fp8(torch.from_numpy(x).cuda(), q, s, act=act)
    assert whole() and swhole()
    return F.values(q.view(F.E4M3)), F.values(s.view(F.E8M0) if e8m0 else s)


def check(x, act=rq.RQ_ACT_NONE, e8m0=True):
    q, s = run(x, act, e8m0)
    want, scales = F.quant_ref(F.act(x, act))
    assert F.same(s, scales)
    assert F.same(q, want)


@pytest.mark.parametrize("act", [rq.RQ_ACT_NONE, rq.RQ_ACT_RELU2])
@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("M,K", [(1, 128), (1, 768), (3, 256), (5, 1152), (17, 640), (64, 2048),
                                 (129, 384), (1, 16384), (257, 128)])
def test_rows(M, K, dtype, act):
    g = np.random.default_rng(M * 7919 + K)
    x = g.standard_normal((M, K)) * np.exp(2 * g.standard_normal((M, K // 128, 1))).repeat(
        128, 2).reshape(M, K)
    check(x.astype(dtype), act, e8m0=(M + K // 128) % 2 == 0)


@pytest.mark.parametrize("e8m0", [True, False])
def test_ties_and_borders_of_scales(e8m0):
    """Every E4M3 value and every middle of two, at every place of a scale's border."""
    up, down = np.float32(np.inf), np.float32(0)
    rows = []
    for top in (448.0, np.nextafter(np.float32(448), up), np.nextafter(np.float32(448), down),
                256.0, 300.0, 224.0, 449.0, 512.0):
        for scale in (1.0, 2.0 ** -30, 2.0 ** 40):
            grid = np.concatenate([F.POSITIVE, F.MIDDLE])
            near = np.concatenate([grid, np.nextafter(grid.astype(np.float32), up),
                                   np.nextafter(grid.astype(np.float32), down)])
            near = near[np.abs(near) <= top].astype(np.float32)
            near = np.concatenate([near, -near])
            near = np.concatenate([near, np.zeros(-len(near) % 127, np.float32)])
            blocks = near.reshape(-1, 127)
            rows.append(np.concatenate([blocks, np.full((len(blocks), 1), top, np.float32)], 1)
                        * np.float32(scale))
    check(np.concatenate(rows), e8m0=e8m0)


def test_zeros_and_the_smallest_values():
    x = np.zeros((6, 256), np.float32)
    x[1, 5] = 2.0 ** -149
    x[2, :128] = 2.0 ** -126
    x[2, 128:] = 448 * 2.0 ** -126
    x[3, 0] = np.nextafter(np.float32(448 * 2.0 ** -126), np.float32(1))
    x[4] = -0.0
    x[5, ::3] = 1e-38
    for e8m0 in (True, False):
        check(x, e8m0=e8m0)
        check(x, rq.RQ_ACT_RELU2, e8m0)
    q, s = run(x)
    assert np.all(s[0] == 2.0 ** -126) and not q[0].any()
    h = np.zeros((2, 128), np.float16)
    h[1, ::2] = np.float16(6e-8)
    check(h)


def test_the_largest_values():
    x = np.random.default_rng(1).standard_normal((3, 384)).astype(np.float32)
    x[0, 7] = np.finfo(np.float32).max
    x[1, 300] = -np.finfo(np.float32).max
    x[2] *= np.float32(1e19)          # squares past binary32
    check(x, e8m0=False)
    check(x, rq.RQ_ACT_RELU2)
    h = np.full((1, 128), 65504, np.float16)
    check(h)
    check(h, rq.RQ_ACT_RELU2)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("act", [rq.RQ_ACT_NONE, rq.RQ_ACT_RELU2])
def test_what_is_not_finite_becomes_nan_and_moves_no_scale(dtype, act):
    x = np.random.default_rng(2).standard_normal((8, 512)).astype(dtype)
    x[0, 3], x[1, 130], x[2, 511], x[3, 256:384] = np.inf, -np.inf, np.nan, np.nan
    x[4, ::2] = np.inf
    check(x, act)
    q, _ = run(x, act)
    # minus infinity is below zero
    assert np.isnan(q[1, 130]) == (act == rq.RQ_ACT_NONE)
    assert not np.isnan(q[5:]).any()


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_a_long_list_of_blocks(dtype):
    """More blocks than workgroups are resident, against the same rows one by one."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((20011, 1408), generator=g, device="cuda").to(dtype)
    q = torch.empty(x.shape, dtype=F.E4M3, device="cuda")
    s = torch.empty((20011, 11), device="cuda")
    rq.rq_quant_fp8(x, q, s)
    for rows in (slice(0, 3), slice(9990, 10001), slice(20008, 20011)):
        want, scales = F.quant_ref(x[rows].cpu().numpy())
        assert F.same(F.values(q[rows]), want) and F.same(F.values(s[rows]), scales)
    back = q.float().view(20011, 11, 128) * s[..., None]
    worst = ((back - x.float().view(20011, 11, 128)).abs() - s[..., None] * 2.0 ** -10) \
        / x.float().view(20011, 11, 128).abs().clamp(min=1e-30)
    assert float(worst.max()) <= 2.0 ** -4


def test_graph_replays():
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((33, 640), generator=g, device="cuda").half()
    q = torch.empty(x.shape, dtype=F.E4M3, device="cuda")
    s = torch.empty((33, 5), dtype=F.E8M0, device="cuda")
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = rq.prepare("rq_quant_fp8", x, q, s, stream=st)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for k in range(3):
        x.mul_(-3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, scales = F.quant_ref(x.cpu().numpy())
        assert F.same(F.values(q), want) and F.same(F.values(s), scales)
