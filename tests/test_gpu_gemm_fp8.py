"""rq_gemm_fp8 against its formula in 64 bits (bounds of every output, derived in
fp8test.gemm_bound)."""
import numpy as np
import pytest
import torch

import gemm_rwkv_decode_amd as rq
from tests import aroundtest as R
from tests import fp8test as F

pytestmark = pytest.mark.gpu
OUTS = ("f32", "f16", "e4m3")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def say(msg):
    print(msg, flush=True)


def operands(M, N, K, e8m0, seed, spread=False):
    g = torch.Generator().manual_seed(seed)
    w = F.random_codes(g, N, K, spread=spread)
    x = F.random_codes(g, M, K, spread=spread)
    return (w, F.random_scales(g, (N + 127) // 128, K // 128, e8m0), x,
            F.random_scales(g, M, K // 128, e8m0))


def output(M, N, out, e8m0):
    """(what the call takes as y, check that nothing around it was written)"""
    if out == "e4m3":
        q, c1 = R.guarded((M, N), torch.uint8, 0x55)
        s, c2 = R.guarded((M, N // 128), torch.uint8 if e8m0 else torch.float32, 0x55)
        return (q, s), lambda: c1() and c2()
    return R.guarded((M, N), torch.float16 if out == "f16" else torch.float32, -3.0)


def run(ops, out="f32", y_in=None, act=rq.RQ_ACT_NONE, workspace=rq.AUTO):
    w, ws, x, xs = ops
    M, N = x.shape[0], w.shape[0]
    y, whole = output(M, N, out, ws.dtype != torch.float32)
    rq.rq_gemm_fp8([(w, ws, x, xs, y_in, y, N, w.shape[1])], act=act, workspace=workspace)
    assert whole()
    return y


def check(ops, out="f32", y_in=None, workspace=rq.AUTO):
    y = run(ops, out, y_in, workspace=workspace)
    want, mag = F.gemm_ref(*ops, y_in)
    bound = F.gemm_bound(want, mag, ops[0].shape[1], out).clamp(min=1e-300)  # 0 / 0 is 0
    worst = float(((y.double() - want).abs() / bound).max())
    assert worst <= 1, worst
    return y


def two_calls(ops, act, workspace=rq.AUTO):
    """What the binary16 output quantized by itself gives."""
    h = run(ops, "f16", workspace=workspace)
    e8m0 = ops[1].dtype != torch.float32
    q = torch.empty(h.shape, dtype=torch.uint8, device="cuda")
    s = torch.empty((h.shape[0], h.shape[1] // 128), device="cuda",
                    dtype=torch.uint8 if e8m0 else torch.float32)
    rq.rq_quant_fp8(h, q, s, act=act)
    return q, s


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("M,N,K", [
    (1, 128, 128), (1, 768, 768), (2, 256, 384), (3, 1024, 640), (15, 128, 1152), (16, 384, 256),
    (17, 128, 2048), (31, 256, 128), (33, 640, 1024), (48, 128, 256), (63, 256, 896),
    (64, 512, 512), (65, 384, 384), (100, 256, 1280), (127, 128, 128), (128, 256, 256),
    (129, 512, 640), (200, 1024, 384), (255, 256, 1024), (257, 768, 512), (300, 2048, 256),
    (513, 640, 768), (700, 1280, 384), (1100, 768, 256), (1100, 1152, 384), (140, 8448, 640),
    (1281, 1408, 1152), (50, 16640, 256), (2400, 4352, 384), (650, 16384, 128), (4500, 3968, 256),
    (1, 16384, 256), (3, 16512, 1152), (9, 16640, 640), (16, 65536, 256), (7, 4096, 4096),
    (12, 4096, 4224), (61, 32768, 384), (800, 4096, 256)])
def test_sizes(M, N, K, out):
    e8m0 = (M + N // 128 + K // 128) % 2 == 0
    say(f"[gemm_fp8] M {M} N {N} K {K} {out} e8m0 {e8m0}")
    ops = operands(M, N, K, e8m0, M + N + K)
    if out == "e4m3":
        for act in (rq.RQ_ACT_NONE, rq.RQ_ACT_RELU2):
            got, want = run(ops, out, act=act), two_calls(ops, act)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    else:
        check(ops, out)


@pytest.mark.parametrize("e8m0", [True, False])
@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("N", [1, 2, 3, 5, 7, 9, 17, 65, 127, 129, 131, 255, 257, 321, 514])
@pytest.mark.parametrize("M", [1, 20, 70, 140, 300])
def test_odd_numbers_of_outputs(M, N, out, e8m0):
    say(f"[gemm_fp8] odd N {N} M {M} {out}")
    check(operands(M, N, 384, e8m0, M * 1000 + N), out)


@pytest.mark.parametrize("e8m0", [True, False])
@pytest.mark.parametrize("M,N", [(1300, 1025), (129, 8705), (2050, 1157), (2401, 4345), (2305, 4610)])
def test_many_odd_binary16_outputs(M, N, e8m0):
    say(f"[gemm_fp8] M {M} odd N {N}")
    check(operands(M, N, 384, e8m0, M + N), "f16")


@pytest.mark.parametrize("e8m0", [True, False])
@pytest.mark.parametrize("M,N,K,ranges", [
    (1100, 1152, 1024, 1), (130, 8320, 2176, 1), (130, 8192, 2176, 1), (1500, 1408, 4224, 1),
    (1500, 1280, 4224, 2), (257, 4096, 10240, 2), (1025, 1024, 1536, 1), (1100, 1152, 4096, 2),
    (130, 8192, 4224, 2), (1025, 1024, 6272, 3)])
def test_ranges_of_k_through_a_workspace(M, N, K, ranges, e8m0):
    """Sizes on both sides of splitting K, with the workspace and without; binary16
    and E4M3 alike."""
    tiles = -(-M // 128) * -(-N // 128)
    size = rq.rq_gemm_fp8_workspace_size([(N, K)], M, int(e8m0), rq.RQ_TYPE_F16)
    assert size == (65536 + tiles * ranges * 65536 if ranges > 1 else 0)
    ops = operands(M, N, K, e8m0, M + N + K)
    for ws in (rq.AUTO, None, rq.AUTO):
        check(ops, "f16", workspace=ws)
        got, want = run(ops, "e4m3", act=1, workspace=ws), two_calls(ops, 1, ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("M", [1, 5, 16, 40, 64, 90, 250, 520])
@pytest.mark.parametrize("K", [128, 768, 2560, 4224, 10240])
def test_long_rows_with_a_residual(M, K):
    """K kept whole and split; y_in apart, in place and absent."""
    N = 384
    say(f"[gemm_fp8] long K {K} M {M}")
    ops = operands(M, N, K, K % 256 == 0, M + K)
    y_in = torch.randn((M, N), generator=torch.Generator().manual_seed(1)).cuda() * 100
    for ws in (rq.AUTO, None):
        y = check(ops, "f32", y_in, ws)
        z = y_in.clone()
        rq.rq_gemm_fp8([(*ops, z, z, N, K)], workspace=ws)
        assert torch.equal(z, y)
        check(ops, "f32", None, ws)
        check(ops, "f16", None, ws)
        got, want = run(ops, "e4m3", act=1, workspace=ws), two_calls(ops, 1, ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("out", ["f32", "f16"])
@pytest.mark.parametrize("M", [1, 30, 130, 600])
def test_codes_of_every_size(M, out):
    """All finite codes alike: products from 2^-18 to 2^17 in one sum."""
    for e8m0 in (True, False):
        check(operands(M, 300, 640, e8m0, M, spread=True), out)


@pytest.mark.parametrize("M,N", [(1300, 1100), (4200, 3900)])
def test_codes_of_every_size_in_large_tiles(M, N):
    for e8m0 in (True, False):
        ops = operands(M, N, 640, e8m0, M, spread=True)
        # binary16 outputs stay finite: codes to 448 twice, 640 of them, scales to 2^-3
        check((ops[0], ops[1], ops[2], (ops[3].float() * 2.0 ** -11).to(ops[3].dtype)), "f16")


def test_binary32_outputs_keep_binary32_sums():
    """The 2-norm of the errors beside that of y, on normal values: 640 products
    and five block sums of independent errors of at most 2 U of a partial sum."""
    for M in (1, 40, 300, 1000):
        ops = operands(M, 512, 640, True, M)
        want, _ = F.gemm_ref(*ops)
        y = run(ops, "f32").double()
        assert float((y - want).norm() / want.norm()) <= 16 * F.U


@pytest.mark.parametrize("M", [1, 20, 100, 300])
def test_several_problems_in_a_call(M):
    """Different N and K side by side; each as by itself to the bit where the plan
    of the call is the same, within its bound always."""
    shapes = [(256, 384), (130, 128), (1, 1024), (512, 2560), (77, 256), (128, 128), (300, 640),
              (64, 768)]
    for count in (2, 3, 8):
        for out in ("f32", "f16"):
            for e8m0 in (True, False):
                ops = [operands(M, n, k, e8m0, 100 * M + i) for i, (n, k) in
                       enumerate(shapes[:count])]
                ys = [output(M, n, out, e8m0) for n, _ in shapes[:count]]
                rq.rq_gemm_fp8([(*o, None, y, n, k) for o, (y, _), (n, k) in
                                zip(ops, ys, shapes)])
                for o, (y, whole), (n, k) in zip(ops, ys, shapes):
                    assert whole()
                    want, mag = F.gemm_ref(*o)
                    b = F.gemm_bound(want, mag, k, out)
                    assert float(((y.double() - want).abs() / b).max()) <= 1


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("M", [4, 50, 150, 400])
def test_rows_are_independent_and_nan_reaches_its_outputs(M, out):
    N, K = 256, 640
    w, ws, x, xs = operands(M, N, K, True, M)
    clean = run((w, ws, x, xs), out)
    x2, xs2, w2 = x.clone(), xs.clone(), w.clone()
    x2.view(torch.uint8)[1, 200] = 0x7F       # NaN in a row of x
    xs2.view(torch.uint8)[2, 3] = 0xFF        # a NaN scale
    w2.view(torch.uint8)[130, 7] = 0xFF       # NaN in an output's weights
    got = run((w2, ws, x2, xs2), out)
    hit = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    hit[1:3] = True
    hit[:, 130] = True
    if out == "e4m3":
        want = two_calls((w2, ws, x2, xs2), 0)
        a, b = F.values(got[0].view(F.E4M3)), F.values(want[0].view(F.E4M3))
        assert F.same(a, b) and torch.equal(got[1], want[1])
        assert np.isnan(a[hit.cpu().numpy()]).all()
        far = (~hit).clone()
        far[:, 128:] = False                  # the second block's scale may move
        assert torch.equal(got[0][far], clean[0][far])
    else:
        assert torch.isnan(got[hit]).all() and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("e8m0", [True, False])
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("M,N", [(1300, 1024), (4200, 3840)])
def test_nan_and_independent_rows_in_large_tiles(M, N, out, e8m0):
    """NaN in a row of x, in a row's scales, in an output's weights and in the scales
    of 128 outputs; other values of the rows before do not matter."""
    K = 640
    w, ws, x, xs = operands(M, N, K, e8m0, M, spread=True)
    clean = run((w, ws, x, xs), out)
    x2, xs2, w2, ws2 = x.clone(), xs.clone(), w.clone(), ws.clone()
    x2.view(torch.uint8)[M - 1, 200] = 0x7F
    x2.view(torch.uint8)[1] = x2.view(torch.uint8)[1].flip(0)
    w2.view(torch.uint8)[130, 7] = 0xFF
    if e8m0:
        xs2.view(torch.uint8)[M // 2, 3] = 0xFF
        ws2.view(torch.uint8)[3, 4] = 0xFF
    else:
        xs2[M // 2, 3] = float("nan")
        ws2[3, 4] = float("nan")
    got = run((w2, ws2, x2, xs2), out)
    hit = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    hit[M - 1] = hit[M // 2] = True
    hit[:, 130] = True
    hit[:, 384:512] = True
    rest = ~hit
    rest[1] = False
    if out == "e4m3":
        q = (got[0] & 127) == 127
        assert bool(q[hit].all())
        rest[:, 128:256] = False                  # the scale of 130's block may move
        assert torch.equal(got[0][rest], clean[0][rest])
    else:
        assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("M", [3, 40, 200])
def test_zero_blocks_and_extreme_scales(M):
    N, K = 200, 512
    for e8m0 in (True, False):
        w, ws, x, xs = operands(M, N, K, e8m0, M)
        x.view(torch.uint8)[0] = 0
        x.view(torch.uint8)[-1, :256] = 0
        if e8m0:
            xs.view(torch.uint8)[0] = 1       # 2^-126, the scale of a block of zeros
            xs.view(torch.uint8)[1] = 127 + 60
            ws.view(torch.uint8)[:, 1] = 127 - 70
        else:
            xs[0], xs[1], ws[:, 1] = 2.0 ** -126, 2.0 ** 60, 2.0 ** -70
        y = check((w, ws, x, xs), "f32")
        assert not bool(y[0].any())


@pytest.mark.parametrize("M,N,K", [(1, 512, 4096), (40, 256, 4096), (150, 384, 2560)])
def test_graph_replays_and_the_workspace_stays_zero(M, N, K):
    ops = operands(M, N, K, True, 3)
    st = torch.cuda.Stream()
    y = torch.empty((M, N), device="cuda")
    size = rq.rq_gemm_fp8_workspace_size([(N, K)], M, rq.RQ_SCALE_E8M0, rq.RQ_TYPE_F32)
    area = torch.zeros(max(size, 65536) // 4, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    call = rq.prepare("rq_gemm_fp8", [(*ops, None, y, N, K)], stream=st, workspace=area)
    x = ops[2].view(torch.uint8)
    eager = []
    for k in range(2):
        call()
        torch.cuda.synchronize()
        eager.append(y.clone())
        x.bitwise_xor_(0x80)                  # -x
    assert not torch.equal(*eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for k in range(4):
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[k % 2])
        assert not bool(area[:16384].any())
        x.bitwise_xor_(0x80)


def test_graph_replays_with_ranges_of_k():
    M, N, K = 1100, 1152, 5120
    ops = operands(M, N, K, True, 3)
    size = rq.rq_gemm_fp8_workspace_size([(N, K)], M, rq.RQ_SCALE_E8M0, rq.RQ_TYPE_F16)
    area = torch.zeros(size // 4, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    y = torch.empty((M, N), dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    call = rq.prepare("rq_gemm_fp8", [(*ops, None, y, N, K)], stream=st, workspace=area)
    x = ops[2].view(torch.uint8)
    eager = []
    for k in range(2):
        call()
        torch.cuda.synchronize()
        eager.append(y.clone())
        x.bitwise_xor_(0x80)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for k in range(4):
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[k % 2])
        assert not bool(area[:16384].any())
        x.bitwise_xor_(0x80)


def test_two_streams_at_once():
    """Each stream's calls with the workspace that the binding keeps for it."""
    work = [(operands(40, 512, 8192, True, s), operands(200, 384, 2560, False, s),
             operands(300, 4096, 5120, False, s)) for s in (1, 2)]
    outs = ("f32", "f32", "f16")

    def step(w):
        return [run(o, out) for o, out in zip(w, outs)]
    want = [step(w) for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(20):
        for w, s, g in zip(work, streams, got):
            with torch.cuda.stream(s):
                ys = []
                for o, out in zip(w, outs):
                    y = torch.empty((o[2].shape[0], o[0].shape[0]), device="cuda",
                                    dtype=torch.float16 if out == "f16" else torch.float32)
                    rq.rq_gemm_fp8([(*o, None, y, *o[0].shape)])
                    ys.append(y)
                g.append(ys)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for ys in g:
            assert all(torch.equal(a, b) for a, b in zip(ys, w))


def test_two_graphs_at_once():
    """Graphs of calls that would split K, captured on one stream that has a workspace
    and replayed on two: each gives what the call without a workspace does."""
    M, N, K = 1100, 1152, 5120
    work = [operands(M, N, K, True, s) for s in (1, 2)]
    want = [run(o, "f16", workspace=None) for o in work]
    ys = [torch.empty((M, N), dtype=torch.float16, device="cuda") for _ in work]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    with torch.cuda.stream(side):
        for o, y in zip(work, ys):
            rq.rq_gemm_fp8([(*o, None, y, N, K)])
    torch.cuda.synchronize()
    for o, y in zip(work, ys):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            for _ in range(10):
                rq.rq_gemm_fp8([(*o, None, y, N, K)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for y in ys:
            y.fill_(float("nan"))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for y, w in zip(ys, want))


@pytest.mark.parametrize("out", OUTS)
def test_zero_blocks_beside_the_smallest_scales(out):
    """A row that rq_quant_fp8 makes of zeros (scales of 2^-126) and weights with
    scales of 2^-20: the products of the scales are below 2^-126, and add zero."""
    for M, N in ((3, 256), (40, 384), (300, 384), (1300, 1024), (4200, 3840)):
        w, ws, x, xs = operands(M, N, 256, True, M)
        x.view(torch.uint8)[1] = 0
        xs.view(torch.uint8)[1] = 1
        ws.view(torch.uint8)[:] = 107
        y = run((w, ws, x, xs), out)
        if out == "e4m3":
            assert not bool((y[0][1] & 127).any()) and bool((y[1][1] == 1).all())
        else:
            check((w, ws, x, xs), out)
            assert not bool(y[1].any())


def test_the_same_call_gives_the_same_bits():
    ops = operands(61, 1000, 5120, False, 9)
    first = run(ops)
    for _ in range(10):
        assert torch.equal(run(ops), first)


def test_a_run_of_the_calls_together():
    """Mixes quantized, three products, their norm quantized, the output product
    onto a residual, FFN key and value: against the same steps in 64 bits on the
    values that each call was given."""
    D, H = 512, 8
    g = torch.Generator().manual_seed(5)
    for T in (1, 24, 170):
        x = (torch.randn((3, T, D), generator=g)).half().cuda()
        mats = {n: (F.random_codes(g, *s), F.random_scales(g, s[0] // 128, s[1] // 128, True,
                                                         -16, -14))
                for n, s in (("r", (D, D)), ("k", (D, D)), ("v", (D, D)), ("o", (D, D)),
                             ("key", (4 * D, D)), ("value", (D, 4 * D)))}

        def blocks(m, n):
            return (torch.empty((m, n), dtype=F.E4M3, device="cuda"),
                    torch.empty((m, n // 128), dtype=F.E8M0, device="cuda"))
        q, s = blocks(3 * T, D)
        rq.rq_quant_fp8(x.view(3 * T, D), q, s)
        want, scales = F.quant_ref(x.view(3 * T, D).cpu().numpy())
        assert F.same(F.values(q), want) and F.same(F.values(s), scales)
        ys = [torch.empty((T, D), device="cuda") for _ in range(3)]
        ins = [(q[i * T:(i + 1) * T], s[i * T:(i + 1) * T]) for i in range(3)]
        if (T * D) % 16 == 0:
            rq.rq_gemm_fp8([(*mats[n], *xi, None, y, D, D) for n, xi, y in zip("rkv", ins, ys)])
        for n, xi, y in zip("rkv", ins, ys):
            ref, mag = F.gemm_ref(*mats[n], *xi)
            assert bool(((y.double() - ref).abs() <= F.gemm_bound(ref, mag, D, "f32")).all())
        w, r_k = 1 + 0.1 * torch.randn(D, generator=g), 0.1 * torch.randn(D, generator=g)
        gate = torch.randn((T, D), generator=g)
        r, k, v = ys
        o, h = blocks(T, D), torch.empty((T, D), dtype=torch.float16, device="cuda")
        args = (r * k, H, w.cuda(), None, 64e-5)
        more = dict(bonus=(r, k, r_k.cuda(), v), gate=gate.cuda())
        rq.rq_groupnorm(*args, o, **more)
        rq.rq_groupnorm(*args, h, **more)
        n = lambda t: t.cpu().numpy()  # noqa: E731
        ref, b = F.norm_ref(n(r * k), H, n(w), None, 64e-5, (n(r), n(k), n(r_k), n(v)), n(gate), 0)
        assert np.all(np.abs(n(h) - ref) <= b + F.HALF * (np.abs(ref) + b) + 2.0 ** -25)
        want, scales = F.quant_ref(n(h))
        assert F.same(F.values(o[0]), want) and F.same(F.values(o[1]), scales)
        stream = torch.randn((T, D), generator=g).cuda()
        before = stream.clone()
        rq.rq_gemm_fp8([(*mats["o"], *o, stream, stream, D, D)])
        ref, mag = F.gemm_ref(*mats["o"], *o, before)
        assert bool(((stream.double() - ref).abs() <= F.gemm_bound(ref, mag, D, "f32")).all())
        key = blocks(T, 4 * D)
        rq.rq_gemm_fp8([(*mats["key"], *o, None, key, 4 * D, D)], act=rq.RQ_ACT_RELU2)
        want = two_calls((*mats["key"], *o), rq.RQ_ACT_RELU2)
        assert torch.equal(key[0].view(torch.uint8), want[0])
        assert torch.equal(key[1].view(torch.uint8), want[1])
        before = stream.clone()
        rq.rq_gemm_fp8([(*mats["value"], *key, stream, stream, D, 4 * D)])
        ref, mag = F.gemm_ref(*mats["value"], *key, before)
        assert bool(((stream.double() - ref).abs() <= F.gemm_bound(ref, mag, 4 * D, "f32")).all())
