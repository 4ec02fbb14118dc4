"""The block-scaled FP8 calls and the group norm at their largest sizes: arrays whose
bytes, values or work-items pass 2^31 and 2^32.  The data repeats, and so has what
comes out to the bit; one period is checked against the formula."""
import gc

import pytest
import torch

import gemm_rwkv_decode_amd as rq
from tests import fp8test as F

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _room():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("not enough free memory")
    yield
    gc.collect()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def say(msg):
    print(msg, flush=True)


def repeated(t, rows):
    """t's rows over and over, ``rows`` in all."""
    out = torch.empty((rows,) + t.shape[1:], dtype=t.dtype, device="cuda")
    src, dst = (t, out) if t.element_size() > 1 else (t.view(torch.uint8), out.view(torch.uint8))
    n = src.shape[0]
    whole = rows // n * n
    dst[:whole].view(rows // n, *src.shape).copy_(src.expand(rows // n, *src.shape))
    dst[whole:] = src[:rows - whole]
    return out


def assert_repeats(t, first):
    if t.element_size() == 1:
        t, first = t.view(torch.uint8), first.view(torch.uint8)
    n, step = first.shape[0], max(1, (1 << 28) // first.numel())
    for i in range(0, t.shape[0] // n, step):
        part = t[i * n:min((i + step) * n, t.shape[0] // n * n)]
        assert bool((part.view(-1, *first.shape) == first).all()), i
    rest = t.shape[0] % n
    assert torch.equal(t[t.shape[0] - rest:], first[:rest])


@pytest.mark.parametrize("half", [True, False])
def test_quant_past_32_bits(half):
    n, K, M = 1000, 4096, (1 << 20) + 7
    g = torch.Generator().manual_seed(1)
    x = torch.randn((n, K), generator=g).to(torch.float16 if half else torch.float32).cuda()
    q, s = torch.empty((n, K), dtype=torch.uint8, device="cuda"), torch.empty((n, 32), device="cuda")
    rq.rq_quant_fp8(x, q, s, act=rq.RQ_ACT_RELU2)
    say(f"[quant] {M} x {K}")
    qq = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    ss = torch.empty((M, 32), device="cuda")
    rq.rq_quant_fp8(repeated(x, M), qq, ss, act=rq.RQ_ACT_RELU2)
    assert_repeats(qq, q)
    assert_repeats(ss, s)


@pytest.mark.parametrize("T,C,H", [(1 << 24, 32, 1), ((1 << 23) + 5, 1024, 16)])
def test_groupnorm_past_32_bits_of_work_items(T, C, H):
    """In place; 2^24 tokens of one small group, and more than 2^31 lanes."""
    n = 1000
    g = torch.Generator().manual_seed(2)
    y = torch.randn((n, C), generator=g).cuda()
    w, b = torch.randn(C, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    small = torch.empty_like(y)
    rq.rq_groupnorm(y, H, w, b, 1e-5, small)
    want = torch.nn.functional.group_norm(y.double(), H, w.double(), b.double(), eps=1e-5)
    assert float((small.double() - want).abs().max()) <= 1e-4
    say(f"[groupnorm] {T} x {C}")
    big = repeated(y, T)
    rq.rq_groupnorm(big, H, w, b, 1e-5, big)
    assert_repeats(big, small)


def operands(M, N, K, e8m0):
    g = torch.Generator().manual_seed(M + N)
    return (F.random_codes(g, N, K), F.random_scales(g, (N + 127) // 128, K // 128, e8m0),
            F.random_codes(g, M, K), F.random_scales(g, M, K // 128, e8m0))


def within(y, ops, out):
    want, mag = F.gemm_ref(*ops)
    bound = F.gemm_bound(want, mag, ops[0].shape[1], out)
    assert bool(((y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("out", ["f32", "f16", "e4m3"])
def test_gemm_rows_past_32_bits(out):
    n, N, K, M = 512, 256, 4096, (1 << 20) + 131
    w, ws, x, xs = ops = operands(n, N, K, out == "f32")
    say(f"[gemm_fp8] {M} rows of {K}")
    args = (w, ws, repeated(x, M), repeated(xs, M), None)
    if out == "e4m3":
        y = torch.empty((M, N), dtype=torch.uint8, device="cuda"), torch.empty((M, 2), device="cuda")
        h = torch.empty((M, N), dtype=torch.float16, device="cuda")
        rq.rq_gemm_fp8([(*args, y, N, K)])
        rq.rq_gemm_fp8([(*args, h, N, K)])
        q, s = torch.empty_like(y[0]), torch.empty_like(y[1])
        rq.rq_quant_fp8(h, q, s)
        assert torch.equal(q, y[0]) and torch.equal(s, y[1])
    else:
        y = torch.empty((M, N), dtype=torch.float16 if out == "f16" else torch.float32,
                        device="cuda")
        rq.rq_gemm_fp8([(*args, y, N, K)])
        within(y[:n], ops, out)
        assert_repeats(y, y[:n].clone())


@pytest.mark.parametrize("M,out", [(1, "f32"), (9, "f32"), (40, "f32"), (40, "f16"), (130, "f16"),
                                   (130, "f32")])
def test_gemm_weights_past_32_bits(M, out):
    n, K, N = 512, 4096, (1 << 20) + 256
    w, ws, x, xs = ops = operands(M, n, K, True)
    say(f"[gemm_fp8] M {M}, {N} outputs of {K}")
    y = torch.empty((M, N), dtype=torch.float16 if out == "f16" else torch.float32, device="cuda")
    rq.rq_gemm_fp8([(repeated(w, N), repeated(ws, N // 128), x, xs, None, y, N, K)])
    within(y[:, :n], ops, out)
    t = y.t().contiguous()
    assert_repeats(t, t[:n].clone())


@pytest.mark.parametrize("M", [1, 3])
def test_gemm_most_outputs(M):
    """Eight products of 2^24 outputs: as many tiles as one call can have."""
    n, N, K = 512, 1 << 24, 128
    w, ws, x, xs = ops = operands(M, n, K, True)
    big, scales = repeated(w, N), repeated(ws, N // 128)
    ys = [torch.empty((M, N), device="cuda") for _ in range(8)]
    say(f"[gemm_fp8] M {M}, 8 x {N} outputs of {K}")
    rq.rq_gemm_fp8([(big, scales, x, xs, None, y, N, K) for y in ys])
    within(ys[0][:, :n], ops, "f32")
    for y in ys:
        t = y.t().contiguous()
        assert_repeats(t, t[:n].clone())
        assert torch.equal(t, ys[0].t())


def test_gemm_longest_rows():
    """K = 2^22, the largest there is."""
    M, N, K = 3, 40, 1 << 22
    w, ws, x, xs = operands(M, N, K, True)
    ops = w, ws, x, (xs.float() * 2.0 ** -6).to(F.E8M0)  # binary16 outputs stay finite
    say(f"[gemm_fp8] K {K}")
    y = torch.empty((M, N), device="cuda")
    rq.rq_gemm_fp8([(*ops, None, y, N, K)])
    within(y, ops, "f32")
    x = torch.cat([ops[2].view(torch.uint8)] * 7)[:20].contiguous()
    xs = torch.cat([ops[3].view(torch.uint8)] * 7)[:20].contiguous()
    z = torch.empty((20, N), dtype=torch.float16, device="cuda")
    rq.rq_gemm_fp8([(*ops[:2], x, xs, None, z, N, K)])
    within(z, (*ops[:2], x, xs), "f16")
