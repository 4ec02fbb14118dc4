"""rq_lora against the formula in 64 bits.

Tolerance.  A (and x) enter exact products; their sum is accumulated in
binary32 over K/32 steps of 32-term sums, over at most 64 partial sums, and
then over rank/32 steps of the second product: at most (K/32 + 32 + 64 +
rank/32 + 32 + 4) units of 2^-24 of the sum of absolute products.  The split of
t in two binary16 parts adds 2^-22 of the row's largest t, itself below the sum
of absolute products divided by |B|; 2^-21 covers it for the B used here."""
import numpy as np
import pytest
import torch

import gemm_rwkv_decode_amd as rq
from tests import aroundtest as R
from tests.rqtest import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def pool(N, K, ranks, seed, ascale=None):
    g = torch.Generator().manual_seed(seed)
    total = sum(ranks)
    a = R.randn(g, total, K, scale=ascale or K ** -0.5, dtype=torch.float16)
    b = R.randn(g, total * N, scale=0.2, dtype=torch.float16)
    return a, b


def rows(M, N, K, seed, massive=True):
    g = torch.Generator().manual_seed(seed)
    x = R.randn(g, M, K, dtype=torch.float16)
    if massive:
        x[:, K // 3] *= 50
    return x, R.randn(g, M, N)


def run(probs, ids, off, scales, max_rank, mode="apart", **kw):
    """mode: y_in apart, in place, or none."""
    out, checks = [], []
    arg = []
    for a, b, x, y_in, N, K in probs:
        y, ok = R.guarded((x.shape[0], N), torch.float32, float("nan"))
        yi = None
        if mode == "apart":
            yi = y_in.cuda()
        elif mode == "inplace":
            y.copy_(y_in)
            yi = y
        arg.append((a.cuda(), b.cuda(), x.cuda(), yi, y, N, K))
        out.append(y)
        checks.append(ok)
    rq.rq_lora(arg, R.dev_ints(ids), R.dev_ints(off),
               None if scales is None else scales.cuda(), max_rank, **kw)
    assert all(ok() for ok in checks)
    return out


def compare(out, probs, ids, off, scales, max_rank, mode="apart", what=""):
    for y, (a, b, x, y_in, N, K) in zip(out, probs):
        yi = None if mode == "none" else y_in.numpy()
        ref, bound = R.lora_ref((a.numpy(), b.numpy(), x.numpy(), yi, N, K), ids, off,
                                None if scales is None else scales.numpy(), a.shape[0], max_rank)
        tol = ((K / 32 + 132 + max_rank / 32) * R.EPS + 2.0 ** -21) * bound + 1e-37
        err = np.abs(y.cpu().double().numpy() - ref)
        bad = ~(err <= tol)
        assert not bad.any(), f"{what}: {bad.sum()} outside, worst {np.nanmax(err / tol):.3g}"


@pytest.mark.parametrize("N,K", [(768, 768), (4096, 2048), (1000, 512), (37, 8), (1, 40), (261, 1096),
                                 (2049, 264)])
@pytest.mark.parametrize("M", [1, 2, 17, 64, 65, 150])
def test_sizes(N, K, M):
    say(f"[lora] M {M} N {N} K {K}")
    ranks = [8, 64, 16, 128, 40]
    off = R.offsets_of(ranks)
    a, b = pool(N, K, ranks, N + K)
    x, y_in = rows(M, N, K, M)
    ids = torch.randint(-1, len(ranks), (M,), generator=torch.Generator().manual_seed(M)).tolist()
    scales = torch.tensor([0.5, 1.0, 2.0, -1.5, 0.25])
    probs = [(a, b, x, y_in, N, K)]
    for mode in ("apart", "inplace", "none"):
        out = run(probs, ids, off, scales, 128, mode)
        compare(out, probs, ids, off, scales, 128, mode, f"{N}x{K} M={M} {mode}")


@pytest.mark.parametrize("rank", list(range(8, 129, 8)))
def test_every_rank(rank):
    N, K, M = 300, 320, 21
    off = [0, rank, 2 * rank]
    a, b = pool(N, K, [rank, rank], rank)
    x, y_in = rows(M, N, K, rank)
    ids = [i % 3 - 1 for i in range(M)]
    probs = [(a, b, x, y_in, N, K)]
    compare(run(probs, ids, off, None, rank), probs, ids, off, None, rank)


@pytest.mark.parametrize("ids", [[0] * 64, [2] * 130, list(range(64)), [-1] * 70, [63 - i for i in range(64)],
                                 [5] * 3 + [-1] + [5] * 60, [1000, -1000, 2 ** 31 - 1, -2 ** 31, 64, 0]])
def test_groups_of_rows(ids):
    """All rows one adapter, every row its own, none, and ids out of range."""
    N, K, M = 272, 256, len(ids)
    ranks = [8 + 8 * (i % 4) for i in range(64)]
    off = R.offsets_of(ranks)
    a, b = pool(N, K, ranks, 1)
    x, y_in = rows(M, N, K, 2)
    probs = [(a, b, x, y_in, N, K)]
    scales = torch.rand(64, generator=torch.Generator().manual_seed(3)) + 0.5
    for mode in ("apart", "inplace", "none"):
        compare(run(probs, ids, off, scales, 32, mode), probs, ids, off, scales, 32, mode)


def test_projections_of_different_sizes_in_one_call():
    ranks, M = [16, 8, 32], 33
    off = R.offsets_of(ranks)
    probs = []
    for i, (N, K) in enumerate([(768, 768), (3072, 768), (768, 3072), (5, 16)]):
        a, b = pool(N, K, ranks, i)
        x, y_in = rows(M, N, K, 10 + i)
        probs.append((a, b, x, y_in, N, K))
    ids = [i % 4 - 1 for i in range(M)]
    compare(run(probs, ids, off, None, 32), probs, ids, off, None, 32)


def test_offsets_that_describe_no_adapter_leave_the_row():
    """Ranks that are empty, too large, no multiple of 8, or outside the pool."""
    N, K = 64, 64
    a, b = pool(N, K, [64], 1)
    for off in ([0, 0, 8], [8, 0, 8], [0, 40, 48], [0, 4, 12], [-8, 0, 8], [0, 72, 80],
                [64, 72, 2 ** 31 - 8], [-2 ** 31, 2 ** 31 - 8, 0]):
        ids = [0, 1, 0, 1]
        x, y_in = rows(4, N, K, 5)
        probs = [(a, b, x, y_in, N, K)]
        compare(run(probs, ids, off, None, 32), probs, ids, off, None, 32, what=str(off))


def test_large_activations_and_a_zero_row():
    """t far above binary16's range, tiny t, and a row of zeros."""
    N, K, M = 128, 1024, 6
    a, b = pool(N, K, [16], 1, ascale=1.0)
    x, y_in = rows(M, N, K, 3, massive=False)
    x[0] = 60000.0
    x[1] *= 1e-6
    x[2] = 0
    probs = [(a, b, x, y_in, N, K)]
    compare(run(probs, [0] * M, [0, 16], None, 16, "none"), probs, [0] * M, [0, 16], None, 16, "none")
    out = run(probs, [0] * M, [0, 16], None, 16, "none")[0]
    assert not bool(out[2].any())


def test_a_row_that_is_not_finite_stays_alone():
    N, K, M = 96, 256, 20
    a, b = pool(N, K, [24, 8], 1)
    x, y_in = rows(M, N, K, 3)
    ids = [i % 3 - 1 for i in range(M)]
    clean = run([(a, b, x, y_in, N, K)], ids, [0, 24, 32], None, 24)[0].clone()
    x2 = x.clone()
    x2[4, 7] = float("inf")   # id 0
    x2[9, 0] = float("nan")   # id -1: no adapter reads it
    got = run([(a, b, x2, y_in, N, K)], ids, [0, 24, 32], None, 24)[0]
    keep = [m for m in range(M) if m != 4]
    assert torch.equal(got[keep], clean[keep])
    assert not bool(torch.isfinite(got[4]).all())


def test_results_do_not_depend_on_the_order_of_rows():
    N, K, M = 260, 1024, 64
    ranks = [16] * 9
    off = R.offsets_of(ranks)
    a, b = pool(N, K, ranks, 1)
    x, y_in = rows(M, N, K, 2)
    g = torch.Generator().manual_seed(4)
    ids = torch.randint(-1, 9, (M,), generator=g)
    p = torch.randperm(M, generator=g)
    y = run([(a, b, x, y_in, N, K)], ids.tolist(), off, None, 16)[0]
    z = run([(a, b, x[p], y_in[p], N, K)], ids[p].tolist(), off, None, 16)[0]
    assert torch.equal(y[p.cuda()], z)


def test_a_pool_past_two_gib():
    """Adapter blocks that start beyond 2^31 bytes of a and b."""
    N = K = 4096
    R_total, M = 280000, 3  # 2.3 GB each
    a = torch.zeros(R_total, K, dtype=torch.float16, device="cuda")
    b = torch.zeros(R_total * N, dtype=torch.float16, device="cuda")
    lo = R_total - 16
    sa, sb = pool(N, K, [16], 1)
    a[lo:] = sa.cuda()
    b[lo * N:] = sb.cuda()
    x, y_in = rows(M, N, K, 2)
    y = torch.empty(M, N, device="cuda")
    rq.rq_lora([(a, b, x.cuda(), y_in.cuda(), y, N, K)], R.dev_ints([0] * M),
               R.dev_ints([lo, R_total]), None, 16)
    compare([y], [(sa, sb, x, y_in, N, K)], [0] * M, [0, 16], None, 16)


def test_graph_reads_ids_at_replay_and_streams_have_their_own_workspace():
    N, K, M = 512, 2048, 8
    ranks = [16, 32, 8]
    off = R.offsets_of(ranks)
    a, b = pool(N, K, ranks, 1)
    x, y_in = rows(M, N, K, 2)
    ids = R.dev_ints([0] * M)
    y = torch.empty(M, N, device="cuda")
    s = torch.cuda.Stream()
    dev = [a.cuda(), b.cuda(), x.cuda(), y_in.cuda()]
    offd = R.dev_ints(off)
    torch.cuda.synchronize()
    call = rq.prepare("rq_lora", [(*dev, y, N, K)], ids, offd, None, 32, stream=s)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for k in range(4):
        now = [(k + m) % 4 - 1 for m in range(M)]
        ids.copy_(torch.tensor(now, dtype=torch.int32))
        y.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        compare([y], [(a, b, x, y_in, N, K)], now, off, None, 32)


def test_a_workspace_of_the_queried_size():
    N, K, M = 256, 4096, 5
    a, b = pool(N, K, [24], 1)
    x, y_in = rows(M, N, K, 2)
    need = rq.rq_lora_workspace_size([(N, K)], M, 1, 24)
    assert need > 0
    ws, ok = R.guarded((need // 4,), torch.float32, 3.0)
    probs = [(a, b, x, y_in, N, K)]
    out = run(probs, [0] * M, [0, 24], None, 24, workspace=ws)
    assert ok()
    compare(out, probs, [0] * M, [0, 24], None, 24)
    want = run(probs, [0] * M, [0, 24], None, 24)
    assert torch.equal(out[0], want[0])
    y = torch.full((M, N), 2.0, device="cuda")
    with pytest.raises(rq.RqError) as e:
        rq.rq_lora([(a.cuda(), b.cuda(), x.cuda(), None, y, N, K)], R.dev_ints([0] * M),
                   R.dev_ints([0, 24]), None, 24, workspace=ws[:-4])
    assert e.value.status == rq.RQ_ERR_SCRATCH
    torch.cuda.synchronize()
    assert bool((y == 2.0).all())


@pytest.mark.parametrize("M,size", [(7, 1.0), (7, 3000.0), (70, 3000.0)])
def test_an_infinite_entry_of_an_adapter_gives_what_the_formula_gives(M, size):
    """Infinities of the formula's sign, beside large finite entries as well; NaN
    where it multiplies a zero."""
    N, K, rank = 200, 256, 16
    a, b = pool(N, K, [rank], 1)
    x, y_in = rows(M, N, K, 2, massive=False)
    x = (x * size).clamp(-6e4, 6e4)
    x[3, 5] = 0
    a[2, 5] = float("inf")
    b.view(N, rank)[11, 2] = 0
    probs = [(a, b, x, y_in, N, K)]
    scales = torch.tensor([-0.5])
    got = run(probs, [0] * M, [0, rank], scales, rank)[0].cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref, _ = R.lora_ref((a.numpy(), b.numpy(), x.numpy(), y_in.numpy(), N, K), [0] * M,
                            [0, rank], scales.numpy(), rank, rank)
    assert np.isinf(ref).sum() == (M - 1) * (N - 1) and np.isnan(ref).sum() == M + N - 1
    assert np.array_equal(got.astype(np.float64), ref, equal_nan=True)
