"""rq_lora and rq_logits on two streams at once, each with the workspace the
binding keeps for its stream, between products that split K in the same
workspaces: every result is the one of the same calls in turn on one stream,
to the bit, and the records at a workspace's start are zero afterwards."""
import pytest
import torch

import gemm_rwkv_decode_amd as rq
from gemm_rwkv_decode_amd import synth as S
from tests import aroundtest as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


class Work:
    """A decode step's calls around one product, on inputs of their own."""

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        M, N, K, V = 32, 2048, 2048, 40001
        self.M, self.N, self.K, self.V = M, N, K, V
        f = S.INT4_G64
        codes = torch.randint(-7, 8, (N, K), generator=g).to(torch.int8)
        scales = torch.rand((N, K // f.group), generator=g).half() * 0.02
        p = S.encode(codes, f, scales=scales)
        self.fmt, self.q, self.s = f, p.qweight.cuda(), p.scales.cuda()
        ranks = [16, 32, 8, 24]
        self.off = R.dev_ints(R.offsets_of(ranks))
        self.ids = R.dev_ints(torch.randint(-1, 4, (M,), generator=g).tolist())
        self.a = R.randn(g, sum(ranks), K, scale=K ** -0.5, dtype=torch.float16).cuda()
        self.b = R.randn(g, sum(ranks) * N, scale=0.2, dtype=torch.float16).cuda()
        self.x = R.randn(g, M, K, dtype=torch.float16).cuda()
        self.z = R.randn(g, M, V).cuda()
        lens = torch.randint(0, 300, (M,), generator=g).tolist()
        self.hist = torch.randint(0, V, (sum(lens),), generator=g, dtype=torch.int32).cuda()
        self.hoff = R.dev_ints(R.offsets_of(lens))
        self.freq = torch.rand(M, generator=g).cuda()

    def step(self):
        y, out = torch.empty(self.M, self.N, device="cuda"), torch.empty_like(self.z)
        tok = torch.empty(self.M, dtype=torch.int32, device="cuda")
        f = self.fmt
        rq.rq_gemm_smallm(self.q, self.s, None, self.x, y, self.M, self.N, self.K, f.bits, f.group,
                          f.layout)
        rq.rq_lora([(self.a, self.b, self.x, y, y, self.N, self.K)], self.ids, self.off, None, 32)
        rq.rq_logits(self.z, out, tok, history=(self.hist, self.hoff, None), frequency=self.freq)
        return y, out, tok


def test_two_streams_at_once():
    work = [Work(1), Work(2)]
    want = [w.step() for w in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    assert streams[0].cuda_stream != streams[1].cuda_stream
    got = [[], []]
    for _ in range(20):
        for w, s, g in zip(work, streams, got):
            with torch.cuda.stream(s):
                g.append(w.step())
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for k, step in enumerate(g):
            assert all(torch.equal(a, b) for a, b in zip(step, w)), k
    areas = [rq.gemm_workspace(s) for s in streams]
    assert areas[0].data_ptr() != areas[1].data_ptr()
    for a in areas:
        assert not bool(a[:rq.RQ_LOGITS_WORKSPACE_BYTES // 4].any())
