"""rq_logits against the documented steps, each rounded to binary32 in the
documented order: the outputs have to be the same bits, and the tokens equal
(ties to the lowest)."""
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


def make(M, V, L, nb, nm, seed):
    """Logits and the host form of every option (rows of ragged length)."""
    g = np.random.default_rng(seed)
    z = (g.standard_normal((M, V)) * 3).astype(np.float32)
    hist = []
    for m in range(M):
        n = int(g.integers(0, L + 1)) if L else 0
        hist.append(((g.random(n) ** 3 * V).astype(np.int64), int(g.integers(0, n + 1))))
    pen = {k: g.random(M).astype(np.float32) + (1 if k == "repetition" else 0)
           for k in ("repetition", "presence", "frequency")}
    bias = []
    for m in range(M):
        n = int(g.integers(0, nb + 1)) if nb else 0
        bias.append((g.integers(0, V, n), (g.standard_normal(n) * 5).astype(np.float32)))
    bits = g.random((nm, V)) < 0.6
    which = g.integers(-1, nm + 1, M) if nm else None  # nm itself: out of range
    return z, hist, pen, bias, bits, which


def ragged(rows, dtype):
    off = R.offsets_of([len(r) for r in rows])
    flat = np.concatenate([np.asarray(r) for r in rows]) if off[-1] else np.zeros(0)
    return torch.from_numpy(flat.astype(dtype)).cuda(), R.dev_ints(off)


def device_args(hist=None, pen=None, bias=None, bits=None, which=None, prompt=True):
    kw = {}
    if hist is not None:
        toks, off = ragged([h[0] for h in hist], np.int32)
        given = R.dev_ints([h[1] for h in hist]) if prompt else None
        kw["history"] = (toks, off, given)
        for k, v in (pen or {}).items():
            kw[k] = torch.from_numpy(v).cuda()
    if bias is not None:
        ids, off = ragged([b[0] for b in bias], np.int32)
        vals, _ = ragged([b[1] for b in bias], np.float32)
        kw["bias"] = (ids, vals, off)
    if bits is not None and which is not None:
        kw["masks"] = (R.pack_masks(bits).cuda(), R.dev_ints([int(w) for w in which]))
    return kw


def same_bits(got, want):
    g, w = got.cpu().numpy(), want
    nan = np.isnan(w)
    return np.array_equal(np.isnan(g), nan) and np.array_equal(g.view(np.int32)[~nan],
                                                               w.view(np.int32)[~nan])


def run(z, inplace=False, tokens=True, **kw):
    M, V = z.shape
    out, ok = R.guarded((M, V), torch.float32, -77.0)
    src = torch.from_numpy(z).cuda()
    if inplace:
        out.copy_(src)
        src = out
    tok, t_ok = R.guarded((M,), torch.int32, -9)
    rq.rq_logits(src, out, tok if tokens else None, **kw)
    assert ok() and t_ok()
    return out, tok


@pytest.mark.parametrize("V", [1, 3, 31, 33, 4095, 4096, 4097, 10001, 65536, 65529])
@pytest.mark.parametrize("M", [1, 5])
def test_everything_together(M, V):
    say(f"[logits] M {M} V {V}")
    z, hist, pen, bias, bits, which = make(M, V, 600, 40, 3, V + M)
    want, tok = R.logits_ref(z, hist, **pen, bias=bias, masks=(bits, which))
    for inplace in (False, True):
        out, got = run(z, inplace, **device_args(hist, pen, bias, bits, which))
        assert same_bits(out, want)
        assert np.array_equal(got.cpu().numpy(), tok)


@pytest.mark.parametrize("parts", ["h", "b", "m", "hb", "hm", "bm", ""])
def test_each_step_alone(parts):
    M, V = 4, 9001
    z, hist, pen, bias, bits, which = make(M, V, 300, 20, 2, 11)
    h, b, m = (hist if "h" in parts else None), (bias if "b" in parts else None), "m" in parts
    want, tok = R.logits_ref(z, h, **(pen if h else {}), bias=b,
                             masks=(bits, which) if m else None)
    kw = device_args(h, pen if h else None, b, bits if m else None, which if m else None)
    out, got = run(z, **kw)
    assert same_bits(out, want) and np.array_equal(got.cpu().numpy(), tok)
    out, _ = run(z, tokens=False, **kw)
    assert same_bits(out, want)


@pytest.mark.parametrize("which", ["repetition", "presence", "frequency"])
def test_one_penalty_and_no_prompt(which):
    M, V = 3, 5000
    z, hist, pen, _, _, _ = make(M, V, 2000, 0, 0, 12)
    one = {which: pen[which]}
    all_generated = [(t, 0) for t, _ in hist]
    want, tok = R.logits_ref(z, all_generated, **one)
    out, got = run(z, **device_args(hist, one, prompt=False))
    assert same_bits(out, want) and np.array_equal(got.cpu().numpy(), tok)


@pytest.mark.parametrize("L", [1, 63, 4096, 20000])
def test_long_histories_of_one_token(L):
    """The same token L times (the count is exact), and a history of prompts only."""
    V = 8200
    z = np.random.default_rng(1).standard_normal((2, V)).astype(np.float32)
    hist = [(np.full(L, 4100), 0), (np.arange(L) % V, L)]
    pen = {"repetition": np.float32([1.3, 1.7]), "presence": np.float32([0.5, 0.5]),
           "frequency": np.float32([0.01, 0.01])}
    want, tok = R.logits_ref(z, hist, **pen)
    out, got = run(z, **device_args(hist, pen))
    assert same_bits(out, want) and np.array_equal(got.cpu().numpy(), tok)


def test_a_bias_given_twice_counts_once_the_last():
    V = 5000
    z = np.zeros((2, V), np.float32)
    bias = [(np.array([7, 7, 4999, 7, 4999]), np.float32([1, 2, 3, 4, 5])),
            (np.array([7] * 1000), np.arange(1000, dtype=np.float32))]
    out, tok = run(z, **device_args(bias=bias))
    o = out.cpu().numpy()
    assert o[0, 7] == 4 and o[0, 4999] == 5 and o[1, 7] == 999
    assert tok.tolist() == [4999, 7]


def test_rows_whose_mask_leaves_nothing():
    V = 9000
    z = np.random.default_rng(2).standard_normal((3, V)).astype(np.float32)
    bits = np.zeros((2, V), bool)
    bits[1, 8999] = True
    out, tok = run(z, **device_args(bits=bits, which=[0, 1, -1]))
    assert tok.tolist() == [-1, 8999, int(z[2].argmax())]
    o = out.cpu().numpy()
    assert np.all(np.isneginf(o[0])) and np.isneginf(o[1, :8999]).all() and o[1, 8999] == z[1, 8999]


def test_infinities_and_nan_in_and_out_of_masked_places():
    V = 6000
    g = np.random.default_rng(3)
    z = g.standard_normal((4, V)).astype(np.float32)
    z[0, :10] = np.nan
    z[1, 100], z[1, 200] = np.inf, np.nan
    z[2] = -np.inf
    z[3] = np.finfo(np.float32).min
    bits = np.ones((1, V), bool)
    bits[0, :150] = False
    for which in ([0, 0, 0, 0], [-1, -1, -1, -1]):
        want, tok = R.logits_ref(z, masks=(bits, which))
        out, got = run(z, **device_args(bits=bits, which=which))
        assert same_bits(out, want)
        assert np.array_equal(got.cpu().numpy(), tok)
    assert tok[2] == -1 and tok[3] == 0 and tok[1] == 100


def test_ties_go_to_the_lowest_token():
    V = 65536
    z = np.zeros((4, V), np.float32)
    z[0, [60000, 5000, 40000]] = 2.0
    z[1] = -0.0
    z[1, 9000] = 0.0
    z[2] = -1.0
    z[3, ::2] = -0.0
    out, tok = run(z)
    assert tok.tolist() == [5000, 0, 0, 0]


def test_entries_and_offsets_out_of_range_are_ignored():
    M, V = 3, 4200
    z = np.random.default_rng(4).standard_normal((M, V)).astype(np.float32)
    toks = np.array([-1, V, 2 ** 31 - 1, -2 ** 31, 5, 5])
    pen = {"frequency": np.ones(M, np.float32)}
    want, tok = R.logits_ref(z, [(toks, 0)] * M, **pen)
    out, got = run(z, **device_args([(toks, 0)] * M, pen, bias=[(toks[:4], np.ones(4))] * M))
    assert same_bits(out, want) and np.array_equal(got.cpu().numpy(), tok)
    # offsets beyond the lists, or backwards, are cut to them
    h = (R.dev_ints([1, 2, 3]), R.dev_ints([-4, 2, 1, 99]), R.dev_ints([-5, 7, 0]))
    b = (R.dev_ints([9]), torch.ones(1, device="cuda"), R.dev_ints([50, -3, 0, 1]))
    out, _ = run(z, history=h, frequency=torch.ones(M, device="cuda"), bias=b)
    want, _ = R.logits_ref(z, [([1, 2], 0), ([], 0), ([2, 3], 0)], frequency=[1, 1, 1],
                           bias=[([], []), ([], []), ([9], [1])])
    # the first row's history keeps its place, cut to the list
    assert same_bits(out, want)


def test_empty_lists():
    z = np.random.default_rng(5).standard_normal((2, 100)).astype(np.float32)
    out, tok = run(z, **device_args([([], 0), ([], 0)], None, [([], []), ([], [])]))
    assert same_bits(out, z) and tok.tolist() == z.argmax(1).tolist()


def test_graph_replays_and_the_workspace_stays_zero():
    M, V = 5, 65536
    z, hist, pen, bias, bits, which = make(M, V, 200, 5, 2, 6)
    src = torch.from_numpy(z).cuda()
    out, tok = torch.empty_like(src), torch.empty(M, dtype=torch.int32, device="cuda")
    kw = device_args(hist, pen, bias, bits, which)
    ws = torch.zeros(rq.RQ_LOGITS_WORKSPACE_BYTES // 4, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = rq.prepare("rq_logits", src, out, tok, stream=s, workspace=ws, **kw)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    for k in range(4):
        zk = np.roll(z, 1000 * k, axis=1).copy()
        src.copy_(torch.from_numpy(zk))
        out.fill_(float("nan"))
        tok.fill_(-5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want, t = R.logits_ref(zk, hist, **pen, bias=bias, masks=(bits, which))
        assert same_bits(out, want) and np.array_equal(tok.cpu().numpy(), t)
        assert not bool(ws.any())


def test_more_rows_than_compute_units():
    M, V = 4096, 4100
    z = np.random.default_rng(7).standard_normal((M, V)).astype(np.float32)
    out, tok = run(z)
    assert same_bits(out, z) and np.array_equal(tok.cpu().numpy(), z.argmax(1))


@pytest.mark.parametrize("M,V,L,nb", [(20, 65529, 500, 30), (6, 150001, 800, 0), (260, 40001, 60, 4),
                                      (300, 66003, 40, 0), (400, 1999, 50, 3), (70, 2, 9, 2)])
def test_ranges_of_every_length(M, V, L, nb):
    """Rows dealt out over one and several workgroups, ranges in one and several
    slices."""
    say(f"[logits] M {M} V {V}")
    z, hist, pen, bias, bits, which = make(M, V, L, nb, 2, M + V)
    bias = bias if nb else None
    want, tok = R.logits_ref(z, hist, **pen, bias=bias, masks=(bits, which))
    out, got = run(z, **device_args(hist, pen, bias, bits, which))
    assert same_bits(out, want) and got.tolist() == tok.tolist()


@pytest.mark.parametrize("M,V", [(3, 9001), (30, 65529)])
@pytest.mark.parametrize("given", [0, 10, 40000 - 32768, 40000 - 32767, 40000])
def test_counts_past_fifteen_bits(M, V, given):
    """One row with more generated tokens than a 16-bit count holds, and at its
    limit, most of them one token; the others short."""
    say(f"[logits] M {M} V {V} given {given}")
    z, hist, pen, bias, bits, which = make(M, V, 50, 3, 2, 9)
    g = np.random.default_rng(8)
    toks = np.where(g.random(40000) < 0.98, V - 1, g.integers(0, V, 40000))
    hist[1] = (toks, given)
    want, tok = R.logits_ref(z, hist, **pen, bias=bias, masks=(bits, which))
    out, got = run(z, **device_args(hist, pen, bias, bits, which))
    assert same_bits(out, want) and got.tolist() == tok.tolist()


@pytest.mark.parametrize("M,V", [(128, 65536), (256, 32768)])
def test_ranges_of_64_kib_of_counts(M, V):
    """A history alone, counted in exactly 64 KiB of LDS."""
    say(f"[logits] M {M} V {V}")
    z, hist, pen, _, _, _ = make(M, V, 20, 0, 0, M)
    want, tok = R.logits_ref(z, hist, **pen)
    out, got = run(z, **device_args(hist, pen))
    assert same_bits(out, want) and got.tolist() == tok.tolist()
