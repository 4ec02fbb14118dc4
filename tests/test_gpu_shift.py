"""rq_shift against the formula in 64 bits.  The result is rounded once to
binary16 from a binary32 value: |error| <= 2^-11 |out| (half a unit of
binary16) + 2^-22 (|x| + |prev|) (three binary32 roundings) + 2^-25 (half a
subnormal)."""
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


def tensors(T, D, n, nslots, seed):
    g = torch.Generator().manual_seed(seed)
    return (R.randn(g, T, D, dtype=torch.float16), torch.rand((n, D), generator=g).half(),
            R.randn(g, nslots, D, dtype=torch.float16))


def check(out, ref, x, lens, state, slots, start=0):
    got = out.cpu().double().numpy()
    xa = np.abs(x.double().numpy())
    big = max(float(xa.max()), float(np.abs(state.double().numpy()).max()) if state.numel() else 0)
    live = slice(start, start + sum(lens))
    err, r = np.abs(got - ref)[:, live], np.abs(ref)[:, live]
    assert np.all(err <= 2.0 ** -11 * r + 2.0 ** -22 * 2 * big + 2.0 ** -25), err.max()


@pytest.mark.parametrize("D", [8, 64, 768, 2056, 4096])
@pytest.mark.parametrize("lens", [[1], [5], [0, 1, 0, 2], [1] * 9, [17, 3, 0, 8, 1, 4], [40]])
@pytest.mark.parametrize("n", [1, 6, 8])
def test_against_the_formula(D, lens, n):
    T, B = sum(lens), len(lens)
    say(f"[shift] D {D} lens {lens} n {n}")
    x, mu, state0 = tensors(T, D, n, B + 1, D + T)
    slots = torch.randperm(B + 1, generator=torch.Generator().manual_seed(T))[:B].tolist()
    ref, s_ref = R.shift_ref(x.numpy(), mu.numpy(), state0.numpy(), lens, slots)
    state, s_ok = R.guarded((B + 1, D), torch.float16, 5.0)
    state.copy_(state0)
    out, o_ok = R.guarded((n, T, D), torch.float16, float("nan"))
    rq.rq_shift(x.cuda(), mu.cuda(), state, out, R.dev_ints(R.offsets_of(lens)),
                R.dev_ints(slots))
    assert o_ok() and s_ok()
    check(out, ref, x, lens, state0, slots)
    assert np.array_equal(state.cpu().numpy().view(np.uint16), s_ref.view(np.uint16))


def test_mixes_of_zero_and_one_are_exact():
    T, D = 33, 256
    x, _, state0 = tensors(T, D, 2, 1, 1)
    mu = torch.stack([torch.zeros(D), torch.ones(D)]).half()
    out = torch.empty((2, T, D), dtype=torch.float16, device="cuda")
    rq.rq_shift(x.cuda(), mu.cuda(), state0.cuda(), out, R.dev_ints([0, T]))
    assert torch.equal(out[0].cpu(), x)
    # x + (prev - x) in binary32 is exact to the last place of binary16
    want = torch.cat([state0, x[:-1]])
    assert float((out[1].cpu().float() - want.float()).abs().max()) <= 2.0 ** -10 * 4


def test_slots_that_are_not_stored():
    lens, D = [3, 4, 1], 128
    T = sum(lens)
    x, mu, _ = tensors(T, D, 2, 1, 2)
    for state0, slots in ((torch.ones(2, D).half(), [-1, 2, 1]), (None, [0, 1, 2])):
        s = np.zeros((0, D), np.float16) if state0 is None else state0.numpy()
        ref, s_ref = R.shift_ref(x.numpy(), mu.numpy(), s, lens, slots)
        st = None if state0 is None else state0.cuda()
        out = torch.full((2, T, D), float("nan"), dtype=torch.float16, device="cuda")
        rq.rq_shift(x.cuda(), mu.cuda(), st, out, R.dev_ints(R.offsets_of(lens)),
                    R.dev_ints(slots))
        check(out, ref, x, lens, torch.from_numpy(s), slots)
        if st is not None:
            assert np.array_equal(st.cpu().numpy(), s_ref)


def test_offsets_out_of_range_stay_inside():
    """A sequence that leaves 0..T begins nowhere; nothing outside is touched."""
    T, D = 20, 64
    x, mu, state0 = tensors(T, D, 3, 3, 3)
    state, s_ok = R.guarded((3, D), torch.float16, 5.0)
    state.copy_(state0)
    out, o_ok = R.guarded((3, T, D), torch.float16, -1.0)
    rq.rq_shift(x.cuda(), mu.cuda(), state, out, R.dev_ints([-5, 0, 4, T + 100]))
    assert o_ok() and s_ok()
    got = state.cpu()
    assert torch.equal(got[0], state0[0]) and torch.equal(got[2], state0[2])
    assert torch.equal(got[1], x[3])


def test_replays_carry_the_state():
    D, B = 768, 5
    x, mu, state0 = tensors(B, D, 6, B, 4)
    xd, state = x.cuda(), state0.cuda()
    out = torch.empty((6, B, D), dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mud, off = mu.cuda(), R.dev_ints(range(B + 1))
    torch.cuda.synchronize()
    call = rq.prepare("rq_shift", xd, mud, state, out, off, stream=s)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    before = state0.clone()
    state.copy_(state0)
    gen = torch.Generator().manual_seed(9)
    for _ in range(4):
        xn = R.randn(gen, B, D, dtype=torch.float16)
        xd.copy_(xn)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        ref, after = R.shift_ref(xn.numpy(), mu.numpy(), before.numpy(), [1] * B, range(B))
        check(out, ref, xn, [1] * B, before, range(B))
        assert np.array_equal(state.cpu().numpy(), after)
        before = torch.from_numpy(after)


def test_rows_of_a_sequence_that_leaves_the_range():
    """They are mixed with the row before them, the first with zeros."""
    T, D = 20, 64
    x, mu, state0 = tensors(T, D, 3, 3, 5)
    out = torch.empty((3, T, D), dtype=torch.float16, device="cuda")
    state = state0.cuda()
    rq.rq_shift(x.cuda(), mu.cuda(), state, out, R.dev_ints([-5, 3, 8, T + 100]))
    ref, _ = R.shift_ref(x.numpy(), mu.numpy(), state0.numpy(), [3, 5, 12], [-1, 1, -1])
    before = x[7].double().numpy()  # of the third sequence's first row
    ref[:, 8] = x[8].double().numpy() + (before - x[8].double().numpy()) * mu.double().numpy()
    ref[:, 0] = x[0].double().numpy() * (1 - mu.double().numpy())
    check(out, ref, x, [T], state0, [0])
    assert torch.equal(state.cpu()[[0, 2]], state0[[0, 2]])
