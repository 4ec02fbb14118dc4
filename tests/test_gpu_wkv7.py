"""rq_wkv7 against the recurrence in 64 bits: every kernel (token by token,
sixteen tokens at a time with one, two or four state waves), lengths around
the chunk, empty sequences, stored and unstored states, both input types,
values that are not finite, and use on other streams and in graphs.

Tolerance.  With |kappa| <= 1 and eta <= 1 a token's map of the state does not
grow it, so roundings add up: per token at most 64 + 8 units of 2^-24 of the
state row's norm (a 64-term sum and the update), T tokens, and the output's
own 64-term sum with r: |error| <= 72 (T + 1) 2^-24 |S_i| |r|.  Roundings of
random sign grow like a sqrt and are damped by the decay, so over a whole
output the relative error is held to 2^-20 as well (16 units)."""
import numpy as np
import pytest
import torch

import gemm_rwkv_decode_amd as rq
from tests import aroundtest as R
from tests.rqtest import say

pytestmark = pytest.mark.gpu
NAMES = ("r", "w", "k", "v", "kappa", "eta")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def inputs(T, H, seed, dtype=torch.float32, vscale=1.0):
    g = torch.Generator().manual_seed(seed)
    kap = torch.nn.functional.normalize(R.randn(g, T, H, 64), dim=-1)
    ins = {"r": R.randn(g, T, H, 64), "w": R.randn(g, T, H, 64, scale=3.0) - 2.0,
           "k": R.randn(g, T, H, 64), "v": R.randn(g, T, H, 64, scale=vscale), "kappa": kap * 0.999,
           "eta": torch.sigmoid(R.randn(g, T, H, 64))}
    return {n: t.to(dtype) for n, t in ins.items()}


def on_gpu(ins):
    return [ins[n].reshape(ins[n].shape[0], -1).cuda() for n in NAMES]


def as64(ins):
    return {n: t.double().numpy() for n, t in ins.items()}


def check(y, y_ref, norms, r, T, what=""):
    y = y.detach().cpu().double().numpy().reshape(y_ref.shape)
    live = ~np.isnan(y_ref)
    err = np.abs(y - y_ref)
    bound = 72 * (T + 1) * R.EPS * norms * np.sqrt((r ** 2).sum(-1, keepdims=True))
    assert np.all(err[live] <= bound[live]), f"{what}: {np.nanmax(err[live] / bound[live]):.3g}"
    rel = np.linalg.norm((y - y_ref)[live]) / np.linalg.norm(y_ref[live])
    assert rel <= 2.0 ** -20, f"{what}: relative error {rel:.3g}"


CASES = [
    ([1], 1), ([2], 3), ([3, 0, 1, 2], 2), ([0, 0, 1], 5), ([31, 0, 1], 2),   # token by token
    ([33], 1), ([16, 32], 2), ([47, 0, 1], 3), ([64], 4), ([15, 17, 16], 12),  # one state wave
    ([700], 1), ([97], 80),
    ([47, 0, 1, 17, 100], 40), ([49, 2], 60),                                 # two
    ([100, 33, 1, 0, 64, 15, 2, 16], 32), ([40], 257),                        # four
    ([1] * 63 + [70], 5),
]


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("lens,H", CASES)
def test_against_the_recurrence(lens, H, half):
    T, B = sum(lens), len(lens)
    say(f"[wkv7] lens {lens[:8]} H {H} half {half}")
    ins = inputs(T, H, T + H, torch.float16 if half else torch.float32)
    g = torch.Generator().manual_seed(B)
    nslots = B + 2
    state0 = R.randn(g, nslots, H, 64, 64)
    slots = torch.randperm(nslots, generator=g)[:B].tolist()
    y_ref, s_ref, norms = R.wkv7_ref(as64(ins), state0.numpy(), lens, slots)
    state, s_ok = R.guarded((nslots, H, 64, 64), torch.float32, 7.0)
    state.copy_(state0)
    y, y_ok = R.guarded((T, H * 64), torch.float32, float("nan"))
    rq.rq_wkv7(*on_gpu(ins), state, y, R.dev_ints(R.offsets_of(lens)), R.dev_ints(slots))
    assert y_ok() and s_ok()
    check(y, y_ref, norms, as64(ins)["r"], max(lens), f"{lens[:8]} H={H}")
    got = state.cpu().double().numpy()
    untouched = [s for s in range(nslots) if s not in [q for q, n in zip(slots, lens) if n]]
    assert np.array_equal(got[untouched], state0.double().numpy()[untouched])
    err = np.abs(got - s_ref)
    top = max(norms.max(), np.sqrt((s_ref ** 2).sum(-1)).max())
    assert err.max() <= 72 * max(lens) * R.EPS * top
    assert np.linalg.norm(err) <= 2.0 ** -20 * np.linalg.norm(s_ref)


@pytest.mark.parametrize("lens,H", [([2, 1], 2), ([20, 37], 2), ([60, 40], 100), ([50, 40], 130)])
def test_slots_that_are_not_stored_start_from_zero(lens, H):
    T = sum(lens)
    ins = inputs(T, H, 3)
    state0 = torch.ones(1, H, 64, 64)
    for slots, st in (([-1, 1], state0), ([5, -7], None)):
        y_ref, _, norms = R.wkv7_ref(as64(ins), np.zeros((1, H, 64, 64)), lens, [-1, -1])
        y = torch.full((T, H * 64), float("nan"), device="cuda")
        s = None if st is None else st.cuda()
        rq.rq_wkv7(*on_gpu(ins), s, y, R.dev_ints(R.offsets_of(lens)), R.dev_ints(slots))
        torch.cuda.synchronize()
        check(y, y_ref, norms, as64(ins)["r"], max(lens))
        if s is not None:
            assert torch.equal(s.cpu(), state0)


@pytest.mark.parametrize("lens,H", [([2, 3], 2), ([30, 21], 2), ([30, 21], 128)])
def test_rows_of_no_sequence_are_not_written(lens, H):
    """offsets that start after 0 and end before T leave the other rows of y;
    offsets outside 0..T are cut to it."""
    T = sum(lens) + 9
    ins = inputs(T, H, 4)
    off = R.offsets_of(lens, 4)
    y = torch.full((T, H * 64), -3.0, device="cuda")
    state = torch.zeros(2, H, 64, 64, device="cuda")
    rq.rq_wkv7(*on_gpu(ins), state, y, R.dev_ints(off))
    y_ref, _, norms = R.wkv7_ref(as64(ins), np.zeros((2, H, 64, 64)), lens, [0, 1], start=4)
    check(y, y_ref, norms, as64(ins)["r"], max(lens))
    assert bool((y[:4] == -3).all()) and bool((y[off[-1]:] == -3).all())
    y2, ok = R.guarded((T, H * 64), torch.float32, -3.0)
    rq.rq_wkv7(*on_gpu(ins), torch.zeros_like(state), y2, R.dev_ints([-50, 4, T + 1000]))
    assert ok()
    assert bool(torch.isfinite(y2).all())


@pytest.mark.parametrize("H", [1, 100, 256])
def test_two_calls_continue_one(H):
    """A prompt in two calls, the second from the stored state, equals one."""
    T, cut = 75, 41
    ins = inputs(T, H, 5)
    d = on_gpu(ins)
    y1 = torch.empty(T, H * 64, device="cuda")
    s1 = torch.zeros(1, H, 64, 64, device="cuda")
    rq.rq_wkv7(*d, s1, y1, R.dev_ints([0, T]))
    y2, s2 = torch.empty_like(y1), torch.zeros_like(s1)
    rq.rq_wkv7(*[t[:cut] for t in d], s2, y2[:cut], R.dev_ints([0, cut]))
    rq.rq_wkv7(*[t[cut:].contiguous() for t in d], s2, y2[cut:], R.dev_ints([0, T - cut]))
    torch.cuda.synchronize()
    assert float((y1 - y2).norm() / y1.norm()) <= 2.0 ** -20
    assert float((s1 - s2).norm() / s1.norm()) <= 2.0 ** -20


@pytest.mark.parametrize("H,T", [(1, 60), (100, 60), (256, 40), (2, 20)])
@pytest.mark.parametrize("which", ["v", "k", "r", "kappa", "w"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_values_that_are_not_finite_reach_no_earlier_token(H, T, which, bad):
    at = T - 7  # not the first of its chunk of sixteen
    ins = inputs(T, H, 6)
    good = {n: t.clone() for n, t in ins.items()}
    ins[which][at, 0, 11] = bad
    outs = []
    for i in (good, ins):
        y = torch.empty(T, H * 64, device="cuda")
        s = torch.zeros(1, H, 64, 64, device="cuda")
        rq.rq_wkv7(*on_gpu(i), s, y, R.dev_ints([0, T]))
        torch.cuda.synchronize()
        outs.append((y.view(T, H, 64).cpu(), s.cpu()))
    (yg, _), (yb, sb) = outs
    assert torch.isfinite(yb[:at]).all()
    assert float((yb[:at] - yg[:at]).norm() / yg[:at].norm()) <= 2.0 ** -20
    # other heads, and for v the other value rows, never see it
    assert torch.isfinite(yb[:, 1:]).all()
    if which == "v":
        rows = [j for j in range(64) if j != 11]
        assert torch.isfinite(yb[:, 0, rows]).all() and torch.isfinite(sb[0, 0, rows]).all()
        assert not torch.isfinite(yb[at:, 0, 11]).any()
    elif not (which == "w" and bad == float("inf")):  # sigmoid(inf) = 1 is a decay
        assert not torch.isfinite(yb[at, 0]).all()


@pytest.mark.parametrize("H", [1, 100, 256])
@pytest.mark.parametrize("scale", [1e-18, 1e18])
def test_the_size_of_the_values_does_not_matter(H, scale):
    T = 50
    ins = inputs(T, H, 7, vscale=scale)
    y_ref, s_ref, norms = R.wkv7_ref(as64(ins), np.zeros((1, H, 64, 64)), [T], [0])
    y = torch.empty(T, H * 64, device="cuda")
    s = torch.zeros(1, H, 64, 64, device="cuda")
    rq.rq_wkv7(*on_gpu(ins), s, y, R.dev_ints([0, T]))
    check(y, y_ref, norms, as64(ins)["r"], T)


@pytest.mark.parametrize("H", [1, 100, 256])
def test_extreme_decays_and_repeated_keys(H):
    """w at +-60 (decays of exp(-0.61) and 1), the same key at every token
    with a learning rate of 1: the chunk's triangular system at its worst."""
    T = 64
    ins = inputs(T, H, 8)
    ins["w"] = torch.where(torch.rand(T, H, 64, generator=torch.Generator().manual_seed(1)) < 0.5,
                           60.0, -60.0)
    ins["kappa"] = ins["kappa"][:1].expand(T, H, 64).contiguous()
    ins["eta"] = torch.ones(T, H, 64)
    y_ref, s_ref, norms = R.wkv7_ref(as64(ins), np.zeros((1, H, 64, 64)), [T], [0])
    y = torch.empty(T, H * 64, device="cuda")
    s = torch.zeros(1, H, 64, 64, device="cuda")
    rq.rq_wkv7(*on_gpu(ins), s, y, R.dev_ints([0, T]))
    check(y, y_ref, norms, as64(ins)["r"], T)


def test_a_state_pool_past_two_gib():
    H, slot = 64, 2100  # 2100 MiB into the pool
    state = torch.zeros(slot + 1, H, 64, 64, device="cuda")
    for lens in ([1], [40]):
        T = sum(lens)
        ins = inputs(T, H, 9)
        state[slot] = 0.5
        y_ref, s_ref, norms = R.wkv7_ref(as64(ins), np.full((1, H, 64, 64), 0.5), lens, [0])
        y = torch.empty(T, H * 64, device="cuda")
        rq.rq_wkv7(*on_gpu(ins), state, y, R.dev_ints([0, T]), R.dev_ints([slot]))
        check(y, y_ref, norms, as64(ins)["r"], T)
        got = state[slot].cpu().double().numpy()
        assert np.linalg.norm(got - s_ref[0]) <= 2.0 ** -20 * np.linalg.norm(s_ref)
    assert not bool(state[:slot].any())


@pytest.mark.parametrize("lens,H", [([1, 1], 4), ([50], 4), ([50, 40], 64)])
def test_graph_replays_and_other_streams(lens, H):
    """Replays read the index tensors and inputs as they are then."""
    T, B = sum(lens), len(lens)
    ins = inputs(T, H, 10)
    d = on_gpu(ins)
    state, y = torch.zeros(B, H, 64, 64, device="cuda"), torch.empty(T, H * 64, device="cuda")
    off = R.dev_ints(R.offsets_of(lens))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call = rq.prepare("rq_wkv7", *d, state, y, off, stream=s)
    want_y, want_s = [], []
    for _ in range(4):
        call()
        torch.cuda.synchronize()
        want_y.append(y.clone())
        want_s.append(state.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    state.zero_()
    junk = torch.randn(1 << 18, device="cuda")
    for i in range(4):
        y.fill_(float("nan"))
        junk.mul_(1.0001)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want_y[i]) and torch.equal(state, want_s[i])


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("lens,H", [
    ([1] * 31 + [48], 3), ([7, 8, 9, 1, 0, 15, 16, 17], 2), ([7, 8, 9, 1, 0, 15, 16, 17], 20),
    ([2] * 40 + [100], 2), ([8], 5), ([7], 5), ([13, 13, 13], 3), ([12, 12], 80), ([0, 0, 31, 0], 2)])
def test_short_and_long_sequences_in_one_call(lens, H, half):
    """Around the lengths from which sequences go in chunks, in batches of both
    kinds and of one."""
    test_against_the_recurrence(lens, H, half)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("lens,H", [([0] * 63 + [48], 2), ([0] * 40 + [39] + [0] * 23, 64),
                                    ([0, 9] * 30 + [0] * 300, 3), ([0] * 20 + [7], 5)])
def test_mostly_empty_sequences(lens, H, half):
    """Fewer tokens than sequences."""
    test_against_the_recurrence(lens, H, half)
