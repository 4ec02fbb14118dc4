"""rq_wkv7 where the values of one call differ in size: a token's r, k, v,
kappa or eta, a value channel or a state far smaller than its neighbours,
sizes that grow and fall along a sequence, and values near the ends of
binary16 and far outside it.

Tolerance: as in test_gpu_wkv7, per token and value row.  |error of y[t][i]| <=
72 (T + 1) 2^-24 |S_i| |r_t|, with |S_i| the largest 2-norm the state row had
up to this token, so a small row or token is held to its own size; a state
entry likewise to 72 T 2^-24 |S_i|."""
import numpy as np
import pytest
import torch

import gemm_rwkv_decode_amd as rq
from tests import aroundtest as R
from tests.rqtest import say
from tests.test_gpu_wkv7 import as64, check, inputs, on_gpu

pytestmark = pytest.mark.gpu
HEADS = [1, 100, 256]  # one, two and four state waves
SMALL = [(False, 1e-6), (False, 1e-8), (False, 1e-12), (True, 1e-4), (True, 1e-6)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def start_state(H, seed, scale=1.0):
    return R.randn(torch.Generator().manual_seed(seed), 1, H, 64, 64, scale=scale)


def compare(ins, state0, what):
    T, H = ins["r"].shape[:2]
    y_ref, s_ref, norms = R.wkv7_ref(as64(ins), state0.numpy(), [T], [0])
    y = torch.full((T, H * 64), float("nan"), device="cuda")
    s = state0.cuda()
    rq.rq_wkv7(*on_gpu(ins), s, y, R.dev_ints([0, T]))
    torch.cuda.synchronize()
    check(y, y_ref, norms, as64(ins)["r"], T, what)
    err = np.abs(s.cpu().double().numpy() - s_ref)[0].max(-1)
    bound = 72 * T * R.EPS * norms[-1]
    assert np.all(err <= bound), f"{what}: state {(err / bound).max():.3g}"


@pytest.mark.parametrize("half,scale", SMALL)
@pytest.mark.parametrize("which", ["r", "k", "v", "kappa", "eta"])
@pytest.mark.parametrize("H", HEADS)
def test_small_tokens_beside_ordinary_ones(H, which, half, scale):
    """The first token of a sequence and one inside a chunk."""
    T = 53
    for empty in (True, False):
        say(f"[wkv7 range] {which} x {scale} H {H} half {half} empty {empty}")
        ins = inputs(T, H, 20)
        for at in (0, 21):
            ins[which][at] *= scale
        ins = {n: t.to(torch.float16 if half else torch.float32) for n, t in ins.items()}
        compare(ins, start_state(H, 21) * (0 if empty else 1), f"{which} {scale} {empty}")


@pytest.mark.parametrize("half,scale", SMALL)
@pytest.mark.parametrize("H", HEADS)
def test_small_value_channels_beside_ordinary_ones(H, half, scale):
    T = 53
    for empty in (True, False):
        ins = inputs(T, H, 22)
        state0 = start_state(H, 23) * (0 if empty else 1)
        for i in (5, 40):
            ins["v"][:, :, i] *= scale
            state0[:, :, i] *= scale
        ins = {n: t.to(torch.float16 if half else torch.float32) for n, t in ins.items()}
        compare(ins, state0, f"channel {scale} {empty}")


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("scale", [1e-3, 1e-6, 1e-18])
def test_small_everywhere_with_strong_decays(H, scale):
    T = 50
    ins = inputs(T, H, 24)
    ins["w"] = torch.full_like(ins["w"], 8.0)
    ins["r"], ins["k"] = ins["r"] * scale, ins["k"] * scale
    compare(ins, start_state(H, 25) * 0, f"r, k {scale}")
    compare(ins, start_state(H, 25, scale), f"r, k, state {scale}")


@pytest.mark.parametrize("H", HEADS)
def test_a_small_state_before_ordinary_values(H):
    ins = inputs(40, H, 26)
    ins["v"][:5] = 0
    compare(ins, start_state(H, 27, 1e-10), "small state")


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("factor", [4.0, 0.25])
def test_sizes_that_grow_and_fall_along_a_sequence(H, which, factor):
    T = 70
    ins = inputs(T, H, 28)
    ins[which] *= (factor ** (torch.arange(T) - T / 2.0))[:, None, None]
    compare(ins, start_state(H, 29) * 0, f"{which} x {factor} a token")
    compare(ins, start_state(H, 29), f"{which} x {factor} a token, stored")


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("half,sizes", [(False, dict(k=1e6)), (False, dict(r=1e10)),
                                        (False, dict(r=3e15, k=1e15)), (False, dict(v=1e25, r=1e-9)),
                                        (True, dict(k=1e4)), (True, dict(r=1.2e4)),
                                        (True, dict(r=300.0, k=1e3, v=1e4))])
def test_large_values(H, half, sizes):
    T = 50
    ins = inputs(T, H, 30)
    for n, s in sizes.items():
        ins[n] = ins[n] * s
    if half:
        ins = {n: t.clamp(-6e4, 6e4).half() for n, t in ins.items()}
    compare(ins, start_state(H, 31), f"{sizes}")


@pytest.mark.parametrize("H", HEADS)
@pytest.mark.parametrize("size", [1e-1, 1e-2, 1e-4])
def test_small_removal_keys_with_large_rates(H, size):
    """eta |kappa|^2 = 1/2: the same removal as of a key of 1."""
    ins = inputs(50, H, 32)
    ins["kappa"] = ins["kappa"] * size
    ins["eta"] = torch.full_like(ins["eta"], 0.5 / size ** 2)
    compare(ins, start_state(H, 33), f"kappa {size}")


@pytest.mark.parametrize("half,scale", SMALL)
@pytest.mark.parametrize("which", ["r", "k", "v", "channel"])
def test_small_values_in_a_long_sequence(which, half, scale):
    """Long enough for the kernel of long prompts."""
    ins = inputs(600, 2, 34)
    if which == "channel":
        ins["v"][:, :, [5, 40]] *= scale
    else:
        ins[which][[0, 150, 599]] *= scale
    ins = {n: t.to(torch.float16 if half else torch.float32) for n, t in ins.items()}
    compare(ins, start_state(2, 35) * 0, f"long {which} {scale}")
