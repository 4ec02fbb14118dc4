"""rq_wkv7's chunks done token by token: values that are not finite and values
outside an operand's range, in every kernel and both input types.  The
tolerance is test_gpu_wkv7's."""
import numpy as np
import pytest
import torch

import gemm_rwkv_decode_amd as rq
from tests import aroundtest as R
from tests.test_gpu_wkv7 import as64, check, inputs, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def run(ins, T, H):
    y = torch.empty(T, H * 64, device="cuda")
    s = torch.zeros(1, H, 64, 64, device="cuda")
    rq.rq_wkv7(*on_gpu(ins), s, y, R.dev_ints([0, T]))
    torch.cuda.synchronize()
    return y.view(T, H, 64).cpu(), s.cpu()


# one, two and four state waves, and a long prompt's kernel for binary32
@pytest.mark.parametrize("H,T", [(1, 60), (2, 600), (100, 40), (256, 40)])
@pytest.mark.parametrize("which", ["r", "w", "k", "v", "kappa", "eta"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("half", [False, True])
def test_values_that_are_not_finite(H, T, which, bad, half):
    at = T - 23  # inside a chunk, with whole chunks before and after
    ins = inputs(T, H, 40, torch.float16 if half else torch.float32)
    yg, _ = run(ins, T, H)
    ins[which] = ins[which].clone()
    ins[which][at, 0, 11] = bad
    yb, sb = run(ins, T, H)
    assert torch.isfinite(yb[:at]).all()
    assert float((yb[:at] - yg[:at]).norm() / yg[:at].norm()) <= 2.0 ** -20
    assert torch.isfinite(yb[:, 1:]).all() and torch.isfinite(sb[0, 1:]).all()
    if which == "v":
        rows = [j for j in range(64) if j != 11]
        assert torch.isfinite(yb[:, 0, rows]).all() and torch.isfinite(sb[0, 0, rows]).all()
        assert not torch.isfinite(yb[at:, 0, 11]).any()
    elif which == "r":  # reaches its own token only
        assert not torch.isfinite(yb[at, 0]).any()
        assert torch.isfinite(yb[at + 1:]).all() and torch.isfinite(sb).all()
    elif not (which == "w" and bad == float("inf")):  # sigmoid(inf) = 1 is a decay
        assert not torch.isfinite(yb[at:, 0]).all()


@pytest.mark.parametrize("H,T", [(1, 50), (2, 600), (100, 50), (256, 50)])
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("where", ["all", "one"])
def test_keys_and_receptances_past_an_operands_range(H, T, half, where):
    """Sizes of 1000 to 60000 with strong decays, at every token or at one."""
    ins = inputs(T, H, 41)
    ins["w"] = torch.full_like(ins["w"], 6.0)
    tokens = slice(None) if where == "all" else slice(T // 2, T // 2 + 1)
    ins["r"][tokens] *= 1.5e4
    ins["k"][tokens] *= 1e3
    ins = {n: (t.clamp(-6e4, 6e4).half() if half else t) for n, t in ins.items()}
    y_ref, s_ref, norms = R.wkv7_ref(as64(ins), np.zeros((1, H, 64, 64)), [T], [0])
    y, s = run(ins, T, H)
    check(y, y_ref, norms, as64(ins)["r"], T)
    err = np.abs(s.double().numpy() - s_ref)[0].max(-1)
    assert np.all(err <= 72 * T * R.EPS * norms[-1])


@pytest.mark.parametrize("H,T", [(1, 64), (2, 600), (100, 64), (256, 64)])
def test_extreme_decays_in_binary16(H, T):
    ins = inputs(T, H, 42)
    g = torch.Generator().manual_seed(1)
    ins["w"] = torch.where(torch.rand(T, H, 64, generator=g) < 0.5, 60.0, -60.0)
    ins["kappa"] = ins["kappa"][:1].expand(T, H, 64) * 0.998
    ins["eta"] = torch.ones(T, H, 64)
    ins = {n: t.half() for n, t in ins.items()}
    y_ref, _, norms = R.wkv7_ref(as64(ins), np.zeros((1, H, 64, 64)), [T], [0])
    y, _ = run(ins, T, H)
    check(y, y_ref, norms, as64(ins)["r"], T)
