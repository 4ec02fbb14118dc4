"""The serving example: a batch of ragged prompts, then single tokens, through
every call together, against a plain form in 64 bits.

The plain form runs one sequence after another, token by token, on unpacked
weights.  Both sides round activations to binary16 in the same places, but the
bound does not count on the roundings agreeing: every one is a relative change
of at most 2^-11 of its tensor, 8 a layer and 2 at the head, 18 for two layers;
the squared ReLU doubles a change and the residual stream, the norms and the
normalised removal key pass it on, together taken as a factor of 4.  So logits
may differ by 4 * 18 * 2^-11 = 0.035 of their 2-norm.  The planted mistakes
below are several times that.
"""
import numpy as np
import pytest
import torch

from gemm_rwkv_decode_amd import serve as V
from gemm_rwkv_decode_amd import synth as S
from tests import aroundtest as A

BOUND = 4 * 18 * 2.0 ** -11
PROMPTS = [70, 1, 19, 2, 33]  # ragged; one crosses a product call's 64 rows
STEPS = 4
RANKS, SCALES, IDS = [8, 24, 16], [1.0, 0.7, 1.3], [1, 0, -1, 2, 1]


def build(device, fmt):
    model = V.Model(2, 256, 517, fmt, low=32, seed=5, device=device)
    adapters = V.Adapters(model, RANKS, SCALES, seed=6)
    g = torch.Generator().manual_seed(7)
    prompts = [torch.randint(0, model.vocab, (n,), generator=g).tolist() for n in PROMPTS]
    return model, adapters, prompts


def f64(t):
    return t.detach().cpu().numpy().astype(np.float64)


def f16(a):
    return a.astype(np.float16).astype(np.float64)


def unpack(p):
    """The matrix of a symmetric Packed."""
    q = p.qweight.cpu().numpy()
    if p.fmt.bits == 8:
        codes = q.astype(np.float64)
    else:
        codes = np.empty((p.N, p.K))
        codes[:, 0::2], codes[:, 1::2] = q & 0xF, q >> 4
        codes[codes > 7] -= 16
    return codes * np.repeat(f64(p.scales), p.fmt.group, axis=1)


def norm(x, ln, eps=1e-5):
    mean = x.mean(-1, keepdims=True)
    var = ((x - mean) ** 2).mean(-1, keepdims=True)
    return (x - mean) / np.sqrt(var + eps) * f64(ln[0]) + f64(ln[1])


def sigmoid(x):
    return 1 / (1 + np.exp(-x))


class Plain:
    """One sequence of the example, a token at a time, in 64 bits."""

    def __init__(self, model, adapters, ident, plant=None):
        self.m, self.ad, self.ident, self.plant = model, adapters, ident, plant
        self.W = [[unpack(p) for p in w.mats] for w in model.layers]
        self.head = unpack(model.head)
        L, D = len(model.layers), model.width
        self.att, self.ffn = np.zeros((L, D)), np.zeros((L, D))
        self.wkv = np.zeros((L, model.heads, 64, 64))

    def adapter(self, pair, N, x):
        if not 0 <= self.ident < len(RANKS) or self.plant == "adapter":
            return 0.0
        off = self.ad.offsets.tolist()
        lo, hi = off[self.ident], off[self.ident + 1]
        a = f64(pair[0])[lo:hi]
        b = f64(pair[1])[lo * N:hi * N].reshape(N, hi - lo)
        return float(self.ad.scales[self.ident]) * (b @ (a @ x))

    def low(self, w, name, x, act=None):
        t = f16(x @ f64(w.down[name]))
        return f16((f16(act(t)) if act else t) @ f64(w.up[name]))

    def token(self, token):
        m, D, H = self.m, self.m.width, self.m.heads
        x = f64(m.embed[token])
        first = None
        for l, w in enumerate(m.layers):
            xn = f16(norm(x, w.ln1))
            prev = xn if self.plant == "shift" else self.att[l]
            xr, xk, xv, xw, xa, xg = f16(xn + (prev - xn) * f64(w.mu))
            self.att[l] = xn
            r, k, v = [W @ z + self.adapter(p, D, z)
                       for W, p, z in zip(self.W[l], self.ad.rkv[l], (xr, xk, xv))]
            decay = np.exp(-np.exp(-0.5) * sigmoid(f64(w.base["w"]) + self.low(w, "w", xw, np.tanh)))
            eta = sigmoid(f64(w.base["a"]) + self.low(w, "a", xa))
            gate = self.low(w, "g", xg, sigmoid)
            if first is None:
                first = v
            else:
                v = v + (first - v) * sigmoid(f64(w.base["v"]) + self.low(w, "v", xv))
            kap = (k * f64(w.k_k)).reshape(H, 64)
            kap = kap / np.sqrt((kap ** 2).sum(-1, keepdims=True))
            k = k * (1 + (eta - 1) * f64(w.k_a))
            rh, kh, vh, dh, eh = (z.reshape(H, 64) for z in (r, k, v, decay, eta))
            St = self.wkv[l]
            gone = (St * kap[:, None, :]).sum(-1)
            if self.plant == "removal":
                gone = gone * 0
            St = (St * dh[:, None, :] - gone[:, :, None] * (eh * kap)[:, None, :]
                  + vh[:, :, None] * kh[:, None, :])
            self.wkv[l] = St
            y = (St * rh[:, None, :]).sum(-1)
            mean = y.mean(-1, keepdims=True)
            y = (y - mean) / np.sqrt(((y - mean) ** 2).mean(-1, keepdims=True) + 64e-5)
            y = y.reshape(D) * f64(w.lnx[0]) + f64(w.lnx[1])
            own = (r * k * f64(w.r_k)).reshape(H, 64).sum(-1, keepdims=True)
            y = (y + (own * vh).reshape(D)) * gate
            x = x + self.W[l][3] @ f16(y)
            xn = f16(norm(x, w.ln2))
            mixed = f16(xn + (self.ffn[l] - xn) * f64(w.mu_ffn)[0])
            self.ffn[l] = xn
            key = self.W[l][4] @ mixed + self.adapter(self.ad.key[l], m.ffn, mixed)
            x = x + self.W[l][5] @ f16(np.maximum(key, 0) ** 2)
            if self.plant == "state":
                self.wkv[l] = 0
        return self.head @ f16(norm(x, m.ln_out))


def plain_logits(model, adapters, prompts, tokens, plant=None):
    """[step][request]: the logits before each of `tokens` [requests][steps]."""
    out = []
    for ident, p, mine in zip(IDS, prompts, tokens):
        seq = Plain(model, adapters, ident, plant)
        for t in p:
            z = seq.token(t)
        rows = [z]
        for t in mine[:-1]:
            rows.append(seq.token(int(t)))
        out.append(rows)
    return [np.stack([rows[i] for rows in out]) for i in range(len(tokens[0]))]


def difference(got, want):
    return np.linalg.norm(got - want, axis=-1) / np.linalg.norm(want, axis=-1)


@pytest.mark.parametrize("plant", ["adapter", "shift", "removal", "state"])
def test_planted_mistakes_show(plant):
    """The bound separates: a plain form without one of the calls is outside it."""
    model, adapters, prompts = build("cpu", S.INT4_G64)
    tokens = [[1, 2], [3, 4], [5, 6], [7, 8], [9, 10]]
    right = plain_logits(model, adapters, prompts, tokens)
    wrong = plain_logits(model, adapters, prompts, tokens, plant)
    worst = max(difference(w, r).max() for w, r in zip(wrong, right))
    assert worst > 3 * BOUND


def test_models_of_other_layouts_are_refused():
    with pytest.raises(ValueError):
        V.Model(1, 96, 64, device="cpu")
    with pytest.raises(ValueError):
        V.Model(1, 256, 64, S.ASYM4_G32, device="cpu")


def test_empty_prompts_are_refused():
    model = V.Model(1, 64, 64, device="cpu")
    for prompts in ([], [[1, 2], []]):
        with pytest.raises(ValueError):
            V.generate(model, prompts, 2)


def test_histories_on_the_host():
    h = V.Histories([[5, 6, 7], [8]], 5, "cpu")
    h.append(torch.tensor([1, 2], dtype=torch.int32))
    h.append(torch.tensor([3, 4], dtype=torch.int32))
    assert h.tokens.tolist() == [[5, 6, 7, 1, 3], [8, 2, 4, -1, -1]]
    assert h.offsets.tolist() == [0, 5, 10] and h.prompt.tolist() == [3, 1]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [S.INT4_G64, S.INT8_G16], ids=lambda f: f.tag)
def test_prompts_and_steps_against_the_plain_form(fmt):
    model, adapters, prompts = build("cuda", fmt)
    V_ = model.vocab
    bits = np.random.default_rng(3).random((2, V_)) < 0.7
    which = [0, -1, 1, 0, -1]
    bias = ([4, 4, 11], [1.0, 2.5, -3.0], [0, 2, 2, 2, 3, 3])
    pens = dict(repetition=1.2, presence=0.3, frequency=0.2)
    seen = []
    tokens = V.generate(
        model, prompts, STEPS, adapters, IDS, **pens,
        bias=(A.dev_ints(bias[0]), torch.tensor(bias[1], device="cuda"), A.dev_ints(bias[2])),
        masks=(A.pack_masks(bits).cuda(), A.dev_ints(which)),
        on_step=lambda i, z: seen.append(z.cpu().numpy()))
    tokens = tokens.cpu().numpy()
    assert len(seen) == STEPS
    want = plain_logits(model, adapters, prompts, tokens)
    for i in range(STEPS):
        d = difference(seen[i].astype(np.float64), want[i])
        assert (d < BOUND).all(), (i, d)
        # the choice, on the very logits it was made from
        n = len(prompts)
        history = [(p + list(tokens[m, :i]), len(p)) for m, p in enumerate(prompts)]
        rows = [(bias[0][a:b], bias[1][a:b]) for a, b in zip(bias[2], bias[2][1:])]
        _, chosen = A.logits_ref(seen[i], history, *[[pens[k]] * n for k in
                                                    ("repetition", "presence", "frequency")],
                                 bias=rows, masks=(bits, which))
        assert (chosen == tokens[:, i]).all(), i


@pytest.mark.gpu
def test_prompts_at_once_as_token_by_token():
    """One call over a prompt and one call per token leave the same state and
    logits (to the roundings' bound)."""
    model, adapters, prompts = build("cuda", S.INT4_G64)
    p = prompts[0]
    ids = torch.full((len(p),), 1, dtype=torch.int32, device="cuda")
    slot = A.dev_ints([0])
    whole, single = V.State(model, 1), V.State(model, 1)
    a = V.forward(model, whole, A.dev_ints(p), A.dev_ints([0, len(p)]), slot, ids, adapters)
    for t in p:
        b = V.forward(model, single, A.dev_ints([t]), A.dev_ints([0, 1]), slot, ids[:1], adapters)
    assert difference(f64(b), f64(a)).max() < BOUND
    for x, y in ((whole.att, single.att), (whole.ffn, single.ffn), (whole.wkv, single.wkv)):
        x, y = f64(x).reshape(len(model.layers), -1), f64(y).reshape(len(model.layers), -1)
        assert difference(y, x).max() < BOUND


@pytest.mark.gpu
def test_steps_replayed_from_a_graph():
    """Replays, with the host's own work between them, give the eager logits
    and tokens to the bit."""
    model, adapters, prompts = build("cuda", S.INT4_G64)
    runs = []
    for graph in (False, True):
        seen = []
        tokens = V.generate(model, prompts, 7, adapters, IDS, graph=graph,
                            on_step=lambda i, z: seen.append(z.clone().cpu()))
        torch.cuda.synchronize()
        runs.append((tokens.cpu(), seen))
    assert torch.equal(runs[0][0], runs[1][0])
    assert all(torch.equal(a, b) for a, b in zip(runs[0][1], runs[1][1]))


@pytest.mark.gpu
@pytest.mark.parametrize("eager", [False, True])
def test_the_command(capsys, eager):
    V.main(["--layers", "1", "--width", "256", "--vocab", "512", "--requests", "6", "--prompt",
            "80", "--steps", "5", "--adapters", "2", "--rank", "8"] + ["--eager"] * eager)
    lines = capsys.readouterr().out.splitlines()
    assert lines[0].startswith("6 requests") and "tokens/s" in lines[1]
    assert sum(line.startswith("request ") for line in lines) == 3


@pytest.mark.parametrize("prompts,steps,ids", [
    ([[1, 64]], 2, None), ([[1], [-1, 3]], 2, None), ([[1]], 0, None), ([[1]], -1, None),
    ([[1], [2]], 2, [0]), ([[1]], 2, [0, 0])])
def test_what_generate_refuses(prompts, steps, ids):
    """On the host: a token outside the vocabulary would index past the embedding
    on the GPU."""
    model = V.Model(1, 64, 64, device="cpu")
    with pytest.raises(ValueError):
        V.generate(model, prompts, steps, ids=ids)
