"""Serving an RWKV-7-shaped model with the library: prompts of many requests in
one batch, then one token of each per step.

Every request has its own adapter (or none), its own state slot and its own
penalties.  A layer runs

    shift -> receptance, key, value (packed) + adapters -> state recurrence
          -> output (packed) -> shift -> FFN key (packed) + adapter -> FFN value (packed)

(package page "RWKV-7 FP8 Quantized Inference", section "Core Approach: Full
FP8, No Residuals", for the packed matrices and their order), and the head's
logits go through penalties and biases to the next token.  What stands between
those calls (norms, the small dense projections of decay, removal rate, value
mix and gate) is plain torch.  The same code runs prompts and single tokens:
only the offsets differ.

    python -m gemm_rwkv_decode_amd.serve --layers 4 --width 768 --requests 16

Weights are synthetic (seeded, random codes), so the text is not meaningful.
"""
import argparse
import time

import torch
import torch.nn.functional as F

import gemm_rwkv_decode_amd as rq
from gemm_rwkv_decode_amd import step as ST
from gemm_rwkv_decode_amd import synth as S

HEAD = rq.RQ_WKV_HEAD
MIXES = ("r", "k", "v", "w", "a", "g")  # the time mix's shifted inputs


def _packed(N, K, fmt, g, device):
    """Random codes whose rows have a 2-norm of about one (symmetric formats)."""
    top = 2 ** (fmt.bits - 1) - 1
    codes = torch.randint(-top, top + 1, (N, K), generator=g, device=device).to(torch.int8)
    scale = (3.0 / K) ** 0.5 / top
    scales = scale * (0.5 + torch.rand((N, K // fmt.group), generator=g, device=device))
    return S.encode(codes, fmt, scales=scales.half())


class Layer:
    """One layer's weights: packed matrices by ST's indices, the rest dense."""

    def __init__(self, D, FF, low, fmt, g, device):
        def normal(*shape, scale=1.0, dtype=torch.float32):
            return (torch.randn(shape, generator=g, device=device) * scale).to(dtype)

        def mix(n):
            return torch.rand((n, D), generator=g, device=device).half()
        shapes = ((D, D), (D, D), (D, D), (D, D), (FF, D), (D, FF))
        self.mats = [_packed(n, k, fmt, g, device) for n, k in shapes]
        self.mu, self.mu_ffn = mix(len(MIXES)), mix(1)
        self.base = {n: normal(D, scale=0.5) for n in "wav"}
        self.down = {n: normal(D, low, scale=D ** -0.5, dtype=torch.float16) for n in "wavg"}
        self.up = {n: normal(low, D, scale=low ** -0.5, dtype=torch.float16) for n in "wavg"}
        self.k_k, self.k_a, self.r_k = (1 + 0.2 * normal(D), 1 + 0.2 * normal(D), 0.1 * normal(D))
        self.ln1, self.ln2, self.lnx = ((1 + 0.1 * normal(D), 0.1 * normal(D)) for _ in range(3))


class Model:
    """``layers`` layers of ``width`` channels (whole heads of 64) and a packed
    head of ``vocab`` tokens; ``fmt`` is a symmetric format of synth."""

    def __init__(self, layers, width, vocab, fmt=S.INT4_G64, low=64, seed=0, device="cuda"):
        if width % HEAD or fmt.layout != S.LAYOUT_SYM:
            raise ValueError("whole heads of 64 channels and a symmetric format expected")
        g = S.generator(seed, device)
        self.width, self.heads, self.vocab, self.ffn = width, width // HEAD, vocab, 4 * width
        self.device = torch.device(device)
        self.embed = torch.randn((vocab, width), generator=g, device=device)
        self.layers = [Layer(width, self.ffn, low, fmt, g, device) for _ in range(layers)]
        self.ln_out = (torch.ones(width, device=device), torch.zeros(width, device=device))
        self.head = _packed(vocab, width, fmt, g, device)


class Adapters:
    """Low-rank adapters on receptance, key, value and FFN key of every layer,
    in rq_lora's layout.  ``ranks``: one per adapter, multiples of 8."""

    def __init__(self, model, ranks, scales=None, seed=1):
        dev, D, FF = model.device, model.width, model.ffn
        g = S.generator(seed, dev)
        self.total, self.max_rank = sum(ranks), max(ranks)
        off = [0]
        for r in ranks:
            off.append(off[-1] + r)
        self.offsets = torch.tensor(off, dtype=torch.int32, device=dev)
        self.scales = torch.tensor(scales or [1.0] * len(ranks), device=dev)

        def pair(N):
            a = torch.randn((self.total, D), generator=g, device=dev) * D ** -0.5
            b = torch.randn(self.total * N, generator=g, device=dev) * self.max_rank ** -0.5
            return a.half(), b.half()
        self.rkv = [[pair(D) for _ in range(3)] for _ in model.layers]
        self.key = [pair(FF) for _ in model.layers]

    def add(self, pairs, xs, ys, ids):
        """ys[i] += scale * B (A xs[i]) for every row's own adapter."""
        rows = xs[0].shape[0]
        for lo in range(0, rows, rq.RQ_LORA_MAX_M):
            s = slice(lo, min(lo + rq.RQ_LORA_MAX_M, rows))
            rq.rq_lora([(a, b, x[s], y[s], y[s], y.shape[1], x.shape[1])
                        for (a, b), x, y in zip(pairs, xs, ys)],
                       ids[s], self.offsets, self.scales, self.max_rank)


class State:
    """Slots of the sequences being served: what a sequence carries from one
    call to the next."""

    def __init__(self, model, slots):
        L, D, dev = len(model.layers), model.width, model.device
        self.att = torch.zeros((L, slots, D), dtype=torch.float16, device=dev)
        self.ffn = torch.zeros((L, slots, D), dtype=torch.float16, device=dev)
        self.wkv = torch.zeros((L, slots, model.heads, HEAD, HEAD), device=dev)


def products(mats, xs):
    """float32 outputs of packed matrices of one format, RQ_MAX_M rows a call."""
    f, rows = mats[0].fmt, xs[0].shape[0]
    ys = [torch.empty((rows, p.N), device=x.device) for p, x in zip(mats, xs)]
    for lo in range(0, rows, rq.RQ_MAX_M):
        s = slice(lo, min(lo + rq.RQ_MAX_M, rows))
        M = s.stop - s.start
        if len(mats) > 1:
            rq.rq_gemv_batched([(p.qweight, p.scales, p.zeros, x[s], y[s], p.N, p.K)
                                for p, x, y in zip(mats, xs, ys)], M, f.bits, f.group, f.layout)
        else:
            p, call = mats[0], getattr(rq, ST.product_entry(M))
            call(p.qweight, p.scales, p.zeros, xs[0][s], ys[0][s], M, p.N, p.K, f.bits, f.group,
                 f.layout)
    return ys


def _norm(x, ln):
    return F.layer_norm(x, x.shape[-1:], *ln)


def _low(layer, name, x, act=None):
    t = x @ layer.down[name]
    return ((act(t) if act else t) @ layer.up[name]).float()


def forward(model, state, tokens, offsets, slots, ids=None, adapters=None):
    """Logits float32 [sequences][vocab] after each sequence's last token.

    tokens int [T]: all sequences one after another; offsets int32 [sequences +
    1]; slots int32 [sequences]; ids int32 [T]: every token's adapter, outside
    0 .. adapters-1 for none.  No sequence is empty."""
    H, T = model.heads, tokens.shape[0]
    x = model.embed[tokens.long()]
    v_first = None
    for l, w in enumerate(model.layers):
        xn = _norm(x, w.ln1).half()
        mixed = torch.empty((len(MIXES),) + xn.shape, dtype=torch.float16, device=x.device)
        rq.rq_shift(xn, w.mu, state.att[l], mixed, offsets, slots)
        xr, xk, xv, xw, xa, xg = mixed.unbind(0)
        r, k, v = products(w.mats[:3], (xr, xk, xv))
        if adapters is not None:
            adapters.add(adapters.rkv[l], (xr, xk, xv), (r, k, v), ids)
        decay = w.base["w"] + _low(w, "w", xw, torch.tanh)
        eta = torch.sigmoid(w.base["a"] + _low(w, "a", xa))
        gate = _low(w, "g", xg, torch.sigmoid)
        if v_first is None:
            v_first = v
        else:
            v = v + (v_first - v) * torch.sigmoid(w.base["v"] + _low(w, "v", xv))
        kappa = F.normalize((k * w.k_k).view(T, H, HEAD), dim=-1).view(T, -1)
        k = k * (1 + (eta - 1) * w.k_a)
        y = torch.empty_like(r)
        rq.rq_wkv7(r, decay, k, v, kappa, eta, state.wkv[l], y, offsets, slots)
        y = F.group_norm(y, H, *w.lnx, eps=64e-5)
        own = (r * k * w.r_k).view(T, H, HEAD).sum(-1, keepdim=True)
        y = (y + (own * v.view(T, H, HEAD)).view(T, -1)) * gate
        x = x + products(w.mats[3:4], (y.half(),))[0]

        xn = _norm(x, w.ln2).half()
        mixed = torch.empty((1,) + xn.shape, dtype=torch.float16, device=x.device)
        rq.rq_shift(xn, w.mu_ffn, state.ffn[l], mixed, offsets, slots)
        key, = products(w.mats[4:5], (mixed[0],))
        if adapters is not None:
            adapters.add(adapters.key[l:l + 1], (mixed[0],), (key,), ids)
        x = x + products(w.mats[5:6], (torch.relu(key).square().half(),))[0]
    last = x[offsets[1:].long() - 1]
    return products([model.head], (_norm(last, model.ln_out).half(),))[0]


class Histories:
    """The tokens of every request so far, in rows of one capacity: entries not
    written yet are -1, which rq_logits passes over."""

    def __init__(self, prompts, capacity, device):
        rows = len(prompts)
        self.tokens = torch.full((rows, capacity), -1, dtype=torch.int32, device=device)
        for m, p in enumerate(prompts):
            self.tokens[m, :len(p)] = torch.as_tensor(p, dtype=torch.int32, device=device)
        self.offsets = torch.arange(0, (rows + 1) * capacity, capacity, dtype=torch.int32,
                                    device=device)
        self.prompt = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device=device)
        self.length = self.prompt.long()
        self.rows = torch.arange(rows, device=device)

    def append(self, tokens):
        self.tokens[self.rows, self.length] = tokens
        self.length += 1


def choose(logits, histories, repetition, presence, frequency, bias=None, masks=None):
    """Each request's next token; the logits are treated in place.  bias and
    masks as rq_logits takes them."""
    tokens = torch.empty(logits.shape[0], dtype=torch.int32, device=logits.device)
    rq.rq_logits(logits, logits, tokens,
                 history=(histories.tokens.view(-1), histories.offsets, histories.prompt),
                 repetition=repetition, presence=presence, frequency=frequency, bias=bias,
                 masks=masks)
    return tokens


def generate(model, prompts, steps, adapters=None, ids=None, repetition=1.1, presence=0.2,
             frequency=0.1, bias=None, masks=None, on_step=None, graph=False):
    """``steps`` greedy tokens after each prompt, int32 [requests][steps]; -1
    throughout for a request whose mask leaves no token.
    ids: one adapter per request.  on_step(i, logits) sees the head's logits
    before they are treated (i = 0: the prompts').  graph: the steps after the
    first single-token one are replays of a captured graph; the results are
    the same."""
    dev, n = model.device, len(prompts)
    if not n or not all(prompts):
        raise ValueError("a prompt has at least one token")
    if min(map(min, prompts)) < 0 or max(map(max, prompts)) >= model.vocab:
        raise ValueError(f"tokens of 0 .. {model.vocab - 1} expected")
    if steps < 1:
        raise ValueError("at least one step expected")
    if ids is not None and len(ids) != n:
        raise ValueError(f"an adapter for each of {n} requests expected, got {len(ids)}")

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def row(v):
        return torch.full((n,), v, device=dev)
    state, slots = State(model, n), ints(list(range(n)))
    hist = Histories(prompts, max(map(len, prompts)) + steps, dev)
    penalties = row(repetition), row(presence), row(frequency)
    row_ids = None if ids is None else ints(ids)
    offsets = [0]
    for p in prompts:
        offsets.append(offsets[-1] + len(p))
    given = ints([t for p in prompts for t in p])
    given_ids = None
    if row_ids is not None:
        given_ids = torch.repeat_interleave(row_ids, hist.prompt.long())
    singles = torch.arange(n + 1, dtype=torch.int32, device=dev)
    last = torch.empty(n, dtype=torch.int32, device=dev)  # each request's newest token
    seen = torch.empty((n, model.vocab), device=dev) if on_step else None
    out = torch.empty((n, steps), dtype=torch.int32, device=dev)

    def step(tokens, offsets, token_ids):
        logits = forward(model, state, tokens, offsets, slots, token_ids, adapters)
        if on_step:
            seen.copy_(logits)
        last.copy_(choose(logits, hist, *penalties, bias=bias, masks=masks))
        hist.append(last)

    def single():
        step(last, singles, row_ids)

    def done(i):
        out[:, i] = last
        if on_step:
            on_step(i, seen)
    step(given, ints(offsets), given_ids)
    done(0)
    if steps > 2 and graph:
        # the first single-token step runs eagerly on the stream that is captured
        # next: the binding makes that stream's workspace in it
        cur, side = torch.cuda.current_stream(dev), torch.cuda.Stream(dev)
        side.wait_stream(cur)
        with torch.cuda.stream(side):
            single()
        cur.wait_stream(side)
        done(1)
        replay = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replay, stream=side):
            single()
        for i in range(2, steps):
            replay.replay()
            done(i)
        torch.cuda.synchronize(dev)  # the graph and its memory end here
    else:
        for i in range(1, steps):
            single()
            done(i)
    return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--layers", type=int, default=12)
    ap.add_argument("--width", type=int, default=768)
    ap.add_argument("--vocab", type=int, default=65536)
    ap.add_argument("--format", choices=("int4g64", "int8g16"), default="int4g64")
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=128, help="longest prompt")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--adapters", type=int, default=4)
    ap.add_argument("--rank", type=int, default=16)
    ap.add_argument("--eager", action="store_true", help="no graph for the steps")
    a = ap.parse_args(argv)
    model = Model(a.layers, a.width, a.vocab, S.FORMATS[a.format])
    adapters = Adapters(model, [a.rank] * a.adapters) if a.adapters else None
    # one request in adapters + 1 has none
    ids = [m % (a.adapters + 1) - 1 for m in range(a.requests)] if a.adapters else None
    g = S.generator(2, "cpu")
    lens = torch.randint(1, a.prompt + 1, (a.requests,), generator=g).tolist()
    prompts = [torch.randint(0, a.vocab, (n,), generator=g).tolist() for n in lens]
    marks = []

    def mark(i, _):
        torch.cuda.synchronize()
        marks.append(time.perf_counter())
    generate(model, prompts, 3, adapters, ids, graph=not a.eager)  # library handles
    torch.cuda.synchronize()
    begin = time.perf_counter()
    tokens = generate(model, prompts, a.steps, adapters, ids, on_step=mark,
                      graph=not a.eager)
    print(f"{a.requests} requests, prompts of 1..{a.prompt} ({sum(lens)} tokens): "
          f"{1e3 * (marks[0] - begin):.2f} ms")
    if a.steps > 3:  # past the eager step and the capture
        ms = 1e3 * (marks[-1] - marks[2]) / (a.steps - 3)
        print(f"{a.steps - 3} steps of {a.requests} tokens: {ms:.2f} ms each, "
              f"{a.requests / ms * 1e3:.0f} tokens/s")
    for m in range(min(a.requests, 3)):
        print(f"request {m}: {tokens[m, :8].tolist()} ...")


if __name__ == "__main__":
    main()
