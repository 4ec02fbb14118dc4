"""Measured cases of the operators around the packed projections: per-request
low-rank adapters (rq_lora), the token shift (rq_shift), the RWKV-7 state
recurrence (rq_wkv7) and the treatment of the head's logits (rq_logits).

A case names one operator and its sizes.  ``run`` makes one pass, either in
plain float32 torch operations (``own`` false) or through the package's entry
points (``own`` true).  Widths, head counts and the vocabulary are those of
this repository's workloads (gemm_rwkv_decode_amd/synth.py); the rest are
generic.
"""
import math

import torch

own = False

HEAD = 64            # channels of a head
VOCAB = 65536        # rows of the vocabulary head
WIDTHS = (768, 2048, 2560, 4096)
DECAY = math.exp(-0.5)


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one request with an adapter on one projection of the smallest model
        {"name": "lora 1 row 768", "op": "lora", "M": 1, "N": 768, "K": 768, "count": 1,
         "adapters": 4, "rank": 8, "without": 0, "segments": False},
        # a decode batch, each request with its own adapter or none, on receptance, key and
        # value together
        {"name": "lora rkv 32 requests", "op": "lora", "M": 32, "N": 4096, "K": 4096, "count": 3,
         "adapters": 24, "rank": 64, "without": 5, "segments": False},
        # prompts of three adapters, one after another, on an FFN key
        {"name": "lora prompts FFN key", "op": "lora", "M": 2047, "N": 16384, "K": 4096,
         "count": 1, "adapters": 3, "rank": 64, "without": 130, "segments": True},
        # the smallest call there is: one token of the smallest model
        {"name": "shift 1 token", "op": "shift", "tokens": 1, "sequences": 1, "width": 768,
         "mixes": 6},
        # a chunk of prompts with single tokens among them
        {"name": "shift ragged", "op": "shift", "tokens": 4001, "sequences": 23, "width": 2560,
         "mixes": 6},
        # one token of the smallest model
        {"name": "wkv7 1 token", "op": "wkv7", "tokens": 1, "sequences": 1, "heads": 12,
         "half": False},
        # a decode batch of the largest model: the state is the traffic
        {"name": "wkv7 decode 64", "op": "wkv7", "tokens": 64, "sequences": 64, "heads": 64,
         "half": False},
        # prompts and single tokens in one call, binary16 inputs
        {"name": "wkv7 ragged half", "op": "wkv7", "tokens": 1531, "sequences": 9, "heads": 40,
         "half": True},
        # one long prompt
        {"name": "wkv7 prompt 4096", "op": "wkv7", "tokens": 4096, "sequences": 1, "heads": 64,
         "half": False},
        # one request's next token
        {"name": "logits 1 row", "op": "logits", "M": 1, "V": VOCAB, "history": 257, "biases": 3,
         "masks": 1},
        # a decode batch with grammars and biases
        {"name": "logits 64 rows", "op": "logits", "M": 64, "V": VOCAB, "history": 1000,
         "biases": 40, "masks": 9},
        # long conversations, an odd vocabulary (rows start at any 4 bytes)
        {"name": "logits long history", "op": "logits", "M": 200, "V": VOCAB - 7,
         "history": 12000, "biases": 0, "masks": 3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("lora", "shift", "wkv7", "logits"))
    if op == "lora":
        seg = rng.random() < 0.4
        m = _log(rng, 65, 2047) if seg else _log(rng, 1, 64)
        return {"op": op, "M": m, "N": rng.choice(WIDTHS) * rng.choice((1, 4)) - rng.choice((0, 0, 3)),
                "K": rng.choice(WIDTHS), "count": 1 if seg else rng.choice((1, 3)),
                "adapters": rng.randint(1, 5) if seg else _log(rng, 1, 48),
                "rank": 8 * _log(rng, 1, 12), "without": rng.randint(0, m // 4), "segments": seg}
    if op == "shift":
        b = _log(rng, 1, 64)
        return {"op": op, "tokens": max(b, _log(rng, 1, 4001)), "sequences": b,
                "width": 8 * _log(rng, 96, 512), "mixes": rng.choice((1, 6))}
    if op == "wkv7":
        b = _log(rng, 1, 64)
        h = rng.randint(12, 64)
        t = b if rng.random() < 0.4 else max(b, _log(rng, 2, 3000))
        return {"op": op, "tokens": t, "sequences": b, "heads": h, "half": rng.random() < 0.5}
    m = _log(rng, 1, 200)
    return {"op": op, "M": m, "V": _log(rng, 16384, VOCAB), "history": _log(rng, 1, 12000),
            "biases": rng.choice((0, _log(rng, 1, 300))), "masks": rng.randint(0, 8)}


def work(case):
    op = case["op"]
    if op == "lora":
        m, n, k, c = case["M"], case["N"], case["K"], case["count"]
        ranks = _ranks(case)
        rows = m - case["without"]
        used = min(rows, case["adapters"])
        per = [sum(ranks[i] for i in range(used)),
               sum(ranks[j % used] for j in range(rows)) if used else 0]
        return {"bytes": c * (2 * per[0] * (k + n) + 2 * rows * k + 8 * m * n),
                "flops": c * 2 * per[1] * (k + n)}
    if op == "shift":
        t, b, d, n = case["tokens"], case["sequences"], case["width"], case["mixes"]
        return {"bytes": 2 * d * (t + n * t + n + 2 * b), "flops": 3 * n * t * d}
    if op == "wkv7":
        t, b, h = case["tokens"], case["sequences"], case["heads"]
        e = 2 if case["half"] else 4
        return {"bytes": t * h * HEAD * (6 * e + 4) + 2 * 4 * b * h * HEAD * HEAD,
                "flops": 9 * t * h * HEAD * HEAD}
    m, v = case["M"], case["V"]
    return {"bytes": 8 * m * v + case["masks"] * ((v + 31) // 32) * 4 +
            m * (4 * case["history"] + 8 * case["biases"]),
            "flops": 4 * m * v}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _ranks(case):
    """Adapters of mixed ranks: the largest, then halves and quarters of it."""
    return [max(8, case["rank"] // (1, 2, 1, 4)[i % 4] // 8 * 8) for i in range(case["adapters"])]


def _lengths(tokens, sequences, g):
    """Lengths of `sequences` sequences of `tokens` tokens in all; with more
    tokens than sequences about a third of them are single tokens."""
    if tokens == sequences:
        return [1] * sequences
    share = torch.rand(sequences, generator=g, dtype=torch.float64) ** 2 + 0.02
    share[torch.rand(sequences, generator=g) < 0.33] = 0.0
    if float(share.sum()) == 0.0:
        share[0] = 1.0
    extra = (share / share.sum() * (tokens - sequences)).floor().long()
    extra[int(share.argmax())] += tokens - sequences - int(extra.sum())
    return [1 + int(e) for e in extra]


def prepare(case, seed):
    dev = "cuda"
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    s = {"case": case}
    op = case["op"]
    if op == "lora":
        m, n, k = case["M"], case["N"], case["K"]
        ranks = _ranks(case)
        off = [0]
        for r in ranks:
            off.append(off[-1] + r)
        rows = m - case["without"]
        ids = [j % min(rows, case["adapters"]) for j in range(rows)] + [-1] * case["without"]
        if case["segments"]:
            ids.sort()
        else:
            ids = [ids[i] for i in torch.randperm(m, generator=host).tolist()]
        s.update(host_ids=ids, host_off=off, ids=ints(ids), off=ints(off), rank=max(ranks),
                 scales=torch.rand(len(ranks), generator=g, device=dev) + 0.5, problems=[])
        for _ in range(case["count"]):
            a = randn(off[-1], k, dtype=torch.float16, scale=k ** -0.5)
            b = randn(off[-1] * n, dtype=torch.float16, scale=0.1)
            x = randn(m, k, dtype=torch.float16)
            x[:, int(torch.randint(k, (1,), generator=host))] *= 50.0  # a massive channel
            y_in = randn(m, n)
            s["problems"].append((a, b, x, y_in, torch.empty_like(y_in), n, k))
    elif op == "shift":
        t, b, d = case["tokens"], case["sequences"], case["width"]
        lens = _lengths(t, b, host)
        s.update(lens=lens, off=ints([sum(lens[:i]) for i in range(b + 1)]),
                 x=randn(t, d, dtype=torch.float16),
                 mu=torch.rand((case["mixes"], d), generator=g, device=dev).half(),
                 state=randn(b, d, dtype=torch.float16),
                 out=torch.empty((case["mixes"], t, d), dtype=torch.float16, device=dev))
    elif op == "wkv7":
        t, b, h = case["tokens"], case["sequences"], case["heads"]
        dt = torch.float16 if case["half"] else torch.float32
        lens = _lengths(t, b, host)
        kappa = torch.nn.functional.normalize(randn(t, h, HEAD), dim=-1)
        s.update(lens=lens, off=ints([sum(lens[:i]) for i in range(b + 1)]),
                 slots=ints(torch.randperm(b, generator=host).tolist()),
                 r=randn(t, h * HEAD, dtype=dt), w=(randn(t, h * HEAD, scale=2.0) - 2.0).to(dt),
                 k=randn(t, h * HEAD, dtype=dt), v=randn(t, h * HEAD, dtype=dt),
                 kappa=kappa.reshape(t, h * HEAD).to(dt),
                 eta=torch.sigmoid(randn(t, h * HEAD)).to(dt),
                 state=randn(b, h, HEAD, HEAD), y=torch.empty((t, h * HEAD), device=dev))
    else:
        m, v, n, nb = case["M"], case["V"], case["history"], case["biases"]
        rows = [max(0, n - int(i)) for i in torch.randint(0, n // 4 + 1, (m,), generator=host)]
        off = [0]
        for r in rows:
            off.append(off[-1] + r)
        # text repeats itself: a Zipf-like law over the vocabulary
        hist = (torch.rand(off[-1], generator=g, device=dev) ** 4 * v).to(torch.int32).clamp_(max=v - 1)
        words = (v + 31) // 32
        masks = torch.randint(-2 ** 31, 2 ** 31, (case["masks"], words), generator=g, device=dev,
                              dtype=torch.int64).to(torch.int32)
        mask_ids = torch.randint(-1, max(1, case["masks"]), (m,), generator=host)
        s.update(logits=randn(m, v, scale=3.0), out=torch.empty((m, v), device=dev),
                 history=hist, history_off=ints(off), prompt=ints([r // 2 for r in rows]),
                 repetition=torch.rand(m, generator=g, device=dev) + 1.0,
                 presence=torch.rand(m, generator=g, device=dev),
                 frequency=torch.rand(m, generator=g, device=dev),
                 bias_off=ints([i * nb for i in range(m + 1)]),
                 bias_ids=torch.randint(0, v, (m * nb,), generator=g, device=dev, dtype=torch.int32),
                 bias=randn(m * nb, scale=4.0), masks=masks,
                 mask_ids=mask_ids.to(dev, torch.int32) if case["masks"] else None,
                 tokens=torch.empty(m, dtype=torch.int32, device=dev))
    if own:
        s["call"] = _call(s)
    return s


def _call(s):
    """The prepared call that a step loop keeps."""
    import gemm_rwkv_decode_amd as rq
    op = s["case"]["op"]
    if op == "lora":
        return rq.prepare("rq_lora", s["problems"], s["ids"], s["off"], s["scales"], s["rank"])
    if op == "shift":
        return rq.prepare("rq_shift", s["x"], s["mu"], s["state"], s["out"], s["off"])
    if op == "wkv7":
        return rq.prepare("rq_wkv7", s["r"], s["w"], s["k"], s["v"], s["kappa"], s["eta"],
                          s["state"], s["y"], s["off"], s["slots"])
    has_bias, has_mask = s["bias"].numel() > 0, s["mask_ids"] is not None
    return rq.prepare(
        "rq_logits", s["logits"], s["out"], s["tokens"],
        history=(s["history"], s["history_off"], s["prompt"]), repetition=s["repetition"],
        presence=s["presence"], frequency=s["frequency"],
        bias=(s["bias_ids"], s["bias"], s["bias_off"]) if has_bias else None,
        masks=(s["masks"], s["mask_ids"]) if has_mask else None)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
    if op == "lora":
        return [p[4] for p in s["problems"]] if own else _lora(s)
    if op == "shift":
        return {"out": s["out"], "state": s["state"]} if own else _shift(s)
    if op == "wkv7":
        return {"y": s["y"], "state": s["state"]} if own else _wkv7(s)
    return {"logits": s["out"], "tokens": s["tokens"]} if own else _logits(s)


def _lora(s):
    out = []
    for a, b, x, y_in, _, n, _ in s["problems"]:
        y = y_in.clone()
        for i in range(len(s["host_off"]) - 1):
            lo, hi = s["host_off"][i], s["host_off"][i + 1]
            rows = (s["ids"] == i).nonzero().flatten()
            if not len(rows):
                continue
            t = x[rows].float() @ a[lo:hi].float().T
            y[rows] += s["scales"][i] * (t @ b[lo * n:hi * n].view(n, hi - lo).float().T)
        out.append(y)
    return out


def _shift(s):
    x, mu = s["x"].float(), s["mu"].float()
    off = s["off"].long()
    prev = torch.roll(x, 1, 0)
    some = off[1:] > off[:-1]
    prev[off[:-1][some]] = s["state"].float()[some]
    out = (x + (prev - x) * mu[:, None, :]).half()
    s["state"][some] = s["x"][off[1:][some] - 1]
    return {"out": out, "state": s["state"]}


def _wkv7(s):
    b, h = len(s["lens"]), s["case"]["heads"]
    off = s["off"].long()
    steps = max(s["lens"])
    at = off[:-1, None] + torch.arange(steps, device="cuda")           # [b][steps]
    live = at < off[1:, None]
    at = torch.where(live, at, 0)

    def take(x):  # [steps][b][h][HEAD]
        return x.float()[at.T].view(steps, b, h, HEAD)

    on = live.T[:, :, None, None].float()
    r, v, k, kappa = take(s["r"]), take(s["v"]), take(s["k"]) * on, take(s["kappa"]) * on
    d = torch.exp(-DECAY * torch.sigmoid(take(s["w"])))
    d = torch.where(on > 0, d, 1.0)
    ek = take(s["eta"]) * kappa
    slot = s["slots"].long()
    S = s["state"][slot]
    y = torch.empty_like(r)
    for t in range(steps):
        sk = (S * kappa[t, :, :, None, :]).sum(-1, keepdim=True)
        S = S * d[t, :, :, None, :] - sk * ek[t, :, :, None, :] + v[t, :, :, :, None] * k[t, :, :, None, :]
        y[t] = (S * r[t, :, :, None, :]).sum(-1)
    s["state"][slot] = S
    return {"y": y.transpose(0, 1)[live].reshape(-1, h * HEAD), "state": s["state"]}


def _rows(off, m):
    """The row of every entry of a ragged list, and its place in the row."""
    off = off.long()
    at = torch.arange(int(off[-1]), device=off.device)
    row = torch.searchsorted(off, at, right=True) - 1
    return row, at - off[row]


def _logits(s):
    z = s["logits"].float()
    m, v = z.shape
    row, place = _rows(s["history_off"], m)
    tok = s["history"].long()
    ours = place >= s["prompt"].long()[row]
    seen = torch.zeros((m, v), dtype=torch.bool, device="cuda")
    seen[row, tok] = True
    count = torch.zeros((m, v), device="cuda")
    count.view(-1).scatter_add_(0, row * v + tok, ours.float())
    rep = s["repetition"][:, None]
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - s["frequency"][:, None] * count
    z = torch.where(count > 0, z - s["presence"][:, None], z)
    if s["bias"].numel():
        row, place = _rows(s["bias_off"], m)
        last = torch.full((m * v,), -1, device="cuda")
        last.scatter_reduce_(0, row * v + s["bias_ids"].long(),
                             torch.arange(len(row), device="cuda"), "amax")
        last = last.view(m, v)
        z = torch.where(last >= 0, z + s["bias"][last.clamp(min=0)], z)
    if s["mask_ids"] is not None:
        ids = s["mask_ids"].long()
        place = torch.arange(v, device="cuda")
        bits = (s["masks"][ids.clamp(min=0)][:, place // 32] >> (place % 32).int()) & 1
        z = torch.where((bits == 0) & (ids >= 0)[:, None], float("-inf"), z)
    top = z.amax(-1, keepdim=True)
    first = torch.where(z == top, torch.arange(v, device="cuda"), v).amin(-1)
    first = torch.where(top[:, 0] > float("-inf"), first, -1)
    return {"logits": z, "tokens": first.int()}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f8 = torch.float64
    if op == "lora":
        out = []
        for a, b, x, y_in, _, n, _ in s["problems"]:
            y = y_in.to(f8)
            for i in sorted(set(s["host_ids"]) - {-1}):
                lo, hi = s["host_off"][i:i + 2]
                rows = torch.tensor([j for j, q in enumerate(s["host_ids"]) if q == i], device="cuda")
                down = torch.mm(a[lo:hi].to(f8), x[rows].to(f8).T.contiguous())      # [r][rows]
                up = torch.mm(b[lo * n:hi * n].reshape(n, -1).to(f8), down)           # [n][rows]
                y.index_add_(0, rows, up.T.contiguous(), alpha=float(s["scales"][i]))
            out.append(y)
        return out
    if op == "shift":
        x, mu, state = s["x"].to(f8), s["mu"].to(f8), s["state"].to(f8)
        out, end, at = torch.empty(s["out"].shape, dtype=f8, device="cuda"), state.clone(), 0
        for q, n in enumerate(s["lens"]):
            seq = x[at:at + n]
            before = torch.cat([state[q:q + 1], seq[:-1]])
            out[:, at:at + n] = seq * (1 - mu[:, None]) + before * mu[:, None]
            end[q] = seq[-1]
            at += n
        return {"out": out, "state": end}
    if op == "wkv7":
        h = case["heads"]
        r, w, k, v, kappa, eta = (s[c].to(f8).view(-1, h, HEAD, 1) for c in
                                  ("r", "w", "k", "v", "kappa", "eta"))
        d = torch.exp(-math.exp(-0.5) / (1 + torch.exp(-w)))
        state = s["state"].to(f8)
        y, at = torch.empty((case["tokens"], h, HEAD), dtype=f8, device="cuda"), 0
        for n, slot in zip(s["lens"], s["slots"].tolist()):
            S = state[slot].transpose(1, 2).contiguous()     # [h][key][value]
            for t in range(at, at + n):
                gone = (S * kappa[t]).sum(1, keepdim=True)   # [h][1][value]
                S = d[t] * S - (eta[t] * kappa[t]) * gone + k[t] * v[t].transpose(1, 2)
                y[t] = (r[t] * S).sum(1)
            state[slot] = S.transpose(1, 2)
            at += n
        return {"y": y.view(-1, h * HEAD), "state": state}
    z = s["logits"].to(f8)
    m, width = z.shape
    h_off, b_off = s["history_off"].tolist(), s["bias_off"].tolist()
    prompt = s["prompt"].tolist()
    tokens = []
    for i in range(m):
        past = s["history"][h_off[i]:h_off[i + 1]].long()
        count = torch.bincount(past[prompt[i]:], minlength=width)
        seen = torch.bincount(past, minlength=width) > 0
        rep, pres, freq = (float(s[c][i]) for c in ("repetition", "presence", "frequency"))
        u = z[i]
        u = torch.where(seen & (u > 0), u / rep, torch.where(seen, u * rep, u))
        u = u - freq * count - pres * (count > 0)
        which = s["bias_ids"][b_off[i]:b_off[i + 1]].tolist()
        held = dict(zip(which, s["bias"][b_off[i]:b_off[i + 1]].tolist()))  # the last of an id stays
        if held:
            u[torch.tensor(list(held), device="cuda")] += torch.tensor(list(held.values()), dtype=f8,
                                                                       device="cuda")
        q = -1 if s["mask_ids"] is None else int(s["mask_ids"][i])
        if q >= 0:
            word = s["masks"][q].long()[:, None] >> torch.arange(32, device="cuda")
            u = u.masked_fill((word & 1).view(-1)[:width] == 0, float("-inf"))
        z[i] = u
        best = u.max()
        tokens.append(int((u == best).nonzero()[0]) if float(best) > float("-inf") else -1)
    return {"logits": z, "tokens": torch.tensor(tokens, dtype=torch.int32, device="cuda")}
