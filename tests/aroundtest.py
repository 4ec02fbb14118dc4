"""Plain 64-bit forms of the calls around the products, and helpers shared by
their tests.  Everything here runs on the CPU in numpy or torch float64 from
the formulas of include/rq.h."""
import math

import numpy as np
import torch

EPS = 2.0 ** -24  # half a unit in the last place of binary32


def offsets_of(lens, start=0):
    off = [start]
    for n in lens:
        off.append(off[-1] + n)
    return off


def dev_ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def guarded(shape, dtype, fill):
    """A tensor inside a larger allocation, and a check that nothing outside it
    was written."""
    n = int(np.prod(shape)) if len(shape) else 1
    pad = 4096
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    view = whole[pad:pad + n].view(shape)

    def untouched():
        torch.cuda.synchronize()
        edge = torch.cat([whole[:pad], whole[pad + n:]])
        want = torch.full_like(edge, fill)
        same = edge.eq(want) | (edge.isnan() & want.isnan()) if dtype.is_floating_point \
            else edge.eq(want)
        return bool(same.all())
    return view, untouched


def randn(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g) * scale).to(dtype)


# ------------------------------------------------------------------ shift
def shift_ref(x, mu, state, lens, slots, start=0):
    """(out float64 [n][T][D], state) for float16 numpy inputs."""
    x, mu = x.astype(np.float64), mu.astype(np.float64)
    out = np.full((mu.shape[0],) + x.shape, np.nan)
    new = state.copy()
    at = start
    for n, slot in zip(lens, slots):
        ok = 0 <= slot < state.shape[0]
        prev = state[slot].astype(np.float64) if ok else np.zeros(x.shape[1])
        for t in range(at, at + n):
            out[:, t] = x[t] + (prev - x[t]) * mu
            prev = x[t]
        if n and ok:
            new[slot] = x[at + n - 1].astype(np.float16)
        at += n
    return out, new


# ------------------------------------------------------------------- wkv7
def wkv7_ref(ins, state, lens, slots, start=0):
    """(y, state, row norms) in float64: ins maps r, w, k, v, kappa, eta to
    [T][H][64]; the norms are the largest 2-norm each state row had up to and
    at each token, [T][H][64]."""
    T, H, _ = ins["r"].shape
    y = np.full((T, H, 64), np.nan)
    norms = np.zeros((T, H, 64))
    new = state.astype(np.float64).copy()
    at = start
    d = np.exp(-math.exp(-0.5) / (1 + np.exp(-ins["w"])))
    for n, slot in zip(lens, slots):
        ok = 0 <= slot < state.shape[0]
        S = new[slot].copy() if ok else np.zeros((H, 64, 64))
        top = np.sqrt((S ** 2).sum(-1))
        for t in range(at, at + n):
            kap, k, v = ins["kappa"][t], ins["k"][t], ins["v"][t]
            gone = np.einsum("hij,hj->hi", S, kap)
            S = (S * d[t][:, None, :] - gone[:, :, None] * (ins["eta"][t] * kap)[:, None, :]
                 + v[:, :, None] * k[:, None, :])
            y[t] = np.einsum("hij,hj->hi", S, ins["r"][t])
            top = np.maximum(top, np.sqrt((S ** 2).sum(-1)))
            norms[t] = top
        if n and ok:
            new[slot] = S
        at += n
    return y, new, norms


# ------------------------------------------------------------------- lora
def lora_ref(problem, ids, off, scales, total_rank, max_rank):
    """(y, bound) in float64; bound is the sum of absolute products."""
    a, b, x, y_in, N, K = problem
    M = x.shape[0]
    y = np.zeros((M, N)) if y_in is None else y_in.astype(np.float64)
    bound = np.abs(y)
    for m in range(M):
        i = ids[m]
        if not 0 <= i < len(off) - 1:
            continue
        lo, hi = off[i], off[i + 1]
        r = hi - lo
        if lo < 0 or hi > total_rank or r <= 0 or r > max_rank or r % 8 or lo % 8:
            continue
        A = a[lo:hi].astype(np.float64)
        B = b[lo * N:hi * N].reshape(N, r).astype(np.float64)
        s = 1.0 if scales is None else float(scales[i])
        xm = x[m].astype(np.float64)
        y[m] += s * (B @ (A @ xm))
        bound[m] += abs(s) * (np.abs(B) @ (np.abs(A) @ np.abs(xm)))
    return y, bound


# ----------------------------------------------------------------- logits
def logits_ref(z, history=None, repetition=None, presence=None, frequency=None, bias=None,
               masks=None):
    """(float32 logits, tokens), each operation rounded to float32 in the
    documented order.  history: per row (tokens, prompt length); bias: per row
    (ids, values); masks: (bool [n][V], per row index)."""
    z = z.astype(np.float32).copy()
    M, V = z.shape
    tokens = np.empty(M, dtype=np.int32)
    f = np.float32
    for m in range(M):
        if history is not None:
            toks, given = history[m]
            seen, count = {}, {}
            for p, t in enumerate(toks):
                if 0 <= t < V:
                    seen[t] = True
                    if p >= given:
                        count[t] = count.get(t, 0) + 1
            rep = f(1) if repetition is None else f(repetition[m])
            pres = f(0) if presence is None else f(presence[m])
            freq = f(0) if frequency is None else f(frequency[m])
            for t in seen:
                u = z[m, t]
                u = f(u / rep) if u > 0 else f(u * rep)
                c = count.get(t, 0)
                u = f(u - f(freq * f(c)))
                z[m, t] = f(u - pres) if c else u
        if bias is not None:
            held = {}
            for t, v in zip(*bias[m]):
                if 0 <= t < V:
                    held[int(t)] = f(v)
            for t, v in held.items():
                z[m, t] = f(z[m, t] + v)
        if masks is not None:
            bits, which = masks
            if 0 <= which[m] < len(bits):
                z[m, ~bits[which[m]]] = -np.inf
        row = np.where(np.isnan(z[m]), -np.inf, z[m])
        best = int(np.argmax(row))
        tokens[m] = best if row[best] > -np.inf else -1
    return z, tokens


def pack_masks(bits):
    """bool [n][V] -> int32 [n][(V + 31) // 32]."""
    n, V = bits.shape
    words = (V + 31) // 32
    padded = np.zeros((n, words * 32), dtype=np.uint8)
    padded[:, :V] = bits
    return torch.from_numpy(
        np.packbits(padded, axis=1, bitorder="little").view(np.int32).reshape(n, words).copy())
