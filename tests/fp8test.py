"""Plain 64-bit forms of the block-scaled FP8 calls and of the group norm, from the
formulas of include/rq.h, and helpers shared by their tests."""
import numpy as np
import torch

import gemm_rwkv_decode_amd as rq

U = 2.0 ** -24       # half a unit in the last place of binary32, relative
HALF = 2.0 ** -11    # of binary16
BLOCK = 128
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def e4m3_table():
    """The value of every E4M3 code, from the format's definition."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 127) == 127 else (-a if c >> 7 else a)
    return v


TABLE = e4m3_table()
POSITIVE = TABLE[:127]                   # ascending
MIDDLE = (POSITIVE[1:] + POSITIVE[:-1]) / 2


def nearest_e4m3(u):
    """The E4M3 value nearest each |u| <= 448, ties to the even code."""
    a = np.abs(u)
    i = np.searchsorted(MIDDLE, a, side="left")       # a tie goes to the lower code ...
    tie = (i < 126) & (a == MIDDLE[np.minimum(i, 125)])
    i = i + (tie & (i % 2 == 1))                      # ... unless that one is odd
    return np.copysign(POSITIVE[i], u)


def quant_ref(a):
    """(values, scales) in float64 of [M][K] values a."""
    v = np.asarray(a, dtype=np.float64).reshape(len(a), -1, BLOCK)
    fine = np.isfinite(v)
    top = np.where(fine, np.abs(v), 0).max(-1)
    e = np.full(top.shape, -126.0)
    for k in range(-125, 129):
        e = np.where(top > 448.0 * 2.0 ** (k - 1), k, e)
    s = 2.0 ** e
    q = nearest_e4m3(np.where(fine, v, 0) / s[..., None])
    return np.where(fine, q, np.nan).reshape(np.shape(a)), s


def act(x, which):
    """float64 of act(x), the square rounded to binary32."""
    x = np.asarray(x)
    if which == rq.RQ_ACT_NONE:
        return x.astype(np.float64)
    x = x.astype(np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        a = np.where(x < 0, np.float32(0), x)
        return (a * a).astype(np.float64)


def same(a, b):
    """Equal values (NaN equal NaN, the sign of zero aside)."""
    a, b = np.asarray(a), np.asarray(b)
    return a.shape == b.shape and bool(np.all((a == b) | (np.isnan(a) & np.isnan(b))))


def values(t):
    """float64 numpy of an E4M3 or scale tensor."""
    if t.dtype in (E4M3, E8M0):
        return t.cpu().to(torch.float32).double().numpy()
    return t.cpu().double().numpy()


def random_codes(g, *shape, spread=None):
    """E4M3 codes on the GPU: normal values on the whole range, or (spread) all
    finite codes alike."""
    if spread:
        c = torch.randint(0, 254, shape, generator=g, dtype=torch.int64)
        c = torch.where(c >= 127, c + 1, c)            # the codes 127 and 255 are NaN
        return c.to(torch.uint8).cuda().view(E4M3)
    x = torch.randn(shape, generator=g) * 100
    return x.clamp(-448, 448).cuda().to(E4M3)


def random_scales(g, rows, cols, e8m0, lo=-9, hi=-3):
    s = torch.exp2(torch.randint(lo, hi + 1, (rows, cols), generator=g).float())
    if e8m0:
        return s.cuda().to(E8M0)
    return (s * (1 + torch.rand((rows, cols), generator=g))).cuda()


def widen(q, s, rows):
    """float64 [rows][K] of block-scaled values; s has a row for each row of q, or
    one for 128 of them."""
    s = s.to(torch.float32).double()
    if s.shape[0] != rows:
        s = s.repeat_interleave(BLOCK, 0)[:rows]
    return q.to(torch.float32).double() * s.repeat_interleave(BLOCK, 1)


def gemm_ref(w, ws, x, xs, y_in=None):
    """(y, sum of magnitudes) in float64 on the GPU."""
    wd, xd = widen(w, ws, w.shape[0]), widen(x, xs, x.shape[0])
    y, mag = torch.mm(xd, wd.T.contiguous()), torch.mm(xd.abs(), wd.abs().T.contiguous())
    if y_in is not None:
        y, mag = y + y_in, mag + y_in.abs()
    return y, mag


def gemm_bound(y, mag, K, out):
    """Binary32 sums: 128 exact products in any order, an error of at most a unit
    in the last place (2 U) of the magnitudes for each, then one rounding for a
    block, one for its scale, one for y_in.  The FP8 instructions drop at most
    7 of 8 products of a group to 2^-13 of the largest."""
    b = (2 * 128 + K // BLOCK + 4) * U * mag
    if out != "f32":
        b = b + 7 * 2.0 ** -13 * mag
        b = b + HALF * (y.abs() + b) + 2.0 ** -25
    return b


def norm_ref(y, groups, weight, bias, eps, bonus, gate, silu):
    """(out, bound of a binary32 evaluation) in float64 numpy."""
    T, C = y.shape
    G = C // groups
    f = [None if t is None else np.asarray(t, dtype=np.float64) for t in (y, weight, bias, gate)]
    y, weight, bias, gate = f
    y = y.reshape(T, groups, G)
    big = np.abs(y).max(-1, keepdims=True)
    c = y - y.mean(-1, keepdims=True)
    sd = np.sqrt((c ** 2).mean(-1, keepdims=True) + eps)
    ec = 12 * U * big                      # 2 adds in a lane, 6 over lanes, the division, the difference
    n = c / sd
    en = ec / sd + np.abs(n) * (ec / sd + 16 * U)
    w = np.ones(C) if weight is None else weight
    b = np.zeros(C) if bias is None else bias
    n, en = n.reshape(T, C), en.reshape(T, C)
    z, e = n * w + b, en * np.abs(w) + 2 * U * (np.abs(n * w) + np.abs(b))
    if bonus is not None:
        r, k, r_k, v = (np.asarray(t, dtype=np.float64) for t in bonus)
        p = (r * k * r_k).reshape(T, groups, G)
        dot = np.repeat(p.sum(-1), G, axis=-1)
        mag = np.repeat(np.abs(p).sum(-1), G, axis=-1)
        e = e + 14 * U * mag * np.abs(v) + 2 * U * (np.abs(z) + np.abs(dot * v))
        z = z + dot * v
    if gate is not None:
        with np.errstate(over="ignore"):
            g = gate / (1 + np.exp(-gate)) if silu else gate
        e = e * np.abs(g) + (12 if silu else 2) * U * np.abs(z * g) + 2.0 ** -140
        if silu:
            # e^-|gate| below 2^-126 has a spacing of 2^-149: a unit of it, times |gate z|
            e = e + 2.0 ** -148 * np.abs(gate * z)
        z = z * g
    return z, e
