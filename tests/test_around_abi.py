"""What rq_shift, rq_wkv7, rq_lora and rq_logits refuse, on the CPU: every
check runs on the host before any HIP call, so the addresses are never
dereferenced.  A call that passes all checks ends with RQ_ERR_DEVICE where
there is no GPU."""
import ctypes
import os
import re

import pytest
import torch

import gemm_rwkv_decode_amd as rq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
G = 1 << 30
A = 0x7F0000000000


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(rq.LIB_PATH):
        pytest.fail("librq.so is not built (run __graft_entry__.build())")
    return rq.lib()


def passes(status):
    return status == (rq.RQ_ERR_DEVICE if not torch.cuda.is_available() else status) and \
        status in (rq.RQ_OK, rq.RQ_ERR_DEVICE)


no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="the accepted calls would run on made-up addresses")


def test_limits_match_the_header():
    src = open(os.path.join(ROOT, "include", "rq.h")).read()
    for n in ("RQ_MAX_SEQUENCES", "RQ_SHIFT_MAX_MIXES", "RQ_WKV_HEAD", "RQ_LORA_MAX_M",
              "RQ_LORA_MAX_RANK", "RQ_LORA_MAX_BATCH", "RQ_LOGITS_MAX_M"):
        assert getattr(rq, n) == int(re.search(rf"#define {n} (\d+)", src).group(1)), n
    assert rq.RQ_LOGITS_WORKSPACE_BYTES == 64 << 10
    assert re.search(r"RQ_LOGITS_WORKSPACE_BYTES \(64 << 10\)", src)
    assert (rq.RQ_TYPE_F32, rq.RQ_TYPE_F16) == (0, 1)


# ------------------------------------------------------------------ shift
def shift(L, **kw):
    a = dict(x=A, mu=A + G, state=A + 2 * G, out=A + 3 * G, off=A + 8 * G, slots=A + 9 * G, T=10,
             D=64, n=6, seqs=3, nslots=4)
    a.update(kw)
    return L.rq_shift(*[a[k] for k in ("x", "mu", "state", "out", "off", "slots", "T", "D", "n",
                                       "seqs", "nslots")], None)


@no_gpu
@pytest.mark.parametrize("kw", [{}, dict(slots=None), dict(state=None, nslots=0), dict(n=8),
                                dict(seqs=65536), dict(off=A + 8 * G + 4), dict(D=8)])
def test_shift_accepts(L, kw):
    if kw.get("seqs"):
        kw["nslots"] = 70000
    assert passes(shift(L, **kw))


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), "NULL"), (dict(mu=None), "NULL"), (dict(out=None), "NULL"),
    (dict(off=None), "NULL"), (dict(state=None), "NULL"),
    (dict(T=0), "SHAPE"), (dict(D=0), "SHAPE"), (dict(D=4), "SHAPE"), (dict(D=68), "SHAPE"),
    (dict(n=0), "SHAPE"), (dict(n=9), "SHAPE"), (dict(seqs=0), "SHAPE"),
    (dict(seqs=65537), "SHAPE"), (dict(nslots=-1), "SHAPE"), (dict(slots=None, nslots=2), "SHAPE"),
    (dict(slots=None, nslots=0, state=None), "SHAPE"),
    (dict(x=A + 8), "ALIGN"), (dict(mu=A + G + 2), "ALIGN"), (dict(out=A + 3 * G + 4), "ALIGN"),
    (dict(state=A + 2 * G + 8), "ALIGN"), (dict(off=A + 8 * G + 2), "ALIGN"),
    (dict(slots=A + 9 * G + 1), "ALIGN"),
    (dict(out=A), "ALIAS"), (dict(out=A + 16 - 6 * 10 * 64 * 2 // 16 * 16), "ALIAS"),
    (dict(state=A), "ALIAS"), (dict(state=A + 3 * G), "ALIAS"), (dict(out=A + 9 * G), "ALIAS"),
    (dict(state=A + 8 * G), "ALIAS"), (dict(mu=A + 3 * G + 64), "ALIAS"),
])
def test_shift_refuses(L, kw, want):
    assert shift(L, **kw) == getattr(rq, "RQ_ERR_" + want)


# ------------------------------------------------------------------- wkv7
WKV = ("r", "w", "k", "v", "kappa", "eta", "type", "state", "y", "off", "slots", "T", "H", "seqs",
       "nslots")


def wkv(L, **kw):
    a = {n: A + i * G for i, n in enumerate(WKV)}
    a.update(type=0, T=10, H=2, seqs=3, nslots=4)
    a.update(kw)
    return L.rq_wkv7(*[a[k] for k in WKV], None)


@no_gpu
@pytest.mark.parametrize("kw", [{}, dict(type=1), dict(slots=None), dict(state=None, nslots=0),
                                dict(H=4096, T=1), dict(k=A, r=A)])
def test_wkv7_accepts(L, kw):
    """Inputs may be the same array."""
    assert passes(wkv(L, **kw))


@pytest.mark.parametrize("kw,want",
                         [({n: None}, "NULL") for n in WKV[:6] + ("y", "off", "state")] +
                         [({n: A + WKV.index(n) * G + 8}, "ALIGN") for n in WKV[:6] + ("y", "state")] +
                         [({"y": A + i * G}, "ALIAS") for i in (0, 1, 2, 3, 4, 5, 7, 9, 10)] +
                         [({"state": A + i * G}, "ALIAS") for i in (0, 1, 2, 3, 4, 5, 9, 10)] + [
    (dict(type=2), "UNSUPPORTED"), (dict(type=-1), "UNSUPPORTED"), (dict(T=0), "SHAPE"),
    (dict(H=0), "SHAPE"), (dict(H=4097), "SHAPE"), (dict(seqs=0), "SHAPE"),
    (dict(seqs=65537), "SHAPE"), (dict(slots=None, nslots=2), "SHAPE"), (dict(off=A + 1), "ALIGN"),
])
def test_wkv7_refuses(L, kw, want):
    assert wkv(L, **kw) == getattr(rq, "RQ_ERR_" + want)


# ------------------------------------------------------------------- lora
def lora(L, problems=({},), **kw):
    arr = (rq.RqLoraProblem * max(1, len(problems)))()
    for i, q in enumerate(problems):
        p = dict(a=A, b=A + G, x=A + 2 * G, y_in=A + (3 + 2 * i) * G, y=A + (4 + 2 * i) * G, N=64,
                 K=128)
        p.update(q)
        arr[i] = rq.RqLoraProblem(*[p[k] for k in ("a", "b", "x", "y_in", "y", "N", "K")])
    c = dict(array=arr, count=len(problems), M=4, ids=A + 20 * G, off=A + 21 * G,
             scales=A + 22 * G, adapters=3, total=48, rank=16, ws=A + 30 * G, wsb=64 << 20)
    c.update(kw)
    return L.rq_lora(*[c[k] for k in ("array", "count", "M", "ids", "off", "scales", "adapters",
                                      "total", "rank", "ws", "wsb")], None)


@no_gpu
@pytest.mark.parametrize("problems,kw", [
    (({},), {}), (({}, {}, {}), {}), (({},) * 8, {}), ((dict(y_in=None),), {}),
    ((dict(y_in=A + 4 * G),), {}), (({},), dict(scales=None)), (({},), dict(M=8192)),
    (({},), dict(rank=128)), ((dict(a=None, b=None),), dict(total=0)),
    (({}, dict(a=A, b=A + G)), {}),
])
def test_lora_accepts(L, problems, kw):
    assert passes(lora(L, problems, **kw))


@pytest.mark.parametrize("problems,kw,want", [
    (({},), dict(array=None), "NULL"), (({},), dict(ids=None), "NULL"),
    (({},), dict(off=None), "NULL"), ((dict(a=None),), {}, "NULL"), ((dict(b=None),), {}, "NULL"),
    ((dict(x=None),), {}, "NULL"), ((dict(y=None),), {}, "NULL"),
    (({},), dict(count=0), "SHAPE"), (({},) * 9, {}, "SHAPE"), (({},), dict(M=0), "SHAPE"),
    (({},), dict(M=8193), "SHAPE"), (({},), dict(adapters=0), "SHAPE"),
    (({},), dict(rank=0), "SHAPE"), (({},), dict(rank=12), "SHAPE"),
    (({},), dict(rank=136), "SHAPE"), (({},), dict(total=-8), "SHAPE"),
    ((dict(K=12),), {}, "SHAPE"), ((dict(K=0),), {}, "SHAPE"), ((dict(N=0),), {}, "SHAPE"),
    ((dict(a=A + 8),), {}, "ALIGN"), ((dict(x=A + 2 * G + 2),), {}, "ALIGN"),
    ((dict(y=A + 4 * G + 4),), {}, "ALIGN"), (({},), dict(ws=A + 30 * G + 8), "ALIGN"),
    (({},), dict(ids=A + 20 * G + 2), "ALIGN"),
    ((dict(y=A + 3 * G + 16),), {}, "ALIAS"), ((dict(y=A + 2 * G),), {}, "ALIAS"),
    ((dict(y=A),), {}, "ALIAS"), ((dict(y=A + 20 * G),), {}, "ALIAS"),
    (({}, dict(y=A + 4 * G)), {}, "ALIAS"), (({}, dict(y_in=A + 4 * G)), {}, "ALIAS"),
    (({}, dict(x=A + 4 * G)), {}, "ALIAS"), (({},), dict(ws=A), "ALIAS"),
    (({},), dict(ws=A + 4 * G), "ALIAS"), (({},), dict(ws=A + 20 * G), "ALIAS"),
    (({},), dict(ws=None), "SCRATCH"), (({},), dict(wsb=16), "SCRATCH"),
])
def test_lora_refuses(L, problems, kw, want):
    assert lora(L, problems, **kw) == getattr(rq, "RQ_ERR_" + want)


def test_lora_workspace_size(L):
    assert rq.rq_lora_workspace_size([(4096, 4096)], 1, 1, 8) >= 16 * 4
    big = rq.rq_lora_workspace_size([(4096, 16384)] * 8, 8192, 100000, 128)
    assert big <= rq.RQ_GEMM_WORKSPACE_MAX_BYTES - rq.RQ_LOGITS_WORKSPACE_BYTES
    for M in (1, 2, 63, 64, 65, 500, 8192):
        for rank in (8, 64, 128):
            for n in (1, 3, 8):
                assert rq.rq_lora_workspace_size([(768, 16384)] * n, M, 64, rank) <= \
                    rq.RQ_GEMM_WORKSPACE_MAX_BYTES - rq.RQ_LOGITS_WORKSPACE_BYTES
    for args in (([(0, 64)], 1, 1, 8), ([(64, 60)], 1, 1, 8), ([(64, 64)], 0, 1, 8),
                 ([(64, 64)], 1, 0, 8), ([(64, 64)], 1, 1, 9), ([], 1, 1, 8)):
        with pytest.raises(rq.RqError) as e:
            rq.rq_lora_workspace_size(*args)
        assert e.value.status == rq.RQ_ERR_SHAPE
    b = ctypes.c_size_t(7)
    assert L.rq_lora_workspace_size(None, 1, 1, 1, 8, ctypes.byref(b)) == rq.RQ_ERR_NULL
    assert b.value == 0
    arr = (rq.RqLoraProblem * 1)()
    assert L.rq_lora_workspace_size(arr, 1, 1, 1, 8, None) == rq.RQ_ERR_NULL


# ----------------------------------------------------------------- logits
FIELDS = [f[0] for f in rq.RqLogitsArgs._fields_]


def logits(L, ws=A + 30 * G, wsb=64 << 10, null=False, **kw):
    a = {n: A + i * G for i, n in enumerate(FIELDS)}
    a.update(M=4, V=1000, history_len=100, bias_len=10, nmasks=2)
    a.update(kw)
    s = rq.RqLogitsArgs(**a)
    return L.rq_logits(None if null else ctypes.byref(s), ws, wsb, None)


ADDR = {n: A + i * G for i, n in enumerate(FIELDS)}


@no_gpu
@pytest.mark.parametrize("kw", [
    {}, dict(out=ADDR["logits"]), dict(tokens=None, ws=None, wsb=0),
    dict(history=None, history_offsets=None, history_len=-5), dict(bias_ids=None, bias=None),
    dict(masks=None, nmasks=0, mask_ids=None), dict(prompt=None, repetition=None, presence=None),
    dict(history_len=0, bias_len=0), dict(M=4096, V=16), dict(history=A + 4, tokens=ADDR["tokens"] + 4,
                                                             logits=A + 40 * G)])
def test_logits_accepts(L, kw):
    assert passes(logits(L, **kw))


@pytest.mark.parametrize("kw,want", [
    (dict(null=True), "NULL"), (dict(logits=None), "NULL"), (dict(out=None), "NULL"),
    (dict(history_offsets=None), "NULL"), (dict(bias=None), "NULL"),
    (dict(bias_offsets=None), "NULL"), (dict(mask_ids=None), "NULL"),
    (dict(M=0), "SHAPE"), (dict(M=4097), "SHAPE"), (dict(V=0), "SHAPE"),
    (dict(history_len=-1), "SHAPE"), (dict(bias_len=-1), "SHAPE"), (dict(nmasks=0), "SHAPE"),
    (dict(logits=A + 4), "ALIGN"), (dict(out=ADDR["out"] + 8), "ALIGN"),
    (dict(tokens=ADDR["tokens"] + 2), "ALIGN"), (dict(masks=ADDR["masks"] + 1), "ALIGN"),
    (dict(ws=A + 30 * G + 8), "ALIGN"),
    (dict(out=A + 16), "ALIAS"), (dict(tokens=ADDR["out"]), "ALIAS"),
    (dict(tokens=ADDR["logits"]), "ALIAS"), (dict(tokens=ADDR["masks"]), "ALIAS"),
    (dict(ws=ADDR["out"]), "ALIAS"), (dict(ws=ADDR["tokens"]), "ALIAS"),
    (dict(ws=ADDR["history"]), "ALIAS"), (dict(ws=None), "SCRATCH"),
    (dict(wsb=(64 << 10) - 1), "SCRATCH")] +
    [(dict([(n, ADDR["out"])]), "ALIAS") for n in
     ("history", "history_offsets", "prompt", "repetition", "presence", "frequency", "bias_ids",
      "bias", "bias_offsets", "masks", "mask_ids")])
def test_logits_refuses(L, kw, want):
    assert logits(L, **kw) == getattr(rq, "RQ_ERR_" + want)


# ---------------------------------------------------------------- binding
def test_the_binding_refuses_types_shapes_and_host_tensors():
    f, h, i = torch.float32, torch.float16, torch.int32
    z = lambda *s, dtype=f: torch.zeros(s, dtype=dtype)  # noqa: E731
    off = z(3, dtype=i)
    calls = [
        lambda: rq.rq_shift(z(4, 64), z(2, 64, dtype=h), z(2, 64, dtype=h), z(2, 4, 64, dtype=h), off),
        lambda: rq.rq_shift(z(4, 64, dtype=h), z(2, 32, dtype=h), z(2, 64, dtype=h),
                            z(2, 4, 64, dtype=h), off),
        lambda: rq.rq_shift(z(4, 64, dtype=h), z(2, 64, dtype=h), z(2, 64, dtype=h),
                            z(2, 5, 64, dtype=h), off),
        lambda: rq.rq_shift(z(4, 64, dtype=h), z(2, 64, dtype=h), z(2, 64, dtype=h),
                            z(2, 4, 64, dtype=h), off.long()),
        lambda: rq.rq_shift(z(4, 64, dtype=h), z(2, 64, dtype=h), z(2, 64, dtype=h),
                            z(2, 4, 64, dtype=h), off, z(3, dtype=i)),
        lambda: rq.rq_wkv7(*[z(4, 96)] * 6, z(2, 1, 64, 64), z(4, 96), off),
        lambda: rq.rq_wkv7(*[z(4, 64)] * 5, z(4, 64, dtype=h), z(2, 1, 64, 64), z(4, 64), off),
        lambda: rq.rq_wkv7(*[z(4, 64)] * 6, z(2, 2, 64, 64), z(4, 64), off),
        lambda: rq.rq_wkv7(*[z(4, 64)] * 6, z(2, 1, 64, 64), z(4, 64, dtype=h), off),
        lambda: rq.rq_lora([(z(8, 64, dtype=h), z(512), z(2, 64, dtype=h), None, z(2, 64), 64, 64)],
                           z(2, dtype=i), z(2, dtype=i), None, 8),
        lambda: rq.rq_lora([(z(8, 64, dtype=h), z(500, dtype=h), z(2, 64, dtype=h), None, z(2, 64),
                             64, 64)], z(2, dtype=i), z(2, dtype=i), None, 8),
        lambda: rq.rq_lora([(z(8, 64, dtype=h), z(512, dtype=h), z(2, 64, dtype=h), None, z(2, 64),
                             64, 64)], z(2, dtype=i), z(2, dtype=i), z(2), 8),
        lambda: rq.rq_logits(z(2, 100, dtype=h), z(2, 100)),
        lambda: rq.rq_logits(z(2, 100), z(2, 99)),
        lambda: rq.rq_logits(z(2, 100), z(2, 100), z(2)),
        lambda: rq.rq_logits(z(2, 100), z(2, 100), masks=(z(1, 3, dtype=i), z(2, dtype=i))),
        # right in every way but on the host
        lambda: rq.rq_shift(z(4, 64, dtype=h), z(2, 64, dtype=h), z(2, 64, dtype=h),
                            z(2, 4, 64, dtype=h), off),
        lambda: rq.rq_wkv7(*[z(4, 64)] * 6, z(2, 1, 64, 64), z(4, 64), off),
        lambda: rq.rq_lora([(z(8, 64, dtype=h), z(512, dtype=h), z(2, 64, dtype=h), None, z(2, 64),
                             64, 64)], z(2, dtype=i), z(2, dtype=i), None, 8),
        lambda: rq.rq_logits(z(2, 100), z(2, 100)),
    ]
    for k, c in enumerate(calls):
        with pytest.raises(ValueError):
            c()
            pytest.fail(f"call {k} was accepted")
    with pytest.raises(TypeError):
        rq.prepare("rq_gemv", 1, bias=None)


# ------------------------------------------------- sizes the kernels' indexes allow
def test_sizes_past_the_limits_are_refused(L):
    src = open(os.path.join(ROOT, "include", "rq.h")).read()
    assert re.search(r"#define RQ_MAX_TOKENS \(1 << 24\)", src) and rq.RQ_MAX_TOKENS == 1 << 24
    big = 1 << 24
    far = dict(out=A + 400 * G, state=None, nslots=0)
    assert shift(L, T=big + 1, D=8, **far) == rq.RQ_ERR_SHAPE
    assert shift(L, D=big + 8, T=1, **far) == rq.RQ_ERR_SHAPE
    assert wkv(L, T=big + 1, y=A + 9000 * G, state=None, nslots=0) == rq.RQ_ERR_SHAPE
    assert wkv(L, seqs=1025, H=4096, state=None, nslots=0) == rq.RQ_ERR_SHAPE
    assert lora(L, (dict(N=big + 1),)) == rq.RQ_ERR_SHAPE
    assert lora(L, (dict(K=big + 8),)) == rq.RQ_ERR_SHAPE
    assert logits(L, V=G + 1) == rq.RQ_ERR_SHAPE
    assert logits(L, history_len=G + 1) == rq.RQ_ERR_SHAPE
    assert logits(L, bias_len=G + 1) == rq.RQ_ERR_SHAPE


@no_gpu
def test_sizes_at_the_limits_are_accepted(L):
    big = 1 << 24
    apart = {n: A + (i + 1) * 4096 * G for i, n in enumerate(("x", "mu", "out"))}
    assert passes(shift(L, T=big, D=8, state=None, nslots=0, **apart))
    assert passes(shift(L, T=1, D=big, state=None, nslots=0, **apart))
    apart = {n: A + i * 65536 * G for i, n in enumerate(WKV) if n not in
             ("type", "T", "H", "seqs", "nslots", "state")}
    assert passes(wkv(L, T=big, H=1, state=None, nslots=0, **apart))
    assert passes(wkv(L, T=1, H=4096, seqs=1024, state=None, nslots=0, **apart))
    spread = dict(logits=A + 500 * G, out=A + 100 * G, history=A + 200 * G, masks=A + 300 * G)
    assert passes(logits(L, M=1, V=G, history_len=G, bias_ids=None, bias=None, **spread))
