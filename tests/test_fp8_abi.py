"""What rq_quant_fp8, rq_gemm_fp8 and rq_groupnorm refuse, on the CPU: every check
runs on the host before any HIP call, so the addresses are never dereferenced.
A call that passes all checks ends with RQ_ERR_DEVICE where there is no GPU."""
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


no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="the accepted calls would run on made-up addresses")


def err(want):
    return getattr(rq, "RQ_ERR_" + want)


def test_limits_match_the_header():
    src = open(os.path.join(ROOT, "include", "rq.h")).read()
    for n in ("RQ_TYPE_F32", "RQ_TYPE_F16", "RQ_TYPE_E4M3", "RQ_SCALE_F32", "RQ_SCALE_E8M0",
              "RQ_ACT_NONE", "RQ_ACT_RELU2", "RQ_ACT_SILU"):
        assert getattr(rq, n) == int(re.search(rf"\b{n} = (\d+)", src).group(1)), n
    assert rq.RQ_FP8_BLOCK == int(re.search(r"#define RQ_FP8_BLOCK (\d+)", src).group(1))
    assert rq.RQ_FP8_MAX_BATCH == int(re.search(r"#define RQ_FP8_MAX_BATCH (\d+)", src).group(1))
    assert re.search(r"RQ_FP8_MAX_K \(1 << 22\)", src) and rq.RQ_FP8_MAX_K == 1 << 22
    assert re.search(r"RQ_FP8_MAX_VALUES \(1ll << 34\)", src) and rq.RQ_FP8_MAX_VALUES == 1 << 34


# ------------------------------------------------------------------ quant
def quant(L, **kw):
    a = dict(x=A, type=0, act=0, q=A + 8 * G, s=A + 16 * G, kind=0, M=10, K=256)
    a.update(kw)
    return L.rq_quant_fp8(*[a[k] for k in ("x", "type", "act", "q", "s", "kind", "M", "K")], None)


@no_gpu
@pytest.mark.parametrize("kw", [{}, dict(type=1), dict(act=1), dict(kind=1), dict(K=128, M=1),
                                dict(s=A + 16 * G + 4), dict(kind=1, s=A + 16 * G + 1),
                                dict(M=1 << 12, K=1 << 22, q=A + 64 * G, s=A + 128 * G)])
def test_quant_accepts(L, kw):
    assert quant(L, **kw) == rq.RQ_ERR_DEVICE


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), "NULL"), (dict(q=None), "NULL"), (dict(s=None), "NULL"),
    (dict(type=2), "UNSUPPORTED"), (dict(type=-1), "UNSUPPORTED"), (dict(act=2), "UNSUPPORTED"),
    (dict(act=-1), "UNSUPPORTED"), (dict(kind=2), "UNSUPPORTED"),
    (dict(M=0), "SHAPE"), (dict(M=-1), "SHAPE"), (dict(M=(1 << 24) + 1), "SHAPE"),
    (dict(K=0), "SHAPE"), (dict(K=64), "SHAPE"), (dict(K=129), "SHAPE"), (dict(K=-128), "SHAPE"),
    (dict(K=(1 << 22) + 128), "SHAPE"), (dict(M=(1 << 12) + 1, K=1 << 22), "SHAPE"),
    (dict(x=A + 8), "ALIGN"), (dict(q=A + 8 * G + 4), "ALIGN"), (dict(s=A + 16 * G + 2), "ALIGN"),
    (dict(q=A), "ALIAS"), (dict(q=A + 10 * 256 * 4 - 16), "ALIAS"), (dict(s=A), "ALIAS"),
    (dict(s=A + 8 * G + 2556), "ALIAS"), (dict(x=A + 8 * G + 2544), "ALIAS"),
])
def test_quant_refuses(L, kw, want):
    assert quant(L, **kw) == err(want)


# ------------------------------------------------------------------- gemm
def gemm(L, count=1, M=10, kind=0, out=0, act=0, ws=None, ws_bytes=0, size=False, first=None,
         **kw):
    """`count` problems 64 GiB apart; kw changes the last one, first the first."""
    arr = (rq.RqFp8Problem * max(count, 1))()
    for i in range(max(count, 1)):
        a = dict(w=A, w_scales=A + 8 * G, x=A + 16 * G, x_scales=A + 24 * G, y_in=0, y=A + 32 * G,
                 y_scales=A + 40 * G if out == 2 else 0, N=256, K=384)
        a = {k: v + i * 64 * G if k not in "NK" and v else v for k, v in a.items()}
        if i == max(count, 1) - 1:
            a.update(kw)
        if i == 0 and first:
            a.update(first)
        for k, v in a.items():
            setattr(arr[i], k, v if k in "NK" else (v or None))
    if size:
        b = ctypes.c_size_t(7)
        return L.rq_gemm_fp8_workspace_size(arr, count, M, kind, out, ctypes.byref(b)), b.value
    return L.rq_gemm_fp8(arr, count, M, kind, out, act, ws, ws_bytes, None)


W = dict(ws=A + 600 * G, ws_bytes=64 << 20)


@no_gpu
@pytest.mark.parametrize("kw", [
    {}, W, dict(count=8), dict(out=1), dict(out=2), dict(out=2, act=1), dict(kind=1),
    dict(y_in=A + 32 * G), dict(y_in=A + 48 * G), dict(N=1), dict(N=257), dict(K=128),
    dict(M=1 << 24, x=A + 1000 * G, x_scales=A + 1100 * G, y=A + 1200 * G), dict(w_scales=A + 8 * G + 4),
    dict(kind=1, x_scales=A + 24 * G + 3), dict(count=3, K=128), dict(M=1, K=16384, **W),
    dict(M=32, N=4096, K=16384, **W), dict(M=64, **W), dict(M=300, **W)])
def test_gemm_accepts(L, kw):
    assert gemm(L, **kw) == rq.RQ_ERR_DEVICE


@pytest.mark.parametrize("kw,want", [
    (dict(w=0), "NULL"), (dict(w_scales=0), "NULL"), (dict(x=0), "NULL"), (dict(x_scales=0), "NULL"),
    (dict(y=0), "NULL"), (dict(out=2, y_scales=0), "NULL"),
    (dict(count=0), "SHAPE"), (dict(count=9), "SHAPE"), (dict(M=0), "SHAPE"),
    (dict(M=(1 << 24) + 1), "SHAPE"), (dict(N=0), "SHAPE"), (dict(N=(1 << 24) + 1), "SHAPE"),
    (dict(K=0), "SHAPE"), (dict(K=64), "SHAPE"), (dict(K=192), "SHAPE"),
    (dict(K=(1 << 22) + 128), "SHAPE"), (dict(M=1 << 20, N=(1 << 14) + 1), "SHAPE"),
    (dict(out=2, N=130), "SHAPE"), (dict(count=3, K=100), "SHAPE"),
    (dict(out=3), "UNSUPPORTED"), (dict(kind=2), "UNSUPPORTED"), (dict(act=1), "UNSUPPORTED"),
    (dict(out=1, act=1), "UNSUPPORTED"), (dict(out=2, act=2), "UNSUPPORTED"),
    (dict(out=1, y_in=A + 48 * G), "UNSUPPORTED"), (dict(out=2, y_in=A + 48 * G), "UNSUPPORTED"),
    (dict(w=A + 8), "ALIGN"), (dict(x=A + 16 * G + 4), "ALIGN"), (dict(y=A + 32 * G + 8), "ALIGN"),
    (dict(y_in=A + 48 * G + 4), "ALIGN"), (dict(x_scales=A + 24 * G + 2), "ALIGN"),
    (dict(ws=A + 600 * G + 8, ws_bytes=64 << 20), "ALIGN"),
    (dict(y=A), "ALIAS"), (dict(y=A + 8 * G), "ALIAS"), (dict(y=A + 16 * G), "ALIAS"),
    (dict(y=A + 24 * G), "ALIAS"), (dict(y_in=A + 32 * G + 16), "ALIAS"),
    (dict(out=2, y_scales=A + 32 * G), "ALIAS"), (dict(out=2, y_scales=A), "ALIAS"),
    (dict(count=2, y=A + 32 * G), "ALIAS"), (dict(count=2, w=A + 32 * G), "ALIAS"),
    (dict(count=2, first=dict(y=A + 64 * G)), "ALIAS"),
    (dict(count=2, y_in=A + 32 * G), "ALIAS"),
])
def test_gemm_refuses(L, kw, want):
    assert gemm(L, **kw) == err(want)


def test_gemm_workspace(L):
    """The size that is reported is the size that is asked for, checked against the
    operands, and at most RQ_GEMM_WORKSPACE_MAX_BYTES."""
    split = 0
    for M in (1, 7, 16, 17, 32, 33, 61, 64, 100, 128, 200, 256, 300, 600, 2000):
        for N, K in ((128, 128), (768, 768), (4096, 4096), (2560, 10240), (4096, 16384),
                     (16384, 4096), (65529, 2048), (1, 1 << 22), (1 << 20, 128)):
            for out in (0, 1, 2):
                if out == 2 and N % 128:
                    continue
                st, need = gemm(L, M=M, N=N, K=K, out=out, size=True)
                assert st == rq.RQ_OK and 0 <= need <= rq.RQ_GEMM_WORKSPACE_MAX_BYTES
                if not need:
                    continue
                split += 1
                wide = dict(M=M, N=N, K=K, out=out, x=A + 700 * G, y=A + 800 * G, w=A + 900 * G,
                            w_scales=A + 950 * G, x_scales=A + 970 * G)
                if out == 2:
                    wide["y_scales"] = A + 990 * G
                assert gemm(L, ws=A + 600 * G, ws_bytes=need - 1, **wide) == rq.RQ_ERR_SCRATCH
                for k in ("x", "y", "w", "x_scales"):
                    bad = dict(wide, ws=wide[k] - need + 16, ws_bytes=need)
                    assert gemm(L, **bad) == rq.RQ_ERR_ALIAS, k
                if not torch.cuda.is_available():
                    assert gemm(L, ws=A + 600 * G, ws_bytes=need, **wide) == rq.RQ_ERR_DEVICE
    for kw, want in ((dict(count=0), "SHAPE"), (dict(K=64), "SHAPE"), (dict(out=5), "UNSUPPORTED"),
                     (dict(kind=9), "UNSUPPORTED")):
        st, need = gemm(L, size=True, **kw)
        assert st == err(want) and need == 0
    assert L.rq_gemm_fp8_workspace_size(None, 1, 1, 0, 0,
                                        ctypes.byref(ctypes.c_size_t())) == rq.RQ_ERR_NULL
    assert L.rq_gemm_fp8_workspace_size((rq.RqFp8Problem * 1)(), 1, 1, 0, 0, None) == rq.RQ_ERR_NULL
    assert L.rq_gemm_fp8(None, 1, 1, 0, 0, 0, None, 0, None) == rq.RQ_ERR_NULL


# ------------------------------------------------------------------- norm
def norm(L, **kw):
    a = dict(y=A, weight=A + 8 * G, bias=A + 9 * G, r=A + 10 * G, k=A + 20 * G, r_k=A + 30 * G,
             v=A + 40 * G, gate=A + 50 * G, out=A + 60 * G, out_scales=A + 70 * G, input_type=0,
             act=0, out_type=0, scale_type=0, T=10, C=512, groups=8, eps=1e-5)
    a.update(kw)
    g = rq.RqGroupnormArgs(**{k: (v or None) if isinstance(v, int) and k in (
        "y", "weight", "bias", "r", "k", "r_k", "v", "gate", "out", "out_scales") else v
        for k, v in a.items()})
    return L.rq_groupnorm(ctypes.byref(g), None)


@no_gpu
@pytest.mark.parametrize("kw", [
    {}, dict(weight=0), dict(bias=0), dict(gate=0), dict(r=0, k=0, r_k=0, v=0), dict(r=0, k=3),
    dict(out=A), dict(out_type=1), dict(out_type=2), dict(out_type=2, scale_type=1),
    dict(input_type=1), dict(act=2), dict(C=32, groups=1), dict(C=96, groups=3),
    dict(C=512, groups=2), dict(C=512, groups=16), dict(eps=0.0), dict(scale_type=9),
    dict(out_type=2, out_scales=A + 70 * G + 4), dict(T=1 << 24, C=1024, groups=8, y=A + 500 * G,
                                                      r=A + 700 * G, k=A + 900 * G, v=A + 1100 * G,
                                                      gate=A + 1300 * G, out=A + 1500 * G)])
def test_norm_accepts(L, kw):
    assert norm(L, **kw) == rq.RQ_ERR_DEVICE


@pytest.mark.parametrize("kw,want", [
    (dict(y=0), "NULL"), (dict(out=0), "NULL"), (dict(k=0), "NULL"), (dict(r_k=0), "NULL"),
    (dict(v=0), "NULL"), (dict(out_type=2, out_scales=0), "NULL"),
    (dict(input_type=2), "UNSUPPORTED"), (dict(act=1), "UNSUPPORTED"), (dict(act=3), "UNSUPPORTED"),
    (dict(out_type=3), "UNSUPPORTED"), (dict(out_type=2, scale_type=2), "UNSUPPORTED"),
    (dict(T=0), "SHAPE"), (dict(T=(1 << 24) + 1), "SHAPE"), (dict(C=0), "SHAPE"),
    (dict(groups=0), "SHAPE"), (dict(groups=-8), "SHAPE"), (dict(groups=7), "SHAPE"),
    (dict(groups=1), "SHAPE"), (dict(groups=32), "SHAPE"), (dict(C=(1 << 20) + 64, groups=16385), "SHAPE"),
    (dict(C=192, groups=3, out_type=2), "SHAPE"), (dict(T=1 << 24, C=2048, groups=8), "SHAPE"),
    (dict(eps=-1e-5), "SHAPE"), (dict(eps=float("nan")), "SHAPE"), (dict(eps=float("inf")), "SHAPE"),
    (dict(y=A + 4), "ALIGN"), (dict(weight=A + 8 * G + 4), "ALIGN"), (dict(r=A + 10 * G + 8), "ALIGN"),
    (dict(gate=A + 50 * G + 2), "ALIGN"), (dict(out=A + 60 * G + 8), "ALIGN"),
    (dict(out_type=2, out_scales=A + 70 * G + 2), "ALIGN"),
    (dict(out=A + 16), "ALIAS"), (dict(out=A, out_type=1), "ALIAS"), (dict(out=A + 8 * G), "ALIAS"),
    (dict(out=A + 10 * G), "ALIAS"), (dict(out=A + 30 * G), "ALIAS"), (dict(out=A + 50 * G), "ALIAS"),
    (dict(out_type=2, out_scales=A + 60 * G), "ALIAS"), (dict(out_type=2, out_scales=A), "ALIAS"),
])
def test_norm_refuses(L, kw, want):
    assert norm(L, **kw) == err(want)


def test_norm_without_arguments(L):
    assert L.rq_groupnorm(None, None) == rq.RQ_ERR_NULL


# ---------------------------------------------------------------- binding
def test_the_binding_checks_types_and_shapes():
    f, e4, e8 = torch.zeros, torch.float8_e4m3fn, torch.float8_e8m0fnu

    def z(shape, dtype=torch.float32):
        return f(shape, dtype=torch.uint8).view(dtype) if dtype in (e4, e8) else f(shape, dtype=dtype)
    x, q, s = z((4, 256)), z((4, 256), e4), z((4, 2), e8)
    bad = [lambda: rq.rq_quant_fp8(x, q, s),                                  # not on the GPU
           lambda: rq.rq_quant_fp8(x.double(), q, s), lambda: rq.rq_quant_fp8(x, x, s),
           lambda: rq.rq_quant_fp8(x, q, z((4, 2), torch.float16)),
           lambda: rq.rq_quant_fp8(x, q, z((4, 3))), lambda: rq.rq_quant_fp8(z((4, 100)), q, s)]
    w, ws, y = z((130, 256), e4), z((2, 2), e8), z((4, 130))

    def gemm(w=w, ws=ws, x=q, xs=s, y_in=None, y=y, N=130, K=256):
        return rq.rq_gemm_fp8([(w, ws, x, xs, y_in, y, N, K)])
    bad += [gemm, lambda: gemm(N=129), lambda: gemm(K=128), lambda: gemm(K=200),
            lambda: gemm(xs=z((4, 2))), lambda: gemm(ws=z((1, 2), e8)), lambda: gemm(w=z((130, 256))),
            lambda: gemm(y=z((4, 130), torch.bfloat16)), lambda: gemm(y=(z((4, 130), e4), s)),
            lambda: gemm(y_in=z((4, 130), torch.float16)),
            lambda: rq.rq_gemm_fp8([(w, ws, q, s, None, y, 130, 256),
                                    (w, ws, q, s, None, y.half(), 130, 256)])]
    t, c = z((4, 256)), z(256)

    def norm(y=t, g=4, weight=c, bias=c, out=t, **kw):
        return rq.rq_groupnorm(y, g, weight, bias, 1e-5, out, **kw)
    bad += [norm, lambda: norm(weight=z(255)), lambda: norm(y=t.half()), lambda: norm(out=t.double()),
            lambda: norm(gate=t.bfloat16()), lambda: norm(bonus=(t, t.half(), c, t)),
            lambda: norm(bonus=(t, t, c, t), gate=t.half()), lambda: norm(out=(q, z((4, 3), e8)))]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            print(i)
