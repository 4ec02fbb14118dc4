"""Python binding of librq (include/rq.h): group-wise low-bit weight
dequantization and dequantize-and-multiply on MI355X (gfx950).

Argument marshalling only.  Every computation runs in the HIP kernels of
``librq.so``; there is no CPU fallback.  If the library is missing, every call
raises ``RqLibraryMissing`` (build it with ``python gemm_rwkv_decode_amd/build.py``
or ``__graft_entry__.build()``).

Tensors are torch tensors on the GPU, contiguous:

* ``qweight``: uint8 ``[N][K/2]`` (4-bit) or int8 ``[N][K]`` (8-bit);
* ``scales``: float16 ``[N][K/group]`` (symmetric) or uint8 ``[N][K/256][8]``
  superblock records (asymmetric); ``zeros``: ``None`` (symmetric) or uint8
  records (asymmetric);
* ``x``: float16 ``[M][K]``; ``y``: float32 ``[M][N]``.

Around the products (``rq_shift``, ``rq_lora``, ``rq_wkv7``, ``rq_logits``,
``rq_groupnorm``) sizes are read from the tensors, whose types and shapes are
checked here; index tensors are int32 on the GPU.  So are those of the
block-scaled FP8 calls (``rq_quant_fp8``, ``rq_gemm_fp8``): E4M3 values are
float8_e4m3fn or uint8 tensors, scales float32, float8_e8m0fnu or uint8 (E8M0).

Work is enqueued on torch's current stream (or the ``stream`` given).
"""
import ctypes
import os
import threading

__all__ = [
    "RQ_OK", "RQ_LAYOUT_SYM", "RQ_LAYOUT_ASYM_SB", "RQ_LAYOUT_FP8_TENSOR", "RQ_OUT_F32",
    "RQ_OUT_CODES_I8",
    "RQ_MAX_M", "RQ_MAX_BATCH", "RqError", "RqLibraryMissing", "rq_dequant", "rq_gemv",
    "rq_gemv_batched", "rq_gemm_smallm", "rq_gemm_smallm_ws", "rq_gemm_smallm_workspace_size",
    "rq_gemm_smallm_noalloc", "rq_shift", "rq_lora", "rq_lora_workspace_size", "rq_wkv7",
    "rq_logits", "rq_quant_fp8", "rq_gemm_fp8", "rq_gemm_fp8_workspace_size", "rq_groupnorm",
    "RQ_ACT_NONE", "RQ_ACT_RELU2", "RQ_ACT_SILU", "rq_status_string", "rq_version", "prepare",
    "gemm_workspace", "lib", "LIB_PATH",
]

RQ_OK = 0
RQ_ERR_NULL, RQ_ERR_SHAPE, RQ_ERR_UNSUPPORTED, RQ_ERR_ALIGN = 1, 2, 3, 4
RQ_ERR_LAUNCH, RQ_ERR_ALIAS, RQ_ERR_DEVICE, RQ_ERR_SCRATCH = 5, 6, 7, 8
RQ_NOALLOC_SCRATCH_BYTES = (8 << 20) + (64 << 10)
RQ_GEMM_WORKSPACE_MAX_BYTES = 64 << 20
RQ_LAYOUT_SYM, RQ_LAYOUT_ASYM_SB, RQ_LAYOUT_FP8_TENSOR = 0, 1, 2
RQ_OUT_F32, RQ_OUT_CODES_I8 = 0, 1
RQ_MAX_M = 64
RQ_MAX_BATCH = 64
RQ_MAX_SEQUENCES = 65536
RQ_MAX_TOKENS = 1 << 24
RQ_SHIFT_MAX_MIXES = 8
RQ_WKV_HEAD = 64
RQ_TYPE_F32, RQ_TYPE_F16, RQ_TYPE_E4M3 = 0, 1, 2
RQ_SCALE_F32, RQ_SCALE_E8M0 = 0, 1
RQ_ACT_NONE, RQ_ACT_RELU2, RQ_ACT_SILU = 0, 1, 2
RQ_FP8_BLOCK, RQ_FP8_MAX_K, RQ_FP8_MAX_BATCH = 128, 1 << 22, 8
RQ_FP8_MAX_VALUES = 1 << 34
RQ_LORA_MAX_M, RQ_LORA_MAX_RANK, RQ_LORA_MAX_BATCH = 8192, 128, 8
RQ_LOGITS_MAX_M = 4096
RQ_LOGITS_WORKSPACE_BYTES = 64 << 10

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librq.so")
_lib = None
_lock = threading.Lock()


class RqProblem(ctypes.Structure):
    """rq_problem of include/rq.h."""
    _fields_ = [("qweight", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("N", ctypes.c_int), ("K", ctypes.c_int)]


class RqLoraProblem(ctypes.Structure):
    """rq_lora_problem of include/rq.h."""
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("y_in", ctypes.c_void_p), ("y", ctypes.c_void_p), ("N", ctypes.c_int),
                ("K", ctypes.c_int)]


class RqLogitsArgs(ctypes.Structure):
    """rq_logits_args of include/rq.h."""
    _fields_ = [("logits", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("tokens", ctypes.c_void_p), ("M", ctypes.c_int), ("V", ctypes.c_int),
                ("history", ctypes.c_void_p), ("history_offsets", ctypes.c_void_p),
                ("prompt", ctypes.c_void_p), ("history_len", ctypes.c_int),
                ("repetition", ctypes.c_void_p), ("presence", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("bias_offsets", ctypes.c_void_p),
                ("bias_len", ctypes.c_int), ("masks", ctypes.c_void_p),
                ("mask_ids", ctypes.c_void_p), ("nmasks", ctypes.c_int)]


class RqFp8Problem(ctypes.Structure):
    """rq_fp8_problem of include/rq.h."""
    _fields_ = [("w", ctypes.c_void_p), ("w_scales", ctypes.c_void_p), ("x", ctypes.c_void_p),
                ("x_scales", ctypes.c_void_p), ("y_in", ctypes.c_void_p),
                ("y", ctypes.c_void_p), ("y_scales", ctypes.c_void_p), ("N", ctypes.c_int),
                ("K", ctypes.c_int)]


class RqGroupnormArgs(ctypes.Structure):
    """rq_groupnorm_args of include/rq.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("y", "weight", "bias", "r", "k", "r_k", "v", "gate",
                                               "out", "out_scales")] + \
               [(n, ctypes.c_int) for n in ("input_type", "act", "out_type", "scale_type", "T",
                                            "C", "groups")] + [("eps", ctypes.c_float)]


class RqLibraryMissing(RuntimeError):
    pass


class RqError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: status {status} ({rq_status_string(status)})")


def lib():
    """The loaded librq (ctypes), signatures declared."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RqLibraryMissing(
                    f"{LIB_PATH} not found: build it with gemm_rwkv_decode_amd/build.py")
            L = ctypes.CDLL(LIB_PATH)
            vp, i = ctypes.c_void_p, ctypes.c_int
            L.rq_dequant.argtypes = [vp, vp, vp, vp, i, i, i, i, i, i, vp]
            L.rq_dequant.restype = i
            for name in ("rq_gemv", "rq_gemm_smallm", "rq_gemm_smallm_noalloc"):
                f = getattr(L, name)
                f.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
                f.restype = i
            L.rq_gemm_smallm_ws.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp,
                                            ctypes.c_size_t, vp]
            L.rq_gemm_smallm_ws.restype = i
            L.rq_gemm_smallm_workspace_size.argtypes = [i, i, i, i, i, i,
                                                        ctypes.POINTER(ctypes.c_size_t)]
            L.rq_gemm_smallm_workspace_size.restype = i
            L.rq_gemv_batched.argtypes = [ctypes.POINTER(RqProblem), i, i, i, i, i, vp]
            L.rq_gemv_batched.restype = i
            L.rq_shift.argtypes = [vp] * 6 + [i] * 5 + [vp]
            L.rq_shift.restype = i
            L.rq_wkv7.argtypes = [vp] * 6 + [i] + [vp] * 4 + [i] * 4 + [vp]
            L.rq_wkv7.restype = i
            L.rq_lora.argtypes = [ctypes.POINTER(RqLoraProblem), i, i, vp, vp, vp, i, i, i, vp,
                                  ctypes.c_size_t, vp]
            L.rq_lora.restype = i
            L.rq_lora_workspace_size.argtypes = [ctypes.POINTER(RqLoraProblem), i, i, i, i,
                                                 ctypes.POINTER(ctypes.c_size_t)]
            L.rq_lora_workspace_size.restype = i
            L.rq_logits.argtypes = [ctypes.POINTER(RqLogitsArgs), vp, ctypes.c_size_t, vp]
            L.rq_logits.restype = i
            L.rq_quant_fp8.argtypes = [vp, i, i, vp, vp, i, i, i, vp]
            L.rq_quant_fp8.restype = i
            L.rq_gemm_fp8.argtypes = [ctypes.POINTER(RqFp8Problem), i, i, i, i, i, vp,
                                      ctypes.c_size_t, vp]
            L.rq_gemm_fp8.restype = i
            L.rq_gemm_fp8_workspace_size.argtypes = [ctypes.POINTER(RqFp8Problem), i, i, i, i,
                                                     ctypes.POINTER(ctypes.c_size_t)]
            L.rq_gemm_fp8_workspace_size.restype = i
            L.rq_groupnorm.argtypes = [ctypes.POINTER(RqGroupnormArgs), vp]
            L.rq_groupnorm.restype = i
            L.rq_status_string.argtypes = [i]
            L.rq_status_string.restype = ctypes.c_char_p
            L.rq_version.argtypes = []
            L.rq_version.restype = i
            # measurement kernels (include/rq_probe.h)
            L.rq_probe_read.argtypes = [vp, ctypes.c_size_t, vp, i, i, vp]
            L.rq_probe_read.restype = i
            L.rq_probe_copy.argtypes = [vp, vp, ctypes.c_size_t, vp]
            L.rq_probe_copy.restype = i
            L.rq_probe_empty.argtypes = [vp]
            L.rq_probe_empty.restype = i
            L.rq_probe_signal.argtypes = [vp, i, i, vp]
            L.rq_probe_signal.restype = i
            L.rq_probe_barrier.argtypes = [vp, i, i, i, i, vp, vp]
            L.rq_probe_barrier.restype = i
            L.rq_probe_mfma.argtypes = [i, i, i, vp, vp]
            L.rq_probe_mfma.restype = i
            L.rq_probe_valu.argtypes = [i, i, i, vp, vp]
            L.rq_probe_valu.restype = i
            L.rq_probe_overlap.argtypes = [i, i, i, i, i, vp, vp]
            L.rq_probe_overlap.restype = i
            L.rq_tuning_reload.argtypes = []
            L.rq_tuning_reload.restype = i
            ip = ctypes.POINTER(ctypes.c_int)
            L.rq_gemm_config.argtypes = [i, i, i, i, i, i, i, ip, ip]
            L.rq_gemm_config.restype = i
            L.rq_gemv_config.argtypes = [i, i, i, i, i, i, ip, ip, ip, ip]
            L.rq_gemv_config.restype = i
            _lib = L
    return _lib


def rq_status_string(status: int) -> str:
    return lib().rq_status_string(int(status)).decode()


def rq_version() -> int:
    return lib().rq_version()


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("librq takes GPU tensors only")
    if not t.is_contiguous():
        raise ValueError("librq takes contiguous tensors only")
    return t.data_ptr()


def _stream(stream, like):
    if stream is not None:
        return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
    import torch
    return int(torch.cuda.current_stream(like.device).cuda_stream)


def rq_dequant(qweight, scales, zeros, out, N, K, bits, group, layout,
               out_kind=RQ_OUT_F32, stream=None):
    """Unpack (out_kind RQ_OUT_CODES_I8, out int8 [N][K]) or dequantize
    (RQ_OUT_F32, out float32 [N][K]) the packed weights."""
    st = lib().rq_dequant(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(out), int(N),
                          int(K), int(bits), int(group), int(layout), int(out_kind),
                          _stream(stream, qweight))
    if st != RQ_OK:
        raise RqError("rq_dequant", st)
    return out


def rq_gemv(qweight, scales, zeros, x, y, M, N, K, bits, group, layout, stream=None):
    """y[m][n] = sum_k x[m][k] w[n][k]; the kernel is chosen for M (vector units
    at M <= 2, matrix cores from M = 3 on), K is never split, nothing is
    allocated."""
    st = lib().rq_gemv(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), int(M),
                       int(N), int(K), int(bits), int(group), int(layout),
                       _stream(stream, qweight))
    if st != RQ_OK:
        raise RqError("rq_gemv", st)
    return y


# Sentinel: the binding's own split-K workspace for the call's stream.
AUTO = "auto"
_workspaces = {}  # (device index, stream handle) -> int32 tensor


def gemm_workspace(stream=None, device=None):
    """The binding's split-K workspace for one stream: a torch tensor of
    RQ_GEMM_WORKSPACE_MAX_BYTES whose arrival counters are zeroed on that
    stream, made by the first call on the stream and kept for the process (the
    library never allocates; PyTorch owns this memory).  None while that
    stream is being captured into a graph and has no workspace yet: the call
    then keeps K whole."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    dev = torch.device(dev)
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    if stream is None:
        h = int(torch.cuda.current_stream(dev).cuda_stream)
    else:
        h = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
    key = (dev.index, h)
    with _lock:
        ws = _workspaces.get(key)
        if ws is not None:
            return ws
        if torch.cuda.is_current_stream_capturing():
            return None
        cur = torch.cuda.current_stream(dev)
        st = cur if int(cur.cuda_stream) == h else torch.cuda.ExternalStream(h, device=dev)
        with torch.cuda.device(dev), torch.cuda.stream(st):
            ws = torch.zeros(RQ_GEMM_WORKSPACE_MAX_BYTES // 4, dtype=torch.int32, device=dev)
        _workspaces[key] = ws
        return ws


def _ws_args(workspace, stream, like):
    """(pointer, bytes) of a workspace argument: AUTO, None or a tensor."""
    if isinstance(workspace, str) and workspace == AUTO:
        workspace = gemm_workspace(stream, like.device)
    if workspace is None:
        return None, 0
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def rq_gemm_smallm(qweight, scales, zeros, x, y, M, N, K, bits, group, layout,
                   stream=None, workspace=AUTO):
    """Same product on the matrix cores (tuned for 16 <= M <= 64).

    ``workspace``: AUTO (default) passes the binding's workspace for the
    stream to rq_gemm_smallm_ws, so K may be split; a tensor passes that one;
    None calls rq_gemm_smallm, which keeps K whole."""
    if workspace is None:
        st = lib().rq_gemm_smallm(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y),
                                  int(M), int(N), int(K), int(bits), int(group), int(layout),
                                  _stream(stream, qweight))
        if st != RQ_OK:
            raise RqError("rq_gemm_smallm", st)
        return y
    return rq_gemm_smallm_ws(qweight, scales, zeros, x, y, M, N, K, bits, group, layout,
                             workspace, stream=stream)


def rq_gemm_smallm_ws(qweight, scales, zeros, x, y, M, N, K, bits, group, layout, workspace,
                      stream=None):
    """rq_gemm_smallm with a caller-owned workspace (a tensor whose first 64 KiB
    are zero before first use, or AUTO, or None to keep K whole)."""
    L = lib()
    ptrs = (_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y))
    wp, wb = _ws_args(workspace, stream, qweight)
    st = L.rq_gemm_smallm_ws(*ptrs, int(M), int(N), int(K), int(bits), int(group), int(layout),
                             wp, wb, _stream(stream, qweight))
    if st != RQ_OK:
        raise RqError("rq_gemm_smallm_ws", st)
    return y


def rq_gemm_smallm_workspace_size(M, N, K, bits, group, layout):
    """Bytes of workspace rq_gemm_smallm_ws uses for one product (0: K kept
    whole).  Host-only."""
    b = ctypes.c_size_t(0)
    st = lib().rq_gemm_smallm_workspace_size(int(M), int(N), int(K), int(bits), int(group),
                                             int(layout), ctypes.byref(b))
    if st != RQ_OK:
        raise RqError("rq_gemm_smallm_workspace_size", st)
    return b.value


def rq_gemm_smallm_noalloc(qweight, scales, zeros, x, y, M, N, K, bits, group, layout,
                           stream=None):
    """rq_gemm_smallm with its split-K partial sums in the library's fixed
    device array: never allocates; calls overlapping on one GPU race."""
    st = lib().rq_gemm_smallm_noalloc(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x),
                                      _ptr(y), int(M), int(N), int(K), int(bits), int(group),
                                      int(layout), _stream(stream, qweight))
    if st != RQ_OK:
        raise RqError("rq_gemm_smallm_noalloc", st)
    return y


def _problems(problems):
    arr = (RqProblem * len(problems))()
    for i, (qweight, scales, zeros, x, y, N, K) in enumerate(problems):
        arr[i] = RqProblem(_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y),
                           int(N), int(K))
    return arr


def rq_gemv_batched(problems, M, bits, group, layout, stream=None):
    """Independent products in as few launches as possible.  ``problems`` is a
    sequence of (qweight, scales, zeros, x, y, N, K); M, bits, group and layout
    are shared."""
    arr = _problems(problems)
    st = lib().rq_gemv_batched(arr, len(problems), int(M), int(bits), int(group),
                               int(layout), _stream(stream, problems[0][0]))
    if st != RQ_OK:
        raise RqError("rq_gemv_batched", st)


def _typed(what, t, dtype, shape):
    """Pointer of a tensor of this type and shape (None in a shape: any size);
    None for None."""
    if t is None:
        return None
    if str(t.dtype) != "torch." + dtype:
        raise ValueError(f"{what}: {dtype} expected, got {t.dtype}")
    if len(t.shape) != len(shape) or any(b is not None and a != b
                                         for a, b in zip(t.shape, shape)):
        raise ValueError(f"{what}: shape {shape} expected, got {tuple(t.shape)}")
    return _ptr(t)


def _batch_args(offsets, slots):
    """(pointer of offsets, pointer of slots, sequences)."""
    n = offsets.numel() - 1
    return (_typed("offsets", offsets, "int32", (n + 1,)), _typed("slots", slots, "int32", (n,)),
            n)


def _shift_cargs(x, mu, state, out, offsets, slots=None, *, stream=None):
    T, D = x.shape
    n = mu.shape[0]
    po, ps, seqs = _batch_args(offsets, slots)
    nslots = 0 if state is None else state.shape[0]
    return (_typed("x", x, "float16", (T, D)), _typed("mu", mu, "float16", (n, D)),
            _typed("state", state, "float16", (nslots, D)),
            _typed("out", out, "float16", (n, T, D)), po, ps, T, D, n, seqs, nslots,
            _stream(stream, x))


def rq_shift(x, mu, state, out, offsets, slots=None, stream=None):
    """Token shift: out[i][t] = x[t] + (prev[t] - x[t]) * mu[i] over a batch of
    sequences.  x float16 [T][D], mu float16 [n][D], state float16 [nslots][D]
    (read for a sequence's first token, then its last row; None: no sequence
    is stored), out float16 [n][T][D], offsets int32 [sequences + 1], slots
    int32 [sequences] or None."""
    st = lib().rq_shift(*_shift_cargs(x, mu, state, out, offsets, slots, stream=stream))
    if st != RQ_OK:
        raise RqError("rq_shift", st)
    return out


def _wkv7_cargs(r, w, k, v, kappa, eta, state, y, offsets, slots=None, *, stream=None):
    T, D = r.shape
    if D % RQ_WKV_HEAD:
        raise ValueError(f"r: whole heads of {RQ_WKV_HEAD} channels expected, got {D}")
    H = D // RQ_WKV_HEAD
    half = str(r.dtype) == "torch.float16"
    dt = "float16" if half else "float32"
    po, ps, seqs = _batch_args(offsets, slots)
    nslots = 0 if state is None else state.shape[0]
    ins = [_typed(n, t, dt, (T, D)) for n, t in (("r", r), ("w", w), ("k", k), ("v", v),
                                                 ("kappa", kappa), ("eta", eta))]
    return (*ins, RQ_TYPE_F16 if half else RQ_TYPE_F32,
            _typed("state", state, "float32", (nslots, H, RQ_WKV_HEAD, RQ_WKV_HEAD)),
            _typed("y", y, "float32", (T, D)), po, ps, T, H, seqs, nslots, _stream(stream, r))


def rq_wkv7(r, w, k, v, kappa, eta, state, y, offsets, slots=None, stream=None):
    """RWKV-7 state recurrence over a batch of sequences: per head of 64
    channels S = S diag(d) - (S kappa)(eta * kappa)^T + v k^T, y = S r, with
    d = exp(-exp(-1/2) sigmoid(w)).  Inputs [T][H*64], all float32 or all
    float16; state float32 [nslots][H][64][64], updated in place (None: no
    sequence is stored); y float32 [T][H*64]; offsets and slots as rq_shift."""
    st = lib().rq_wkv7(*_wkv7_cargs(r, w, k, v, kappa, eta, state, y, offsets, slots,
                                    stream=stream))
    if st != RQ_OK:
        raise RqError("rq_wkv7", st)
    return y


def _lora_problems(problems, M, total_rank):
    arr = (RqLoraProblem * len(problems))()
    for i, (a, b, x, y_in, y, N, K) in enumerate(problems):
        arr[i] = RqLoraProblem(_typed("a", a, "float16", (total_rank, K)),
                               _typed("b", b, "float16", (total_rank * N,)),
                               _typed("x", x, "float16", (M, K)),
                               _typed("y_in", y_in, "float32", (M, N)),
                               _typed("y", y, "float32", (M, N)), int(N), int(K))
    return arr


def _lora_ws(workspace, stream, like):
    """(pointer, bytes) of rq_lora's workspace; AUTO: the binding's workspace
    for the stream past its split-K arrival counters, which stay zero."""
    if isinstance(workspace, str) and workspace == AUTO:
        workspace = gemm_workspace(stream, like.device)
        if workspace is not None:
            workspace = workspace[RQ_LOGITS_WORKSPACE_BYTES // 4:]
    return _ws_args(workspace, stream, like)


def _lora_cargs(problems, ids, offsets, scales, max_rank, *, stream=None, workspace=AUTO):
    M, adapters = ids.numel(), offsets.numel() - 1
    total_rank = problems[0][0].shape[0]
    arr = _lora_problems(problems, M, total_rank)
    return (arr, len(problems), M, _typed("ids", ids, "int32", (M,)),
            _typed("offsets", offsets, "int32", (adapters + 1,)),
            _typed("scales", scales, "float32", (adapters,)), adapters, total_rank,
            int(max_rank), *_lora_ws(workspace, stream, ids), _stream(stream, ids))


def rq_lora(problems, ids, offsets, scales, max_rank, stream=None, workspace=AUTO):
    """Adapters of many requests beside shared projections: y[m] = y_in[m] +
    scales[i] * B_i (A_i x[m]) with i = ids[m] (no adapter outside 0 ..
    adapters-1), for every projection of ``problems``, a sequence of (a, b, x,
    y_in, y, N, K): a float16 [R][K] and b float16 [R * N] hold all adapters
    (adapter i: A rows offsets[i] .. offsets[i+1]-1, B block [N][r_i] at
    offsets[i] * N), y_in float32 [M][N] (y itself, another tensor, or None),
    y float32 [M][N].  ids int32 [M], offsets int32 [adapters + 1], scales
    float32 [adapters] or None.  ``workspace``: AUTO (the binding's, per
    stream) or a tensor of rq_lora_workspace_size bytes."""
    st = lib().rq_lora(*_lora_cargs(problems, ids, offsets, scales, max_rank, stream=stream,
                                    workspace=workspace))
    if st != RQ_OK:
        raise RqError("rq_lora", st)
    return [p[4] for p in problems]


def rq_lora_workspace_size(shapes, M, adapters, max_rank):
    """Bytes of workspace rq_lora uses for projections of these (N, K).
    Host-only."""
    arr = (RqLoraProblem * len(shapes))()
    for i, (N, K) in enumerate(shapes):
        arr[i].N, arr[i].K = int(N), int(K)
    b = ctypes.c_size_t(0)
    st = lib().rq_lora_workspace_size(arr, len(shapes), int(M), int(adapters), int(max_rank),
                                      ctypes.byref(b))
    if st != RQ_OK:
        raise RqError("rq_lora_workspace_size", st)
    return b.value


def _logits_cargs(logits, out, tokens=None, *, history=None, repetition=None, presence=None,
                  frequency=None, bias=None, masks=None, stream=None, workspace=AUTO):
    M, V = logits.shape
    a = RqLogitsArgs(logits=_typed("logits", logits, "float32", (M, V)),
                     out=_typed("out", out, "float32", (M, V)),
                     tokens=_typed("tokens", tokens, "int32", (M,)), M=M, V=V)
    if history is not None:
        toks, off, prompt = history
        a.history = _typed("history", toks, "int32", (None,))
        a.history_len = toks.numel()
        a.history_offsets = _typed("history offsets", off, "int32", (M + 1,))
        a.prompt = _typed("prompt", prompt, "int32", (M,))
        a.repetition = _typed("repetition", repetition, "float32", (M,))
        a.presence = _typed("presence", presence, "float32", (M,))
        a.frequency = _typed("frequency", frequency, "float32", (M,))
    if bias is not None:
        ids, vals, off = bias
        a.bias_ids = _typed("bias ids", ids, "int32", (None,))
        a.bias = _typed("bias", vals, "float32", (ids.numel(),))
        a.bias_len = ids.numel()
        a.bias_offsets = _typed("bias offsets", off, "int32", (M + 1,))
    if masks is not None:
        bits, ids = masks
        a.masks = _typed("masks", bits, "int32", (None, (V + 31) // 32))
        a.nmasks = bits.shape[0]
        a.mask_ids = _typed("mask ids", ids, "int32", (M,))
    ws = (None, 0) if tokens is None else _ws_args(workspace, stream, logits)
    return (ctypes.pointer(a), *ws, _stream(stream, logits))


def rq_logits(logits, out, tokens=None, *, history=None, repetition=None, presence=None,
              frequency=None, bias=None, masks=None, stream=None, workspace=AUTO):
    """Penalties, biases and masks on logits, and the greatest of each row.
    logits and out float32 [M][V] (out may be logits); tokens int32 [M] or
    None.  history: (int32 tokens of all rows, int32 offsets [M + 1], int32
    [M] number of given tokens or None), with the float32 [M] penalties
    repetition, presence and frequency (None: none).  bias: (int32 token ids
    of all rows, float32 values, int32 offsets [M + 1]).  masks: (int32
    [nmasks][(V + 31) // 32] bits of allowed tokens, int32 [M] mask of each
    row, outside 0 .. nmasks-1 none).  ``workspace``: AUTO (the binding's, per stream)
    or a zeroed tensor of RQ_LOGITS_WORKSPACE_BYTES; used with tokens."""
    st = lib().rq_logits(*_logits_cargs(
        logits, out, tokens, history=history, repetition=repetition, presence=presence,
        frequency=frequency, bias=bias, masks=masks, stream=stream, workspace=workspace))
    if st != RQ_OK:
        raise RqError("rq_logits", st)
    return out


def _float_type(what, t):
    """RQ_TYPE_F16 or RQ_TYPE_F32 of a tensor."""
    for name, kind in (("float16", RQ_TYPE_F16), ("float32", RQ_TYPE_F32)):
        if str(t.dtype) == "torch." + name:
            return kind
    raise ValueError(f"{what}: float16 or float32 expected, got {t.dtype}")


def _scale_type(what, t):
    """RQ_SCALE_F32 or RQ_SCALE_E8M0 of a tensor of scales."""
    name = str(t.dtype)
    if name == "torch.float32":
        return RQ_SCALE_F32
    if name in ("torch.float8_e8m0fnu", "torch.uint8"):
        return RQ_SCALE_E8M0
    raise ValueError(f"{what}: float32, float8_e8m0fnu or uint8 expected, got {t.dtype}")


def _scales(what, t, kind, shape):
    """Pointer of a tensor of scales of this kind and shape."""
    if _scale_type(what, t) != kind:
        raise ValueError(f"{what}: scales of one type expected")
    return _typed(what, t, str(t.dtype)[6:], shape)


def _e4m3(what, t, shape):
    """Pointer of a tensor of E4M3 values of this shape."""
    name = str(t.dtype)[6:]
    if name not in ("float8_e4m3fn", "uint8"):
        raise ValueError(f"{what}: float8_e4m3fn or uint8 expected, got {t.dtype}")
    return _typed(what, t, name, shape)


def _blocks_of(what, K):
    if K % RQ_FP8_BLOCK:
        raise ValueError(f"{what}: whole blocks of {RQ_FP8_BLOCK} expected, got {K}")
    return K // RQ_FP8_BLOCK


def _quant_fp8_cargs(x, q, scales, *, act=RQ_ACT_NONE, stream=None):
    M, K = x.shape
    kind = _scale_type("scales", scales)
    return (_ptr(x), _float_type("x", x), int(act), _e4m3("q", q, (M, K)),
            _scales("scales", scales, kind, (M, _blocks_of("x", K))), kind, M, K,
            _stream(stream, x))


def rq_quant_fp8(x, q, scales, act=RQ_ACT_NONE, stream=None):
    """Rows quantized in blocks of 128: a = act(x) (RQ_ACT_NONE, RQ_ACT_RELU2), a
    block's scale the smallest power of two s with |a| <= 448 s (2^-126 at
    least), q the E4M3 number nearest a / s.  x float16 or float32 [M][K], q
    E4M3 [M][K], scales float32 or E8M0 [M][K / 128]."""
    st = lib().rq_quant_fp8(*_quant_fp8_cargs(x, q, scales, act=act, stream=stream))
    if st != RQ_OK:
        raise RqError("rq_quant_fp8", st)
    return q, scales


def _gemm_fp8_cargs(problems, *, act=RQ_ACT_NONE, stream=None, workspace=AUTO):
    arr = (RqFp8Problem * len(problems))()
    M = problems[0][2].shape[0]
    kind = _scale_type("w_scales", problems[0][1])
    first = problems[0][5]
    out = RQ_TYPE_E4M3 if isinstance(first, (tuple, list)) else _float_type("y", first)
    for i, (w, ws, x, xs, y_in, y, N, K) in enumerate(problems):
        kb, nb = _blocks_of("w", K), (N + RQ_FP8_BLOCK - 1) // RQ_FP8_BLOCK
        if isinstance(y, (tuple, list)) != (out == RQ_TYPE_E4M3):
            raise ValueError("y: outputs of one type expected")
        if out == RQ_TYPE_E4M3:
            py = _e4m3("y", y[0], (M, N))
            ps = _scales("y_scales", y[1], kind, (M, _blocks_of("y", N)))
        else:
            py, ps = _typed("y", y, "float16" if out == RQ_TYPE_F16 else "float32", (M, N)), None
        arr[i] = RqFp8Problem(_e4m3("w", w, (N, K)), _scales("w_scales", ws, kind, (nb, kb)),
                              _e4m3("x", x, (M, K)), _scales("x_scales", xs, kind, (M, kb)),
                              _typed("y_in", y_in, "float32", (M, N)), py, ps, int(N), int(K))
    if isinstance(workspace, str) and workspace == AUTO:
        import torch
        # none for graphs, which may be replayed on several streams at once
        if torch.cuda.is_current_stream_capturing() or \
                not _gemm_fp8_bytes(arr, len(problems), M, kind, out)[1]:
            workspace = None
    return (arr, len(problems), M, kind, out, int(act),
            *_ws_args(workspace, stream, problems[0][2]), _stream(stream, problems[0][2]))


def _gemm_fp8_bytes(arr, count, M, kind, out):
    """(status, bytes)"""
    b = ctypes.c_size_t(0)
    st = lib().rq_gemm_fp8_workspace_size(arr, count, M, kind, out, ctypes.byref(b))
    return st, b.value


def rq_gemm_fp8(problems, act=RQ_ACT_NONE, stream=None, workspace=AUTO):
    """Products of block-scaled operands, y = y_in + x W^T, in one launch.
    ``problems`` is a sequence of (w, w_scales, x, x_scales, y_in, y, N, K): w
    E4M3 [N][K] with scales [(N + 127) // 128][K / 128], x E4M3 [M][K] with
    scales [M][K / 128], y_in float32 [M][N] (y itself, another tensor, or
    None), y float32 or float16 [M][N], or a pair (E4M3 [M][N], scales [M][N /
    128]) for the float16 output quantized as rq_quant_fp8 with ``act`` does.
    All share M, the type of scales and the type of y.  Sums of a float32 y are
    held in float32; those of the others from more than 64 tiles of 128 x 128
    outputs on to about 2^-15 (include/rq.h).  ``workspace``: AUTO
    (the binding's, per stream, if the call uses one; None in a graph's
    capture), a tensor of rq_gemm_fp8_workspace_size bytes (zero before its
    first use), or None to keep K whole.  A prepared call keeps the workspace
    that it was prepared with, so give it its own if graphs that hold it run at
    once."""
    st = lib().rq_gemm_fp8(*_gemm_fp8_cargs(problems, act=act, stream=stream,
                                            workspace=workspace))
    if st != RQ_OK:
        raise RqError("rq_gemm_fp8", st)
    return [p[5] for p in problems]


def rq_gemm_fp8_workspace_size(shapes, M, scale_type, out_type):
    """Bytes of workspace rq_gemm_fp8 uses for products of these (N, K).
    Host-only."""
    arr = (RqFp8Problem * len(shapes))()
    for i, (N, K) in enumerate(shapes):
        arr[i].N, arr[i].K = int(N), int(K)
    st, need = _gemm_fp8_bytes(arr, len(shapes), int(M), int(scale_type), int(out_type))
    if st != RQ_OK:
        raise RqError("rq_gemm_fp8_workspace_size", st)
    return need


def _groupnorm_cargs(y, groups, weight, bias, eps, out, *, bonus=None, gate=None,
                     act=RQ_ACT_NONE, stream=None):
    T, C = y.shape
    a = RqGroupnormArgs(y=_typed("y", y, "float32", (T, C)),
                        weight=_typed("weight", weight, "float32", (C,)),
                        bias=_typed("bias", bias, "float32", (C,)), T=T, C=C, groups=int(groups),
                        eps=float(eps), act=int(act))
    like = gate if bonus is None else bonus[0]
    name = "float32"
    if like is not None:
        a.input_type = _float_type("gate" if bonus is None else "r", like)
        name = "float16" if a.input_type == RQ_TYPE_F16 else "float32"
    if bonus is not None:
        r, k, r_k, v = bonus
        a.r, a.k, a.v = (_typed(n, t, name, (T, C)) for n, t in (("r", r), ("k", k), ("v", v)))
        a.r_k = _typed("r_k", r_k, "float32", (C,))
    a.gate = _typed("gate", gate, name, (T, C))
    if isinstance(out, (tuple, list)):
        a.out_type = RQ_TYPE_E4M3
        a.scale_type = _scale_type("out scales", out[1])
        a.out = _e4m3("out", out[0], (T, C))
        a.out_scales = _scales("out scales", out[1], a.scale_type, (T, _blocks_of("out", C)))
    else:
        a.out_type = _float_type("out", out)
        a.out = _typed("out", out, str(out.dtype)[6:], (T, C))
    return ctypes.pointer(a), _stream(stream, y)


def rq_groupnorm(y, groups, weight, bias, eps, out, bonus=None, gate=None, act=RQ_ACT_NONE,
                 stream=None):
    """Group norm of every token's channels with what follows it in the time
    mix: out = (norm(y) * weight + bias + sum(r * k * r_k) * v) * act(gate), the
    norm and the sum over each of ``groups`` groups of 32, 64, 128 or 256
    channels.  y float32 [T][C]; weight and bias float32 [C] or None; bonus
    (r, k, r_k, v) or None, r, k, v [T][C] all float32 or all float16, r_k
    float32 [C]; gate [T][C] of their type or None; act RQ_ACT_NONE or
    RQ_ACT_SILU; out float32 (y itself too) or float16 [T][C], or a pair (E4M3
    [T][C], scales [T][C / 128]) for the float16 output as rq_quant_fp8
    quantizes it."""
    st = lib().rq_groupnorm(*_groupnorm_cargs(y, groups, weight, bias, eps, out, bonus=bonus,
                                              gate=gate, act=act, stream=stream))
    if st != RQ_OK:
        raise RqError("rq_groupnorm", st)
    return out


_CARGS = {"rq_shift": _shift_cargs, "rq_wkv7": _wkv7_cargs, "rq_lora": _lora_cargs,
          "rq_logits": _logits_cargs, "rq_quant_fp8": _quant_fp8_cargs,
          "rq_gemm_fp8": _gemm_fp8_cargs, "rq_groupnorm": _groupnorm_cargs}


def prepare(name, *args, stream=None, workspace=AUTO, **options):
    """Resolve the tensor arguments of one call now and return a callable that
    repeats it with no per-call argument conversion in Python (for step loops
    and graph capture).  ``name`` is "rq_gemv", "rq_gemm_smallm",
    "rq_gemm_smallm_noalloc", "rq_gemv_batched", "rq_dequant", "rq_shift",
    "rq_wkv7", "rq_lora", "rq_logits", "rq_quant_fp8", "rq_gemm_fp8" or
    "rq_groupnorm"; ``args`` (and ``options``, the keyword arguments of the last
    four) are those of the Python function of that name, without ``stream`` (and
    ``workspace``, which rq_gemm_smallm, rq_lora, rq_logits and rq_gemm_fp8 take
    as a keyword, resolved now).  The tensors must stay alive."""
    L = lib()
    if name in _CARGS:
        if name in ("rq_lora", "rq_logits", "rq_gemm_fp8"):
            options["workspace"] = workspace
        return _prepared(name, getattr(L, name), _CARGS[name](*args, stream=stream, **options))
    if options:
        raise TypeError(f"{name} takes no option {sorted(options)[0]!r}")
    if name == "rq_gemm_smallm" and workspace is not None:
        name = "rq_gemm_smallm_ws"
    f = getattr(L, name)
    if name == "rq_gemv_batched":
        problems, M, bits, group, layout = args
        arr = _problems(problems)
        cargs = (arr, len(problems), int(M), int(bits), int(group), int(layout),
                 _stream(stream, problems[0][0]))
    elif name == "rq_dequant":
        qweight, scales, zeros, out, N, K, bits, group, layout, out_kind = args
        cargs = (_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(out), int(N), int(K),
                 int(bits), int(group), int(layout), int(out_kind), _stream(stream, qweight))
    else:
        qweight, scales, zeros, x, y, M, N, K, bits, group, layout = args[:11]
        cargs = (_ptr(qweight), _ptr(scales), _ptr(zeros), _ptr(x), _ptr(y), int(M), int(N),
                 int(K), int(bits), int(group), int(layout))
        if name == "rq_gemm_smallm_ws":
            ws = args[11] if len(args) > 11 else workspace
            cargs += _ws_args(ws, stream, qweight)
        cargs += (_stream(stream, qweight),)
    return _prepared(name, f, cargs)


def _prepared(name, f, cargs):
    def call():
        st = f(*cargs)
        if st != RQ_OK:
            raise RqError(name, st)
    call.args = cargs  # keeps the problem array (or argument structure) alive
    return call


def gemm_config(M, N, K, bits, group, layout, allow_split=True):
    """(plan, splits) of the small-batch matrix-core kernel for one product
    (plan 1-based, as RQ_GEMM_PLAN numbers them), or None when that kernel
    cannot take the shape.  Host-only."""
    plan, splits = ctypes.c_int(0), ctypes.c_int(0)
    st = lib().rq_gemm_config(int(M), int(N), int(K), int(bits), int(group), int(layout),
                              1 if allow_split else 0, ctypes.byref(plan), ctypes.byref(splits))
    if st == RQ_ERR_UNSUPPORTED:
        return None
    if st != RQ_OK:
        raise RqError("rq_gemm_config", st)
    return plan.value, splits.value


GEMV_KERNELS = ("vector", "decode_mfma", "smallm_mfma")


def gemv_config(M, N, K, bits, group, layout):
    """The kernel rq_gemv runs for one product, as (name, lpr, cpl, npass):
    name one of GEMV_KERNELS; lpr, cpl, npass the vector-unit launch shape
    (lanes per row, 0 for the generic kernel; 16-byte chunks per lane; rows
    per lane), zeros for the matrix-core kernels.  Host-only."""
    v = [ctypes.c_int(0) for _ in range(4)]
    st = lib().rq_gemv_config(int(M), int(N), int(K), int(bits), int(group), int(layout),
                              *[ctypes.byref(t) for t in v])
    if st != RQ_OK:
        raise RqError("rq_gemv_config", st)
    return (GEMV_KERNELS[v[0].value],) + tuple(t.value for t in v[1:])


def tuning_reload():
    """Re-read the RQ_* launch-shape override variables (tuning and tests)."""
    lib().rq_tuning_reload()
