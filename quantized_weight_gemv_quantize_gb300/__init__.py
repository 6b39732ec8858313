"""Python binding of libqgemv (the C ABI declared in include/qgemv.h).

Argument marshalling only: every step of the quantizer and the GEMV runs in the CUDA kernels of
``libqgemv.so``.  Arguments may be torch tensors (their device pointer is passed) or raw integer device
addresses; ``stream`` may be a torch.cuda.Stream, a raw cudaStream_t integer, or None (torch's current
stream).  A non-zero status raises :class:`QgemvError`.  There is no fallback of any kind: if the
compiled library is missing, importing the binding's entry points raises.
"""
import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqgemv.so")

QGEMV_Q4_K, QGEMV_Q6_K, QGEMV_Q8_0, QGEMV_W8A16, QGEMV_Q5_K, QGEMV_W8A16_CHANNEL = 1, 2, 3, 4, 5, 6
FMT = {"Q4_K": QGEMV_Q4_K, "Q5_K": QGEMV_Q5_K, "Q6_K": QGEMV_Q6_K, "Q8_0": QGEMV_Q8_0, "W8A16": QGEMV_W8A16,
       "W8A16_CHANNEL": QGEMV_W8A16_CHANNEL}
QGEMV_ACT_Q8_1, QGEMV_ACT_F32, QGEMV_ACT_BF16, QGEMV_ACT_F16 = 0, 1, 2, 3
ACT = {"q8_1": QGEMV_ACT_Q8_1, "f32": QGEMV_ACT_F32, "bf16": QGEMV_ACT_BF16, "f16": QGEMV_ACT_F16}
QGEMV_FLAG_PDL = 1
QGEMV_FLAG_PDL_LATE_TRIGGER = 2
QGEMV_MAX_GROUP = 8
QGEMV_ARGMAX_STATIC_SCRATCH_BYTES = 16384
QGEMV_ROPE_HALF, QGEMV_ROPE_INTERLEAVED = 0, 1
ROPE_LAYOUT = {"half": QGEMV_ROPE_HALF, "interleaved": QGEMV_ROPE_INTERLEAVED}
ROPE_SCALING = {"none": 0, "linear": 1, "base": 2, "parts": 3, "bands": 4}
QGEMV_ATTN_SCRATCH_HEAD = 65536
QGEMV_DEVERR_BAD_INDEX = 4
ROUTE_FUSED, ROUTE_GROUPED, ROUTE_PDL, ROUTE_Q5_K_M1, ROUTE_W8A16_CHANNEL_M1, ROUTE_ARGMAX, ROUTE_M16 = (
    33, 34, 35, 36, 44, 52, 53)
ROUTE_CHUNKED = 54
ROUTE_ROPE, ROUTE_ATTN_ROWS, ROUTE_ATTN_TILES, ROUTE_SAMPLE = 55, 56, 57, 58
STATUS = {0: "QGEMV_OK", 1: "QGEMV_ERR_INVALID_ARG", 2: "QGEMV_ERR_UNSUPPORTED", 3: "QGEMV_ERR_MISALIGNED",
          4: "QGEMV_ERR_CUDA", 5: "QGEMV_ERR_DEVICE", 6: "QGEMV_ERR_OVERLAP"}
NUM_ROUTES = 59

_lib = None


class QgemvMat(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("y", ctypes.c_void_p), ("N", ctypes.c_int)]


_i32, _i64, _vp, _f32 = ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p, ctypes.c_float


class QgemvCache(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_page", _i64), ("k_token", _i64), ("k_head", _i64), ("v_page", _i64),
                ("v_token", _i64), ("v_head", _i64), ("kind", _i32), ("num_pages", _i32), ("page_size", _i32),
                ("heads", _i32), ("dim", _i32)]


class QgemvRopeArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("q_out", _vp), ("k_out", _vp), ("q_token", _i64),
                ("q_head", _i64), ("k_token", _i64), ("k_head", _i64), ("v_token", _i64), ("v_head", _i64),
                ("q_out_token", _i64), ("q_out_head", _i64), ("k_out_token", _i64), ("k_out_head", _i64),
                ("positions", _vp), ("freqs", _vp), ("cache", ctypes.POINTER(QgemvCache)), ("slots", _vp),
                ("x_kind", _i32), ("out_kind", _i32), ("tokens", _i32), ("heads", _i32), ("kv_heads", _i32),
                ("dim", _i32), ("rot_dim", _i32), ("layout", _i32), ("mscale", _f32)]


class QgemvAttnArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("out", _vp), ("lse", _vp), ("q_token", _i64), ("q_head", _i64), ("out_token", _i64),
                ("out_head", _i64), ("cache", ctypes.POINTER(QgemvCache)), ("pages", _vp), ("pages_stride", _i64),
                ("q_start", _vp), ("kv_len", _vp), ("scratch", _vp), ("scratch_bytes", ctypes.c_size_t),
                ("kind", _i32), ("tokens", _i32), ("heads", _i32), ("seqs", _i32), ("max_q", _i32), ("max_kv", _i32),
                ("scale", _f32), ("causal", _i32), ("window", _i32)]


class QgemvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        name = STATUS.get(status, f"status {status}")
        extra = ""
        if status == 4 and _lib is not None:
            extra = f" (cudaError {_lib.qgemv_last_cuda_error()})"
        super().__init__(f"{where}: {name}{extra}")


def lib():
    """Load libqgemv.so (built by ``build()``); raises if it is absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"libqgemv.so not built at {LIB_PATH}; run quantized_weight_gemv_quantize_gb300.build()")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.qgemv_quantize_act.argtypes = [vp, i32, i32, vp, vp]
        L.qgemv.argtypes = [i32, vp, vp, vp, i32, i32, i32, vp]
        L.qgemv_w8a16.argtypes = [vp, vp, vp, i32, i32, i32, vp]
        L.qgemv_quantize_act_ex.argtypes = [vp, i32, i32, vp, ctypes.c_uint, vp]
        L.qgemv_quantize_act_typed.argtypes = [i32, vp, i32, i32, vp, ctypes.c_uint, vp]
        L.qgemv_w8a16_channel.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp]
        L.qgemv_w8a16_channel_ex.argtypes = [vp, vp, vp, vp, i32, i32, i32, ctypes.c_uint, vp]
        L.qgemv_max_k_w8a16_channel.argtypes = [i32]
        L.qgemv_max_k_w8a16_channel.restype = i32
        L.qgemv_tune_pairs.argtypes = [i32]
        L.qgemv_tune_pairs.restype = None
        L.qgemv_argmax_scratch_bytes.argtypes = [i32]
        L.qgemv_argmax_scratch_bytes.restype = sz
        L.qgemv_argmax.argtypes = [i32, vp, vp, i32, i32, i32, vp, sz, vp, vp, ctypes.c_uint, vp]
        L.qgemv_argmax.restype = i32
        L.qgemv_argmax_noalloc.argtypes = [i32, vp, vp, i32, i32, i32, vp, vp, ctypes.c_uint, vp]
        L.qgemv_argmax_noalloc.restype = i32
        L.qgemv_ex.argtypes = [i32, vp, vp, vp, i32, i32, i32, ctypes.c_uint, vp]
        L.qgemv_w8a16_ex.argtypes = [vp, vp, vp, i32, i32, i32, ctypes.c_uint, vp]
        L.qgemv_multi.argtypes = [i32, i32, ctypes.POINTER(QgemvMat), i32, vp, vp, i32, i32, ctypes.c_uint, vp]
        for f in ("qgemv_quantize_act", "qgemv", "qgemv_w8a16", "qgemv_quantize_act_ex", "qgemv_ex",
                  "qgemv_w8a16_ex", "qgemv_multi", "qgemv_quantize_act_typed", "qgemv_w8a16_channel",
                  "qgemv_w8a16_channel_ex"):
            getattr(L, f).restype = i32
        L.qgemv_weight_bytes.argtypes = [i32, i32, i32]
        L.qgemv_weight_bytes.restype = sz
        L.qgemv_act_bytes.argtypes = [i32, i32]
        L.qgemv_act_bytes.restype = sz
        L.qgemv_max_k.argtypes = [i32, i32]
        L.qgemv_max_k.restype = i32
        L.qgemv_max_k_w8a16.argtypes = [i32]
        L.qgemv_max_k_w8a16.restype = i32
        L.qgemv_chunk_k.argtypes = [i32, i32, i32]
        L.qgemv_chunk_k.restype = i32
        L.qgemv_status_string.argtypes = [i32]
        L.qgemv_status_string.restype = ctypes.c_char_p
        L.qgemv_last_cuda_error.argtypes = []
        L.qgemv_last_cuda_error.restype = i32
        L.qgemv_route_counts.argtypes = [ctypes.POINTER(ctypes.c_ulonglong), i32]
        L.qgemv_route_counts.restype = i32
        L.qgemv_route_reset.argtypes = []
        L.qgemv_route_reset.restype = None
        L.qgemv_debug_fail_next.argtypes = [i32, i32]
        L.qgemv_debug_fail_next.restype = None
        L.qgemv_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint), i32]
        L.qgemv_device_error.restype = i32
        L.qgemv_plan_info.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_longlong)]
        L.qgemv_plan_info.restype = i32
        L.qgemv_plan_info_chunk.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.POINTER(ctypes.c_longlong)]
        L.qgemv_plan_info_chunk.restype = i32
        L.qgemv_tune_override.argtypes = [i32, i32, i32, i32, i32]
        L.qgemv_tune_override.restype = None
        dbl, u64p = ctypes.c_double, ctypes.POINTER(ctypes.c_ulonglong)
        L.qgemv_rope_freqs.argtypes = [i32, dbl, i32, dbl, dbl, dbl, dbl, u64p, ctypes.POINTER(ctypes.c_float)]
        L.qgemv_rope_freqs.restype = i32
        L.qgemv_rope.argtypes = [ctypes.POINTER(QgemvRopeArgs), ctypes.c_uint, vp]
        L.qgemv_rope.restype = i32
        L.qgemv_attn.argtypes = [ctypes.POINTER(QgemvAttnArgs), ctypes.c_uint, vp]
        L.qgemv_attn.restype = i32
        L.qgemv_tune_attn.argtypes = [i32]
        L.qgemv_tune_attn.restype = None
        L.qgemv_attn_scratch_bytes.argtypes = [i32] * 7
        L.qgemv_attn_scratch_bytes.restype = sz
        L.qgemv_sample.argtypes = [i32, vp, ctypes.c_longlong, i32, i32, vp, vp, vp, vp, vp, vp, vp, ctypes.c_uint, vp]
        L.qgemv_sample.restype = i32
        ip = ctypes.POINTER(ctypes.c_int)
        L.qgemv_trace_info.argtypes = [ip, ip, ip]
        L.qgemv_trace_info.restype = i32
        L.qgemv_trace_begin.argtypes = []
        L.qgemv_trace_begin.restype = i32
        L.qgemv_trace_read.argtypes = [ctypes.POINTER(ctypes.c_ulonglong), sz, ip]
        L.qgemv_trace_read.restype = i32
        _lib = L
    return _lib


def build(force: bool = False) -> str:
    from . import _build
    return _build.build(force=force)


def use_trace_build() -> str:
    """Build the launch-timeline library (libqgemv_trace.so) and make it the one this process loads; must
    come before the first call that loads the library."""
    global LIB_PATH
    if _lib is not None:
        raise RuntimeError("use_trace_build() must come before the library is loaded")
    from . import _build
    LIB_PATH = _build.build(trace=True)
    return LIB_PATH


def trace_begin() -> None:
    _check(lib().qgemv_trace_begin(), "qgemv_trace_begin")


def trace_read():
    """The timeline records as a uint64 array [launches, ctas, fields] and the number of launches numbered."""
    import numpy as np
    nl, nc, nf = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(lib().qgemv_trace_info(ctypes.byref(nl), ctypes.byref(nc), ctypes.byref(nf)), "qgemv_trace_info")
    buf = np.zeros(nl.value * nc.value * nf.value, dtype=np.uint64)
    n = ctypes.c_int()
    _check(lib().qgemv_trace_read(buf.ctypes.data_as(ctypes.POINTER(ctypes.c_ulonglong)), buf.nbytes,
                                  ctypes.byref(n)), "qgemv_trace_read")
    return buf.reshape(nl.value, nc.value, nf.value), n.value


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _fmt(fmt):
    return FMT[fmt] if isinstance(fmt, str) else int(fmt)


def _check(status: int, where: str):
    if status != 0:
        raise QgemvError(status, where)


def qgemv_quantize_act(x, m: int, K: int, xq, stream=None) -> None:
    _check(lib().qgemv_quantize_act(_ptr(x), m, K, _ptr(xq), _stream(stream)), "qgemv_quantize_act")


def qgemv(fmt, W, xq, y, m: int, N: int, K: int, stream=None) -> None:
    _check(lib().qgemv(_fmt(fmt), _ptr(W), _ptr(xq), _ptr(y), m, N, K, _stream(stream)), "qgemv")


def qgemv_w8a16(W, x_bf16, y, m: int, N: int, K: int, stream=None) -> None:
    _check(lib().qgemv_w8a16(_ptr(W), _ptr(x_bf16), _ptr(y), m, N, K, _stream(stream)), "qgemv_w8a16")


def qgemv_quantize_act_ex(x, m: int, K: int, xq, flags: int = 0, stream=None) -> None:
    _check(lib().qgemv_quantize_act_ex(_ptr(x), m, K, _ptr(xq), flags, _stream(stream)), "qgemv_quantize_act_ex")


def qgemv_quantize_act_typed(x_kind, x, m: int, K: int, xq, flags: int = 0, stream=None) -> None:
    """x_kind: "f32", "bf16", "f16" (or the QGEMV_ACT_* value); x holds m*K values of that kind."""
    xk = ACT[x_kind] if isinstance(x_kind, str) else int(x_kind)
    _check(lib().qgemv_quantize_act_typed(xk, _ptr(x), m, K, _ptr(xq), flags, _stream(stream)),
           "qgemv_quantize_act_typed")


def qgemv_w8a16_channel(Wq, scale, x_bf16, y, m: int, N: int, K: int, flags: int = 0, stream=None) -> None:
    """Per-output-channel INT8 weights (int8 [N, K]) with fp32 row scales [N] against bf16 [m, K]."""
    _check(lib().qgemv_w8a16_channel_ex(_ptr(Wq), _ptr(scale), _ptr(x_bf16), _ptr(y), m, N, K, flags,
                                        _stream(stream)), "qgemv_w8a16_channel")


def qgemv_argmax_scratch_bytes(m: int) -> int:
    return int(lib().qgemv_argmax_scratch_bytes(m))


def qgemv_argmax(fmt, W, xq, m: int, N: int, K: int, scratch, idx_out, val_out, flags: int = 0,
                 stream=None) -> None:
    """Fused GEMV + argmax: idx_out[i] / val_out[i] get the first row with the largest y[i, :]."""
    nbytes = scratch.numel() * scratch.element_size() if hasattr(scratch, "numel") else qgemv_argmax_scratch_bytes(m)
    _check(lib().qgemv_argmax(_fmt(fmt), _ptr(W), _ptr(xq), m, N, K, _ptr(scratch), nbytes, _ptr(idx_out),
                              _ptr(val_out), flags, _stream(stream)), "qgemv_argmax")


def qgemv_argmax_noalloc(fmt, W, xq, m: int, N: int, K: int, idx_out, val_out, flags: int = 0,
                         stream=None) -> None:
    """qgemv_argmax on the library's own static scratch (calls on a device must be ordered)."""
    _check(lib().qgemv_argmax_noalloc(_fmt(fmt), _ptr(W), _ptr(xq), m, N, K, _ptr(idx_out), _ptr(val_out), flags,
                                      _stream(stream)), "qgemv_argmax_noalloc")


def qgemv_max_k_w8a16_channel(m: int) -> int:
    return int(lib().qgemv_max_k_w8a16_channel(m))


def qgemv_ex(fmt, W, xq, y, m: int, N: int, K: int, flags: int = 0, stream=None) -> None:
    _check(lib().qgemv_ex(_fmt(fmt), _ptr(W), _ptr(xq), _ptr(y), m, N, K, flags, _stream(stream)), "qgemv_ex")


def qgemv_w8a16_ex(W, x_bf16, y, m: int, N: int, K: int, flags: int = 0, stream=None) -> None:
    _check(lib().qgemv_w8a16_ex(_ptr(W), _ptr(x_bf16), _ptr(y), m, N, K, flags, _stream(stream)), "qgemv_w8a16_ex")


def mats_array(mats):
    """[(W, y, N), ...] -> ctypes array of qgemv_mat (keep the result alive across the call)."""
    arr = (QgemvMat * len(mats))()
    for j, (W, y, N) in enumerate(mats):
        arr[j].W, arr[j].y, arr[j].N = _ptr(W), _ptr(y), int(N)
    return arr


def qgemv_multi(fmt, mats, act_kind, act, m: int, K: int, xq_out=None, flags: int = 0, stream=None) -> None:
    """mats: [(W, y, N), ...] sharing one activation; act_kind "q8_1" | "f32" | "bf16" (or its code)."""
    arr = mats if isinstance(mats, ctypes.Array) else mats_array(mats)
    kind = ACT[act_kind] if isinstance(act_kind, str) else int(act_kind)
    _check(lib().qgemv_multi(_fmt(fmt), len(arr), arr, kind, _ptr(act), _ptr(xq_out), m, K, flags,
                             _stream(stream)), "qgemv_multi")


_TORCH_ACT = {"torch.float32": QGEMV_ACT_F32, "torch.bfloat16": QGEMV_ACT_BF16, "torch.float16": QGEMV_ACT_F16}


def _kind(t):
    """QGEMV_ACT_* of a tensor's type; types outside the library's are refused."""
    if str(t.dtype) not in _TORCH_ACT:
        raise QgemvError(1, f"tensor of {t.dtype}")
    return _TORCH_ACT[str(t.dtype)]


def _need(ok, what):
    if not ok:
        raise QgemvError(1, what)


def _typed(t, dtype, what):
    """A contiguous tensor of the given type (or a raw address, which is passed on as it is)."""
    if t is None or isinstance(t, int):
        return t
    _need(str(t.dtype) == "torch." + dtype and t.is_contiguous(), f"{what}: a contiguous {dtype} tensor")
    return t


def kv_cache(k, v) -> QgemvCache:
    """The paged cache of two tensors [pages, page_size, heads, dim] (views with any strides; a [pages, heads, page_size,
    dim] allocation is passed as ``t.transpose(1, 2)``).  Keep the tensors alive as long as the result."""
    _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype, "kv_cache: k and v alike, of four dimensions")
    _need(k.stride(3) == 1 and v.stride(3) == 1, "kv_cache: the last dimension contiguous")
    c = QgemvCache(_ptr(k), _ptr(v), *k.stride()[:3], *v.stride()[:3], _kind(k), *k.shape)
    c.tensors = (k, v)
    return c


def _heads_first(t, what):
    _need(t.dim() == 3 and t.stride(2) == 1, f"{what}: [tokens, heads, dim], the last dimension contiguous")
    return t.stride(0), t.stride(1)


def qgemv_rope_freqs(rot_dim: int, theta: float = 10000.0, scaling="none", factor: float = 1.0, trained: float = 0.0,
                     low: float = 1.0, high: float = 32.0):
    """(frequencies, mscale): a CPU int64 tensor of rot_dim/2 turns per position in units of 2^-64, to be copied to the
    device once, and the factor of the rotated values.  scaling: "none", "linear", "base", "parts" or "bands"."""
    import torch
    out = (ctypes.c_ulonglong * max(1, rot_dim // 2))()
    ms = ctypes.c_float()
    code = ROPE_SCALING[scaling] if isinstance(scaling, str) else int(scaling)
    _check(lib().qgemv_rope_freqs(rot_dim, theta, code, factor, trained, low, high, out, ctypes.byref(ms)),
           "qgemv_rope_freqs")
    return torch.tensor([ctypes.c_longlong(v).value for v in out], dtype=torch.int64), float(ms.value)


def rope_args(q, k, v, positions, freqs, q_out=None, k_out=None, cache=None, slots=None, rot_dim=None, layout="half",
              mscale: float = 1.0) -> QgemvRopeArgs:
    """Arguments of qgemv_rope from tensors: q [tokens, heads, dim], k and v [tokens, kv_heads, dim] (q, or k with v, may
    be None).  The result holds the tensors' addresses and keeps the tensors alive; it may be used for many calls."""
    a = QgemvRopeArgs()
    x = q if q is not None else k
    _need(x is not None, "rope_args: q or k")
    for t, name in ((q, "q"), (k, "k"), (v, "v")):
        if t is not None:
            token, head = _heads_first(t, f"rope_args: {name}")
            _need(t.dtype == x.dtype and t.shape[0] == x.shape[0] and t.shape[2] == x.shape[2], f"rope_args: {name} unlike the others")
            setattr(a, name, _ptr(t)), setattr(a, name + "_token", token), setattr(a, name + "_head", head)
    out = q_out if q_out is not None else k_out
    for t, src, name in ((q_out, q, "q_out"), (k_out, k, "k_out")):
        if t is not None:
            token, head = _heads_first(t, f"rope_args: {name}")
            _need(src is not None and t.shape == src.shape and t.dtype == out.dtype, f"rope_args: {name} unlike its input")
            setattr(a, name, _ptr(t)), setattr(a, name + "_token", token), setattr(a, name + "_head", head)
    _need(v is None or (k is not None and v.shape == k.shape), "rope_args: v unlike k")
    a.positions, a.freqs = _ptr(_typed(positions, "int32", "positions")), _ptr(_typed(freqs, "int64", "freqs"))
    a.slots = _ptr(_typed(slots, "int64", "slots"))
    a.tokens, a.dim = x.shape[0], x.shape[2]
    a.heads, a.kv_heads = (0 if q is None else q.shape[1]), (0 if k is None else k.shape[1])
    a.rot_dim = a.dim if rot_dim is None else rot_dim
    for t, name, n in ((positions, "positions", a.tokens), (slots, "slots", a.tokens), (freqs, "freqs", a.rot_dim // 2)):
        _need(t is None or isinstance(t, int) or t.numel() >= n, f"rope_args: {name} too short")
    a.x_kind, a.out_kind = _kind(x), (_kind(out) if out is not None else _kind(x))
    a.layout = ROPE_LAYOUT[layout] if isinstance(layout, str) else int(layout)
    a.mscale = mscale
    if cache is not None:
        a.cache = ctypes.pointer(cache)
    a.tensors = (q, k, v, q_out, k_out, positions, freqs, slots, cache)
    return a


def qgemv_rope(args: QgemvRopeArgs, flags: int = 0, stream=None) -> None:
    """Rotary positions of q and k, with the write of k and v into the cache; args from rope_args()."""
    _check(lib().qgemv_rope(args, flags, _stream(stream)), "qgemv_rope")


def qgemv_attn_scratch_bytes(seqs: int, tokens: int, heads: int, kv_heads: int, dim: int, max_q: int, max_kv: int) -> int:
    """Scratch of every qgemv_attn call with these sizes or smaller seqs, tokens, max_q and max_kv; its first QGEMV_ATTN_SCRATCH_HEAD bytes must start as zeros."""
    return int(lib().qgemv_attn_scratch_bytes(seqs, tokens, heads, kv_heads, dim, max_q, max_kv))


def attn_args(q, cache: QgemvCache, pages, q_start, kv_len, out, scratch, max_q: int, max_kv: int, scale: float,
              causal: bool = True, window: int = 0, lse=None) -> QgemvAttnArgs:
    """Arguments of qgemv_attn from tensors: q and out [tokens, heads, dim], pages int32 [seqs, pages of a row] (a view of longer
    rows too, such as ``table[:, :n]``: context beyond its columns is not read), q_start int32 [seqs + 1], kv_len int32 [seqs], scratch uint8, lse fp32 [tokens, heads] or None.  The result holds the
    tensors' addresses and keeps the tensors alive; it may be used for many calls."""
    a = QgemvAttnArgs()
    a.q_token, a.q_head = _heads_first(q, "attn_args: q")
    a.out_token, a.out_head = _heads_first(out, "attn_args: out")
    _need(q.shape == out.shape and q.dtype == out.dtype and q.shape[2] == cache.dim, "attn_args: q, out and the cache unlike")
    _need(pages.dim() == 2 and str(pages.dtype) == "torch.int32" and (pages.shape[1] == 0 or pages.stride(1) == 1),
          "attn_args: pages int32 [seqs, pages]")
    a.q, a.out, a.lse = _ptr(q), _ptr(out), _ptr(_typed(lse, "float32", "lse"))
    a.cache = ctypes.pointer(cache)
    a.seqs = pages.shape[0]
    # the record's stride is also the length of a row: max_kv holds it to the columns there are
    columns = pages.shape[1]
    _need(a.seqs <= 1 or pages.stride(0) >= columns, "attn_args: rows of pages overlap")
    a.pages, a.pages_stride = _ptr(pages), columns if a.seqs <= 1 or columns == 0 else pages.stride(0)
    max_kv = min(max_kv, columns * cache.page_size)
    a.q_start, a.kv_len = _ptr(_typed(q_start, "int32", "q_start")), _ptr(_typed(kv_len, "int32", "kv_len"))
    _need(isinstance(q_start, int) or q_start.numel() == a.seqs + 1, "attn_args: q_start has seqs + 1 values")
    _need(isinstance(kv_len, int) or kv_len.numel() == a.seqs, "attn_args: kv_len has seqs values")
    _need(lse is None or isinstance(lse, int) or lse.shape == q.shape[:2], "attn_args: lse [tokens, heads]")
    _need(scratch.is_contiguous(), "attn_args: scratch contiguous")
    a.scratch, a.scratch_bytes = _ptr(scratch), scratch.numel() * scratch.element_size()
    a.kind, a.tokens, a.heads = _kind(q), q.shape[0], q.shape[1]
    a.max_q, a.max_kv, a.scale, a.causal, a.window = max_q, max_kv, scale, 1 if causal else 0, window
    a.tensors = (q, cache, pages, q_start, kv_len, out, scratch, lse)
    return a


def qgemv_attn(args: QgemvAttnArgs, flags: int = 0, stream=None) -> None:
    """Attention of new tokens over a paged cache; args from attn_args()."""
    _check(lib().qgemv_attn(args, flags, _stream(stream)), "qgemv_attn")


def qgemv_sample(logits, temperature, top_k, top_p, min_p, u, token_out, prob_out=None, flags: int = 0,
                 stream=None) -> None:
    """One token per row of logits [m, N] from the uniform numbers u [m]; temperature, top_p, min_p fp32 [m] and top_k
    int32 [m], each or None."""
    _need(logits.dim() == 2 and (logits.shape[1] <= 1 or logits.stride(1) == 1), "qgemv_sample: logits [m, N], rows contiguous")
    m, n = logits.shape
    for t, dtype, name in ((temperature, "float32", "temperature"), (top_k, "int32", "top_k"), (top_p, "float32", "top_p"),
                           (min_p, "float32", "min_p"), (u, "float32", "u"), (token_out, "int32", "token_out"),
                           (prob_out, "float32", "prob_out")):
        _need(t is None or isinstance(t, int) or _typed(t, dtype, name).numel() == m, f"qgemv_sample: {name} has m values")
    _check(lib().qgemv_sample(_kind(logits), _ptr(logits), logits.stride(0) if m > 1 else n, m, n, _ptr(temperature),
                              _ptr(top_k), _ptr(top_p), _ptr(min_p), _ptr(u), _ptr(token_out), _ptr(prob_out), flags,
                              _stream(stream)), "qgemv_sample")


def qgemv_weight_bytes(fmt, N: int, K: int) -> int:
    return int(lib().qgemv_weight_bytes(_fmt(fmt), N, K))


def qgemv_act_bytes(m: int, K: int) -> int:
    return int(lib().qgemv_act_bytes(m, K))


def qgemv_chunk_k(fmt, m: int, K: int) -> int:
    """Values per K-chunk of a call at (fmt, m, K): K when the rows take one pass of staging."""
    return int(lib().qgemv_chunk_k(_fmt(fmt), m, K))


def qgemv_max_k(fmt, m: int) -> int:
    return int(lib().qgemv_max_k(_fmt(fmt), m))


def qgemv_max_k_w8a16(m: int) -> int:
    return int(lib().qgemv_max_k_w8a16(m))


def qgemv_status_string(status: int) -> str:
    return lib().qgemv_status_string(status).decode()


def qgemv_route_counts():
    buf = (ctypes.c_ulonglong * NUM_ROUTES)()
    n = lib().qgemv_route_counts(buf, NUM_ROUTES)
    return [int(buf[i]) for i in range(min(n, NUM_ROUTES))]


def qgemv_route_reset() -> None:
    lib().qgemv_route_reset()


def qgemv_debug_fail_next(status: int, count: int = 1) -> None:
    lib().qgemv_debug_fail_next(status, count)


def qgemv_device_error(reset: bool = False) -> int:
    v = ctypes.c_uint(0)
    _check(lib().qgemv_device_error(ctypes.byref(v), 1 if reset else 0), "qgemv_device_error")
    return int(v.value)


PLAN_FIELDS = ("lanes", "rows_per_tile", "num_tiles", "stages", "stage_bytes", "smem", "grid", "row_bytes",
               "units_per_row", "x_stage_bytes", "threads", "team_warps", "red_bytes", "kernel_build")


def qgemv_plan_info(fmt, m: int, N: int, K: int, num_sms: int = 152, ctas_per_sm: int = 1) -> dict:
    """The launch plan for (fmt, m, N, K); fmt "W8A16" (or 4) asks for the W8A16 kernel."""
    f = FMT[fmt] if isinstance(fmt, str) else int(fmt)
    buf = (ctypes.c_longlong * 14)()
    _check(lib().qgemv_plan_info(f, m, N, K, num_sms, ctas_per_sm, buf), "qgemv_plan_info")
    return dict(zip(PLAN_FIELDS, [int(v) for v in buf]))


def qgemv_plan_info_chunk(fmt, m: int, N: int, Kc: int, num_sms: int = 152, ctas_per_sm: int = 1) -> dict:
    """The plan of one K-chunk launch of Kc values per row: qgemv_plan_info's fields plus slot_row_stride."""
    f = FMT[fmt] if isinstance(fmt, str) else int(fmt)
    buf = (ctypes.c_longlong * 15)()
    _check(lib().qgemv_plan_info_chunk(f, m, N, Kc, num_sms, ctas_per_sm, buf), "qgemv_plan_info_chunk")
    return dict(zip(PLAN_FIELDS + ("slot_row_stride",), [int(v) for v in buf]))


def qgemv_tune_pairs(mode: int = 0) -> None:
    """Tuning only: row pairs 0 = planner decides, 1 = whenever they fit, 2 = never."""
    lib().qgemv_tune_pairs(mode)


def qgemv_tune_attn(kernel: int = 0) -> None:
    """Tuning only: attention's kernel 0 = planner decides, 1 = the 16-row kernel, 2 = the 128-row kernel."""
    lib().qgemv_tune_attn(kernel)


def qgemv_tune_override(ctas_per_sm: int = 0, lanes_log2: int = -1, rows_per_tile: int = 0, stages: int = 0,
                        kernel_build: int = 0) -> None:
    """Force plan parameters for sweeps (0 / -1 = planner decides).  Not for production use."""
    lib().qgemv_tune_override(ctas_per_sm, lanes_log2, rows_per_tile, stages, kernel_build)
