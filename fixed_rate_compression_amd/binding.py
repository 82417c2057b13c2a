"""Thin ctypes binding of libcodecgauge.so (include/codec_gauge.h).

Argument marshalling only: the functions keep the C names, take torch CUDA
tensors (or numpy arrays for host arguments), pass raw pointers plus the
current HIP stream, and raise on a negative return code.  All computation
happens in the HIP library; if it is not built, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libcodecgauge.so")

CG_OK = 0
CG_E_INVAL, CG_E_SHAPE, CG_E_UNSUPPORTED, CG_E_SIZE, CG_E_HIP, CG_E_INTERNAL = -1, -2, -3, -4, -5, -6
CG_DTYPE_F32, CG_DTYPE_BF16 = 0, 1
CG_BACKEND_NONE, CG_BACKEND_ZFP, CG_BACKEND_BLOCK_UNIFORM, CG_BACKEND_KIVI = 0, 1, 2, 3
CG_HEADER_BYTES = 64

EXPORTED = ["cg_encoded_bytes", "cg_encode", "cg_decode", "cg_decode_gauged", "cg_roundtrip",
            "cg_gauge_fit_stats", "cg_gauge_fit_grad", "cg_stats_workspace_bytes", "cg_gauge_from_skew",
            "cg_gauge_apply", "cg_write_header", "cg_decode_error_workspace_bytes",
            "cg_decode_error", "cg_decode_error_noalloc", "cg_cache_error_summary", "cg_adamw_update", "cg_gauge_control",
            "cg_second_moment_workspace_bytes", "cg_second_moment", "cg_gauge_grad", "cg_gauge_heads",
            "cg_attend_workspace_bytes", "cg_attend", "cg_append", "cg_evict", "cg_read", "cg_rotate",
            "cg_last_error"]

CG_KEEP_KEYS, CG_KEEP_VALUES = 1, 2
CG_NOALLOC_SCRATCH_BYTES = 16 << 20
CG_CONTROL_IDENTITY, CG_CONTROL_HADAMARD, CG_CONTROL_DCT, CG_CONTROL_ORTHONORMALIZE, CG_CONTROL_KLT = range(5)


class CgShape(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int32), ("kv", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("heads", ctypes.c_int32), ("tokens", ctypes.c_int64),
                ("token_capacity", ctypes.c_int64), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class CgGauge(ctypes.Structure):
    _keep = None    # the tensor G points into (make_gauge)
    _fields_ = [("group", ctypes.c_int32), ("G", ctypes.c_void_p)]


class CgCodec(ctypes.Structure):
    _fields_ = [("backend", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("block_tokens", ctypes.c_int32), ("residual_tokens", ctypes.c_int32)]


class CgFieldError(ctypes.Structure):
    _fields_ = [("sse", ctypes.c_double), ("ref_ss", ctypes.c_double), ("max_abs", ctypes.c_double),
                ("values", ctypes.c_double)]


class CgCacheError(ctypes.Structure):
    _fields_ = [("mse", ctypes.c_double), ("nrmse", ctypes.c_double), ("key_nrmse", ctypes.c_double),
                ("value_nrmse", ctypes.c_double), ("max_abs", ctypes.c_double),
                ("values", ctypes.c_double)]


class CgStats(ctypes.Structure):
    _fields_ = [("L_freq", ctypes.c_double), ("L_rate", ctypes.c_double), ("L", ctypes.c_double),
                ("sum_E", ctypes.c_double)]


class CgAttn(ctypes.Structure):
    _keep = ()      # the tensors lengths and starts point into (make_attn)
    _fields_ = [("layer", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("n_queries", ctypes.c_int32),
                ("causal", ctypes.c_int32), ("scale", ctypes.c_float), ("lengths", ctypes.c_void_p),
                ("starts", ctypes.c_void_p), ("q_batch_stride", ctypes.c_int64),
                ("q_token_stride", ctypes.c_int64)]


class CgRotary(ctypes.Structure):
    _keep = ()      # the tensors freq and the weights point into (make_rotary)
    _fields_ = [("dim", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("dealt", ctypes.c_int32), ("sections", ctypes.c_int32 * 4), ("eps", ctypes.c_float),
                ("magnitude", ctypes.c_float), ("freq", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p)]


class CgRows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("batch_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64)]


class CodecGaugeError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} failed with {code}: {msg}")
        self.code = code


_lib = None


def lib():
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        # torch loads its bundled HIP runtime under the name "libamdhip64.so";
        # importing it first lets this library's libamdhip64.so.7 dependency
        # resolve (by soname) to that same runtime instead of a second copy
        import torch  # noqa: F401
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                               "(there is no CPU fallback)")
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, U64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
        SP, GP, CP = ctypes.POINTER(CgShape), ctypes.POINTER(CgGauge), ctypes.POINTER(CgCodec)
        U64P, AP, RP = ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(CgAttn), ctypes.POINTER(CgRows)
        sig = {
            "cg_encoded_bytes": [SP, CP, U64P, U64P, U64P],
            "cg_encode": [SP, P, GP, CP, I64, I64, P, U64, P, U64, P],
            "cg_decode": [SP, P, U64, P, U64, GP, CP, I64, I64, P, P],
            "cg_decode_gauged": [SP, P, U64, P, U64, GP, CP, I64, I64, I32, P, P],
            "cg_gauge_heads": [SP, GP, I32, I32, I32, I64, I32, P, P, P],
            "cg_roundtrip": [SP, P, GP, CP, P, U64, P, U64, P, P],
            "cg_gauge_fit_stats": [SP, P, I32, P, I32, ctypes.c_float, ctypes.c_float,
                                   ctypes.c_float, P, ctypes.c_size_t, P, P, P],
            "cg_gauge_fit_grad": [SP, P, I32, P, I32, ctypes.c_float, ctypes.c_float,
                                   ctypes.c_float, P, ctypes.c_size_t, P, P, P],
            "cg_stats_workspace_bytes": [SP, I32, I32, ctypes.POINTER(ctypes.c_size_t)],
            "cg_gauge_from_skew": [I64, I32, P, P],
            "cg_gauge_apply": [SP, P, GP, I32, P, P],
            "cg_write_header": [SP, CP, I32, I32, P, U64],
            "cg_decode_error_workspace_bytes": [SP, GP, CP, I64, I64, ctypes.POINTER(ctypes.c_size_t)],
            "cg_decode_error": [SP, P, U64, P, U64, GP, CP, I64, I64, P, P, P, ctypes.c_size_t, P, P],
            "cg_decode_error_noalloc": [SP, P, U64, P, U64, GP, CP, I64, I64, P, P, P, P],
            "cg_cache_error_summary": [SP, P, ctypes.POINTER(CgCacheError)],
            "cg_adamw_update": [I64, P, P, P, P, I64, ctypes.c_double, ctypes.c_double,
                                ctypes.c_double, ctypes.c_double, ctypes.c_double],
            "cg_gauge_control": [I32, I64, I32, P, P],
            "cg_second_moment_workspace_bytes": [SP, I32, ctypes.POINTER(ctypes.c_size_t)],
            "cg_second_moment": [SP, P, I32, P, ctypes.c_size_t, P, P],
            "cg_gauge_grad": [I64, I32, P, P, P],
            "cg_attend_workspace_bytes": [SP, GP, CP, AP, I32, ctypes.POINTER(ctypes.c_size_t)],
            "cg_attend": [SP, P, U64, P, U64, GP, CP, AP, P, P, P, P, P, ctypes.c_size_t, P],
            "cg_append": [SP, GP, CP, I32, I32, P, P, I64, I64, P, P, P, P, U64, P, U64, P],
            "cg_evict": [SP, CP, I32, I32, I32, P, P, U64, P, U64, P, SP, P, U64, P, U64, P, P, P, P],
            "cg_read": [SP, P, U64, P, U64, GP, CP, I32, I32, P, P, P, P, I64, I64, P],
            "cg_rotate": [SP, ctypes.POINTER(CgRotary), I32, I32, P, P, P, RP, RP, RP, RP, P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.cg_last_error.argtypes = []
        L.cg_last_error.restype = ctypes.c_char_p
        _lib = L
    return _lib


def _check(fn, rc):
    if rc != CG_OK:
        raise CodecGaugeError(fn, rc, lib().cg_last_error().decode())


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):          # a raw device address (e.g. a window inside a tensor)
        return t
    if isinstance(t, np.ndarray):
        assert t.flags["C_CONTIGUOUS"]
        return t.ctypes.data
    assert t.is_contiguous(), "tensors must be contiguous"
    return t.data_ptr()


def _nbytes(t):
    if t is None:
        return 0
    if isinstance(t, np.ndarray):
        return t.nbytes
    return t.numel() * t.element_size()


def _span(t):
    """(address, bytes) of an array."""
    try:
        assert t.is_contiguous(), "tensors must be contiguous"
        return t.data_ptr(), t.nbytes
    except AttributeError:          # none, a raw address or a numpy array
        return _ptr(t), _nbytes(t)


def _stream(stream):
    if stream is not None:
        return stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def make_shape(layers, kv, batch, heads, tokens, token_capacity=None, head_dim=128,
               dtype=CG_DTYPE_BF16) -> CgShape:
    return CgShape(layers, kv, batch, heads, tokens,
                   tokens if token_capacity is None else token_capacity, head_dim, dtype)


def make_gauge(group: int, G=None) -> CgGauge:
    gg = CgGauge(group, _ptr(G) if G is not None else None)
    gg._keep = G      # the struct holds a raw pointer: keep the tensor alive with it
    return gg


def make_codec(backend, bits=4, block_tokens=0, residual_tokens=0) -> CgCodec:
    return CgCodec(backend, bits, block_tokens, residual_tokens)


def cg_encoded_bytes(shape: CgShape, codec: CgCodec):
    p, m, h = ctypes.c_uint64(), ctypes.c_uint64(), ctypes.c_uint64()
    _check("cg_encoded_bytes", lib().cg_encoded_bytes(ctypes.byref(shape), ctypes.byref(codec),
                                                      ctypes.byref(p), ctypes.byref(m),
                                                      ctypes.byref(h)))
    return p.value, m.value, h.value


def cg_encode(shape, kv, gauge, codec, t0, nt, payload, meta=None, stream=None):
    _check("cg_encode", lib().cg_encode(ctypes.byref(shape), _ptr(kv), ctypes.byref(gauge),
                                        ctypes.byref(codec), t0, nt, _ptr(payload),
                                        _nbytes(payload), _ptr(meta), _nbytes(meta),
                                        _stream(stream)))


def cg_decode(shape, payload, meta, gauge, codec, t0, nt, kv_out, stream=None):
    _check("cg_decode", lib().cg_decode(ctypes.byref(shape), _ptr(payload), _nbytes(payload),
                                        _ptr(meta), _nbytes(meta), ctypes.byref(gauge),
                                        ctypes.byref(codec), t0, nt, _ptr(kv_out),
                                        _stream(stream)))


def cg_decode_gauged(shape, payload, meta, gauge, codec, t0, nt, keep, kv_out, stream=None):
    """cg_decode leaving the kinds in `keep` (CG_KEEP_KEYS | CG_KEEP_VALUES) gauged."""
    _check("cg_decode_gauged", lib().cg_decode_gauged(
        ctypes.byref(shape), _ptr(payload), _nbytes(payload), _ptr(meta), _nbytes(meta),
        ctypes.byref(gauge), ctypes.byref(codec), t0, nt, keep, _ptr(kv_out), _stream(stream)))


def cg_gauge_heads(shape, gauge, layer, kind, q_heads, rows, dtype, x, y, stream=None):
    """Forward gauge of (layer, kind) on the head segments of x [rows][q_heads*d] -> y."""
    _check("cg_gauge_heads", lib().cg_gauge_heads(
        ctypes.byref(shape), ctypes.byref(gauge), layer, kind, q_heads, rows, dtype, _ptr(x),
        _ptr(y), _stream(stream)))


def cg_decode_error_workspace_bytes(shape, gauge, codec, t0, nt):
    b = ctypes.c_size_t()
    _check("cg_decode_error_workspace_bytes", lib().cg_decode_error_workspace_bytes(
        ctypes.byref(shape), ctypes.byref(gauge), ctypes.byref(codec), t0, nt, ctypes.byref(b)))
    return b.value


def cg_decode_error(shape, payload, meta, gauge, codec, t0, nt, kv_out, kv_ref, workspace, err,
                    stream=None):
    """err: device float64 tensor [n_fields, 4] (sse, ref_ss, max_abs, values)."""
    _check("cg_decode_error", lib().cg_decode_error(
        ctypes.byref(shape), _ptr(payload), _nbytes(payload), _ptr(meta), _nbytes(meta),
        ctypes.byref(gauge), ctypes.byref(codec), t0, nt, _ptr(kv_out), _ptr(kv_ref),
        _ptr(workspace), _nbytes(workspace), _ptr(err), _stream(stream)))


def cg_decode_error_noalloc(shape, payload, meta, gauge, codec, t0, nt, kv_out, kv_ref, err,
                            stream=None):
    """cg_decode_error with the library's built-in device scratch (no workspace)."""
    _check("cg_decode_error_noalloc", lib().cg_decode_error_noalloc(
        ctypes.byref(shape), _ptr(payload), _nbytes(payload), _ptr(meta), _nbytes(meta),
        ctypes.byref(gauge), ctypes.byref(codec), t0, nt, _ptr(kv_out), _ptr(kv_ref),
        _ptr(err), _stream(stream)))


def cg_cache_error_summary(shape, err_host: np.ndarray) -> dict:
    """err_host float64 [n_fields, 4] -> dict of the whole-cache figures."""
    e = np.ascontiguousarray(err_host, np.float64)
    out = CgCacheError()
    _check("cg_cache_error_summary", lib().cg_cache_error_summary(ctypes.byref(shape), e.ctypes.data,
                                                                  ctypes.byref(out)))
    return {k: getattr(out, k) for k, _ in CgCacheError._fields_}


def cg_adamw_update(param, grad, m, v, step, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                    weight_decay=1e-2):
    """In place on host fp64 arrays of equal size."""
    arrs = [param, grad, m, v]
    for a in arrs:
        assert isinstance(a, np.ndarray) and a.dtype == np.float64 and a.flags["C_CONTIGUOUS"]
        assert a.size == param.size
    _check("cg_adamw_update", lib().cg_adamw_update(param.size, *[a.ctypes.data for a in arrs], step,
                                                    lr, beta1, beta2, eps, weight_decay))


def cg_gauge_control(kind, n, g, M=None) -> np.ndarray:
    """-> fp32 [n, g, g] control gauges (M fp64 [n, g, g] for ORTHONORMALIZE / KLT)."""
    G = np.empty((n, g, g), np.float32)
    Mc = np.ascontiguousarray(M, np.float64) if M is not None else None
    if Mc is not None:
        assert Mc.shape == (n, g, g)
    _check("cg_gauge_control", lib().cg_gauge_control(kind, n, g, Mc.ctypes.data if Mc is not None else None,
                                                      G.ctypes.data))
    return G


def cg_second_moment_workspace_bytes(shape, g):
    b = ctypes.c_size_t()
    _check("cg_second_moment_workspace_bytes",
           lib().cg_second_moment_workspace_bytes(ctypes.byref(shape), g, ctypes.byref(b)))
    return b.value


def cg_second_moment(shape, kv, g, workspace, stream=None) -> np.ndarray:
    """-> fp64 [layers, kv, heads, d/g, g, g] second moments (synchronous)."""
    M = np.empty((shape.layers, shape.kv, shape.heads, shape.head_dim // g, g, g), np.float64)
    _check("cg_second_moment", lib().cg_second_moment(ctypes.byref(shape), _ptr(kv), g, _ptr(workspace),
                                                      _nbytes(workspace), M.ctypes.data, _stream(stream)))
    return M


def cg_roundtrip(shape, kv_in, gauge, codec, payload, meta, kv_out, stream=None):
    _check("cg_roundtrip", lib().cg_roundtrip(ctypes.byref(shape), _ptr(kv_in),
                                              ctypes.byref(gauge), ctypes.byref(codec),
                                              _ptr(payload), _nbytes(payload), _ptr(meta),
                                              _nbytes(meta), _ptr(kv_out), _stream(stream)))


def cg_gauge_apply(shape, kv, gauge, direction, out, stream=None):
    _check("cg_gauge_apply", lib().cg_gauge_apply(ctypes.byref(shape), _ptr(kv),
                                                  ctypes.byref(gauge), direction, _ptr(out),
                                                  _stream(stream)))


def cg_gauge_from_skew(A: np.ndarray) -> np.ndarray:
    """A fp64 [n, g, g] (host) -> G = exp(A - A^T) fp32 [n, g, g] (host)."""
    A = np.ascontiguousarray(A, np.float64)
    n, g, _ = A.shape
    G = np.empty((n, g, g), np.float32)
    _check("cg_gauge_from_skew", lib().cg_gauge_from_skew(n, g, A.ctypes.data, G.ctypes.data))
    return G


def cg_gauge_grad(A: np.ndarray, dG: np.ndarray) -> np.ndarray:
    """A, dG fp64 [n, g, g] (host) -> dL/dA fp64 [n, g, g] for G = exp(A - A^T)."""
    A = np.ascontiguousarray(A, np.float64)
    dG = np.ascontiguousarray(dG, np.float64)
    n, g, _ = A.shape
    assert dG.shape == A.shape
    dA = np.empty_like(A)
    _check("cg_gauge_grad", lib().cg_gauge_grad(n, g, A.ctypes.data, dG.ctypes.data, dA.ctypes.data))
    return dA


def cg_stats_workspace_bytes(shape, g, T_b):
    b = ctypes.c_size_t()
    _check("cg_stats_workspace_bytes", lib().cg_stats_workspace_bytes(ctypes.byref(shape), g, T_b,
                                                                      ctypes.byref(b)))
    return b.value


def cg_gauge_fit_stats(shape, kv, g, A_host: np.ndarray, T_b, tau, lambda_f, lambda_r, workspace,
                       grad=True, stream=None):
    """Returns (stats structured array [n_fields], dA fp64 or None)."""
    nf = shape.layers * shape.kv * shape.batch * shape.heads
    out = (CgStats * nf)()
    A = np.ascontiguousarray(A_host, np.float64) if A_host is not None else None
    grad = grad and g != 0
    dA = np.zeros((nf, shape.head_dim // g, g, g), np.float64) if grad else None
    _check("cg_gauge_fit_stats", lib().cg_gauge_fit_stats(
        ctypes.byref(shape), _ptr(kv), g, A.ctypes.data if A is not None else None, T_b, tau,
        lambda_f, lambda_r,
        _ptr(workspace), _nbytes(workspace), ctypes.cast(out, ctypes.c_void_p),
        dA.ctypes.data if grad else None, _stream(stream)))
    stats = np.array([(o.L_freq, o.L_rate, o.L, o.sum_E) for o in out],
                     dtype=[("L_freq", "f8"), ("L_rate", "f8"), ("L", "f8"), ("sum_E", "f8")])
    return stats, dA


def cg_gauge_fit_grad(shape, kv, g, A_host: np.ndarray, T_b, tau, lambda_f, lambda_r, workspace,
                      stream=None):
    """Returns (stats structured array [n_fields], dA fp64 [L, KV, H, D/g, g, g]
    summed over the batch, or None for g = 0)."""
    nf = shape.layers * shape.kv * shape.batch * shape.heads
    out = (CgStats * nf)()
    A = np.ascontiguousarray(A_host, np.float64) if A_host is not None else None
    dA = (np.zeros((shape.layers, shape.kv, shape.heads, shape.head_dim // g, g, g), np.float64)
          if g else None)
    _check("cg_gauge_fit_grad", lib().cg_gauge_fit_grad(
        ctypes.byref(shape), _ptr(kv), g, A.ctypes.data if A is not None else None, T_b, tau,
        lambda_f, lambda_r, _ptr(workspace), _nbytes(workspace), ctypes.cast(out, ctypes.c_void_p),
        dA.ctypes.data if g else None, _stream(stream)))
    stats = np.array([(o.L_freq, o.L_rate, o.L, o.sum_E) for o in out],
                     dtype=[("L_freq", "f8"), ("L_rate", "f8"), ("L", "f8"), ("sum_E", "f8")])
    return stats, dA


def cg_write_header(shape, codec, layer, kv) -> bytes:
    buf = ctypes.create_string_buffer(CG_HEADER_BYTES)
    _check("cg_write_header", lib().cg_write_header(ctypes.byref(shape), ctypes.byref(codec),
                                                    layer, kv, buf, CG_HEADER_BYTES))
    return buf.raw


_dtypes = {}


def _dtype(name):
    """torch's dtype of that name (looked up once)."""
    d = _dtypes.get(name)
    if d is None:
        import torch
        d = _dtypes[name] = getattr(torch, name)
    return d


def _sized(name, t, dtype, count):
    """A device array argument whose size and type the C call cannot see."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype is not (_dtypes.get(dtype) or _dtype(dtype)) or t.numel() < count or not t.is_contiguous():
        raise ValueError(f"{name}: {count} contiguous values of {dtype} are needed, got {t.numel()} of {t.dtype}")
    return t.data_ptr()


def _here(*arrays):
    """Kernels run on the current GPU: arrays elsewhere are refused before a launch.
    -> its number (None if no array was a tensor)."""
    cur = None
    for t in arrays:
        if t is None or type(t) is int:
            continue
        try:
            dev = t.get_device()
        except AttributeError:      # a numpy array
            dev = -1
        if dev == cur:
            continue
        if dev < 0:
            raise ValueError("device tensors are needed, got one in host memory")
        if cur is None:
            cur = _current_device()
        if dev != cur:
            raise ValueError(f"a tensor is on GPU {dev}, the current one is {cur}")
    return cur


_raw_device = None


def _current_device():
    """torch.cuda.current_device of a process that has a device tensor, without its check for a first call."""
    global _raw_device
    if _raw_device is None:
        import torch
        _raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _raw_device()


_raw_stream = None


def _stream_on(stream, device):
    """_stream for a device that is known to be the current one: torch.cuda.current_stream
    makes an object and takes 3 us, a third of a small call."""
    global _raw_stream
    if stream is not None or device is None:
        return _stream(stream)
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


def _gauge_sized(gauge, shape):
    """The gauge's tensor holds what the C call reads of it."""
    G = gauge._keep
    if G is None:
        return
    need = shape.layers * 2 * shape.heads * shape.head_dim * gauge.group
    if hasattr(G, "numel") and (G.dtype != _dtype("float32") or G.numel() < need):
        raise ValueError(f"gauge: {need} values of float32 are needed, got {G.numel()} of {G.dtype}")


def _storage(shape):
    return "bfloat16" if shape.dtype == CG_DTYPE_BF16 else "float32"


def make_attn(layer, q_heads, n_queries, scale, causal=True, lengths=None, starts=None,
              q_strides=(0, 0)) -> CgAttn:
    """lengths, starts: device int32 [batch] (or None); q_strides: elements between
    sequences and between queries of q (0: dense)."""
    for name, t in (("lengths", lengths), ("starts", starts)):
        if t is not None and not isinstance(t, int) and t.dtype != _dtype("int32"):
            raise ValueError(f"{name} must be int32, got {t.dtype}")
    at = CgAttn(layer, q_heads, n_queries, 1 if causal else 0, scale, _ptr(lengths), _ptr(starts),
                q_strides[0], q_strides[1])
    at._keep = (lengths, starts)      # the struct holds raw pointers
    return at


def cg_attend_workspace_bytes(shape, gauge, codec, attn, with_mass=False):
    b = ctypes.c_size_t()
    _check("cg_attend_workspace_bytes", lib().cg_attend_workspace_bytes(
        ctypes.byref(shape), ctypes.byref(gauge), ctypes.byref(codec), ctypes.byref(attn),
        1 if with_mass else 0, ctypes.byref(b)))
    return b.value


def cg_attend(shape, payload, meta, gauge, codec, attn, q, out, lse=None, mass=None, workspace=None,
              stream=None):
    """Attention of q [batch, n, q_heads, 128] (heads contiguous, the other strides those
    of attn) over the encoded layer -> out (dense); see the header for lse and mass."""
    batch, n, heads, d = shape.batch, attn.n_queries, attn.q_heads, shape.head_dim
    rows, st = batch * n * heads, _storage(shape)
    if not isinstance(q, int):
        if q.dtype != _dtype(st) or q.shape != (batch, n, heads, d):
            raise ValueError(f"q must be {st} [batch, n, q_heads, head_dim], got {q.dtype} {tuple(q.shape)}")
        sb, sn, sh, sd = q.stride()
        if rows and ((batch > 1 and sb != (attn.q_batch_stride or n * heads * d)) or
                     (n > 1 and sn != (attn.q_token_stride or heads * d)) or (heads > 1 and sh != d) or sd != 1):
            raise ValueError(f"q of strides {q.stride()} does not lie as attn says")
    blk = codec.block_tokens
    _gauge_sized(gauge, shape)
    for name, t in zip(("lengths", "starts"), attn._keep):
        _sized(name, t, "int32", batch)
    dev = _here(q, out, payload, meta, lse, mass, workspace, gauge._keep, *attn._keep)
    rc = lib().cg_attend(
        shape, *_span(payload), *_span(meta), gauge, codec, attn,
        q if isinstance(q, int) else q.data_ptr(),
        _sized("out", out, st, rows * d), _sized("lse", lse, "float32", rows),
        _sized("mass", mass, "float32", shape.layers * batch * shape.heads * (shape.token_capacity // blk if blk > 0 else 0)),
        *_span(workspace), _stream_on(stream, dev))
    if rc != CG_OK:
        _check("cg_attend", rc)


def _kv_rows(shape, n, named):
    """Rows [batch, n, heads, head_dim] of the storage format with contiguous heads, all lying alike
    -> their addresses and (strides between sequences, between rows)."""
    st, at, ptrs = _dtype(_storage(shape)), None, []
    batch, heads, d = shape.batch, shape.heads, shape.head_dim
    for name, t in named:
        if t is None:
            ptrs.append(None)
            continue
        if t.dtype is not st:
            raise ValueError(f"{name} must be {_storage(shape)}, got {t.dtype}")
        if t.shape != (batch, n, heads, d):
            raise ValueError(f"{name} must be [batch, {n}, heads, head_dim], got {tuple(t.shape)}")
        sb, sr, sh, sd = t.stride()
        if (batch > 1 and sb == 0) or (n > 1 and sr == 0):
            raise ValueError(f"{name}: rows of an expanded tensor")
        lie = (sb if batch > 1 else 0, sr if n > 1 else 0)
        if (sh != d and heads > 1) or sd != 1 or lie != (at or lie):
            raise ValueError(f"{name} of strides {t.stride()}: contiguous heads and equal strides are needed")
        at = lie
        ptrs.append(t.data_ptr())
    return ptrs, at or (0, 0)


def cg_append(shape, gauge, codec, layer, n_new, k_new, v_new, tail, payload, meta, lengths=None,
              starts=None, stream=None):
    """k_new, v_new [batch, n_new, heads, 128] with contiguous heads and the same strides
    between sequences and between rows (of one sequence, or one row each: any)."""
    st, row = _storage(shape), shape.heads * shape.head_dim
    ptrs, (bs, rs) = _kv_rows(shape, n_new, (("k_new", k_new), ("v_new", v_new)))
    _gauge_sized(gauge, shape)
    dev = _here(k_new, v_new, tail, payload, meta, lengths, starts, gauge._keep)
    rc = lib().cg_append(
        shape, gauge, codec, layer, n_new, *ptrs, bs, rs,
        _sized("lengths", lengths, "int32", shape.batch), _sized("starts", starts, "int32", shape.batch),
        _sized("tail", tail, st, shape.layers * 2 * shape.batch * row * codec.block_tokens),
        *_span(payload), *_span(meta), _stream_on(stream, dev))
    if rc != CG_OK:
        _check("cg_append", rc)


def cg_read(shape, payload, meta, gauge, codec, layer, k_out, v_out, lengths=None, starts=None, stream=None):
    """Rows starts .. of every sequence of the layer into k_out and v_out [batch, n, heads, 128] (contiguous
    heads, equal strides; either may be None); rows that a sequence does not have are left as they were."""
    if k_out is None and v_out is None:
        raise ValueError("k_out and v_out are None")
    n = (v_out if k_out is None else k_out).shape[1]
    ptrs, (bs, rs) = _kv_rows(shape, n, (("k_out", k_out), ("v_out", v_out)))
    _gauge_sized(gauge, shape)
    dev = _here(k_out, v_out, payload, meta, lengths, starts, gauge._keep)
    rc = lib().cg_read(
        shape, *_span(payload), *_span(meta), gauge, codec, layer, n,
        _sized("lengths", lengths, "int32", shape.batch), _sized("starts", starts, "int32", shape.batch), *ptrs, bs, rs,
        _stream_on(stream, dev))
    if rc != CG_OK:
        _check("cg_read", rc)


def make_rotary(freq, sections=None, interleaved=False, dealt=False, q_weight=None, k_weight=None, eps=1e-6,
                magnitude=1.0) -> CgRotary:
    """freq: device float32 [dim / 2], radians a position; sections: pairs of each axis (None: one axis);
    q_weight, k_weight: device float32 [head_dim] of the heads' norms (None: no norm)."""
    sec = list(sections) if sections is not None and len(sections) > 1 else []
    if len(sec) > 4:
        raise ValueError(f"{len(sec)} axes: four at most")
    for name, t in (("freq", freq), ("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None and (t.dtype != _dtype("float32") or not t.is_contiguous() or t.dim() != 1):
            raise ValueError(f"{name} must be contiguous float32 of one axis")
    r = CgRotary(2 * freq.numel(), 1 if interleaved else 0, max(1, len(sec)), 1 if dealt else 0,
                 (ctypes.c_int32 * 4)(*sec), eps, magnitude, _ptr(freq), _ptr(q_weight), _ptr(k_weight))
    r._keep = (freq, q_weight, k_weight)
    return r


def _rows(name, t, st, batch, n, heads, d):
    """[batch, n, heads, head_dim] of the storage format -> CgRows."""
    if t.dtype is not st:
        raise ValueError(f"{name} must be {st}, got {t.dtype}")
    if t.shape != (batch, n, heads, d):
        raise ValueError(f"{name} must be [{batch}, {n}, {heads}, {d}], got {tuple(t.shape)}")
    sb, sr, sh, sd = t.stride()
    if batch == 1:
        sb = 0
    elif sb == 0:
        raise ValueError(f"{name}: rows of an expanded tensor")
    if n == 1:
        sr = 0
    elif sr == 0:
        raise ValueError(f"{name}: rows of an expanded tensor")
    if (sh != d and heads > 1) or sd != 1:
        raise ValueError(f"{name} of strides {t.stride()}: contiguous heads are needed")
    return CgRows(t.data_ptr(), sb, sr)


def cg_rotate(shape, rotary, q, k, q_out, k_out, lengths=None, starts=None, positions=None, stream=None):
    """Norm and rotation of q [batch, n, q_heads, 128] and k [batch, n, heads, 128] into q_out and k_out, which
    may be q and k themselves; either pair may be None.  positions: device int32 [axes, batch, n] or None."""
    if (q is None) != (q_out is None) or (k is None) != (k_out is None) or (q is None and k is None):
        raise ValueError("queries or keys, each with its output, are needed")
    lead = k if q is None else q
    if lead.dim() != 4:
        raise ValueError(f"rows must be [batch, n, heads, head_dim], got {tuple(lead.shape)}")
    batch, heads, d, st = shape.batch, shape.heads, shape.head_dim, _dtype(_storage(shape))
    n, q_heads = lead.shape[1], 0 if q is None else q.shape[2]
    qi = ki = rq = rk = None
    if q is not None:
        qi = _rows("q", q, st, batch, n, q_heads, d)
        rq = qi if q_out is q else _rows("q_out", q_out, st, batch, n, q_heads, d)
    if k is not None:
        ki = _rows("k", k, st, batch, n, heads, d)
        rk = ki if k_out is k else _rows("k_out", k_out, st, batch, n, heads, d)
    freq, wq, wk = rotary._keep
    if (wq is not None and wq.numel() != d) or (wk is not None and wk.numel() != d):
        raise ValueError(f"norm weights: {d} values are needed")
    if positions is not None and not isinstance(positions, int) and positions.shape != (rotary.axes, batch, n):
        raise ValueError(f"positions must be [axes, batch, n], got {tuple(positions.shape)}")
    dev = _here(q, k, q_out, k_out, lengths, starts, positions, freq, wq, wk)
    rc = lib().cg_rotate(
        shape, rotary, q_heads, n, _sized("positions", positions, "int32", rotary.axes * batch * n),
        _sized("lengths", lengths, "int32", batch), _sized("starts", starts, "int32", batch), qi, ki, rq, rk,
        _stream_on(stream, dev))
    if rc != CG_OK:
        _check("cg_rotate", rc)


def cg_evict(shape, codec, budget, sink, recent, mass, payload, meta, out_shape, payload_out, meta_out,
             mass_out, kept, lengths_out, lengths=None, stream=None):
    """Keep `budget` blocks a head by mass; the output arrays may be the inputs (in place)."""
    heads = shape.layers * shape.batch * shape.heads
    nblk, nout = (s.token_capacity // codec.block_tokens if codec.block_tokens > 0 else 0
                  for s in (shape, out_shape))
    dev = _here(mass, payload, meta, payload_out, meta_out, mass_out, kept, lengths_out, lengths)
    rc = lib().cg_evict(
        shape, codec, budget, sink, recent,
        _sized("mass", mass, "float32", heads * nblk), *_span(payload), *_span(meta),
        _sized("lengths", lengths, "int32", shape.batch), out_shape,
        *_span(payload_out), *_span(meta_out),
        _sized("mass_out", mass_out, "float32", heads * nout),
        _sized("kept", kept, "int32", heads * max(budget, 0)),
        _sized("lengths_out", lengths_out, "int32", shape.batch), _stream_on(stream, dev))
    if rc != CG_OK:
        _check("cg_evict", rc)


def cg_last_error() -> str:
    return lib().cg_last_error().decode()
