"""ctypes binding of libw4a8.so: the entry points of include/w4a8.h under the
same names, taking torch CUDA tensors.

Argument marshalling only: every step of the linear runs in the library's
CUDA kernels.  There is no fallback: if the library is missing or a call is
rejected, an exception is raised.
"""
from __future__ import annotations

import collections
import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libw4a8.so")

OK = 0
ERR_NULL, ERR_ALIGN, ERR_SHAPE, ERR_WORKSPACE, ERR_CUDA = 1, 2, 3, 4, 5
LAUNCH_PDL = 1
W4A8_MAX_M = 64
W8A16_MAX_M = 64

EXPORTS = [
    "w4_quantize_weights", "w8_quantize_weights", "act_quantize_i8",
    "w4a8_workspace_bytes", "w4a8_gemv", "w4a8_linear",
    "w8a16_workspace_bytes", "w8a16_gemv",
    "w4a8_last_error", "w4a8_device_error", "w4a8_set_tuning", "w4a8_plan_info",
    "w4a8_linear_noalloc", "w4a8_linear_grouped", "w4a8_linear_prefetch", "w4a8_linear_grouped_prefetch",
    "w4g_quantize_weights", "w4a8g_workspace_bytes", "w4a8g_gemv", "w4a8g_linear",
    "w4a8g_linear_grouped", "w4a8g_plan_info",
    "index_softmax_lut", "index_softmax_c_int", "index_softmax_u8",
    "w4_interleave_rows", "w4a8_gate_up_silu_workspace_bytes", "w4a8_gate_up_silu", "w4a8_silu_mul",
    "add_norm", "rope_frequencies", "rope_rotate", "kvq_write", "kvq_read", "kvq_keep",
    "kvq_attention_workspace_bytes", "kvq_attention",
    "rope_rotate_axes", "kvq_write_axes",
    "kvq_plan_workspace_bytes", "kvq_plan", "draft_verify_workspace_bytes", "draft_verify",
    "f8_quantize_weights", "f8_quantize_rows", "f8_gemm", "f8_linear_workspace_bytes", "f8_linear",
]


class W4A8Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__("status %d: %s" % (status, message))
        self.status = status


class _Tuning(ctypes.Structure):
    _fields_ = [("force_splits", ctypes.c_int), ("force_threads_per_row", ctypes.c_int),
                ("ring_bytes", ctypes.c_int), ("ctas_per_sm", ctypes.c_int),
                ("mma_min_m", ctypes.c_int), ("rowdot_max_m", ctypes.c_int),
                ("mma_e4m3", ctypes.c_int), ("qmma_max_m", ctypes.c_int),
                ("qmma_tiles_per_warp", ctypes.c_int), ("stall_test_us", ctypes.c_int),
                ("qmma_operands", ctypes.c_int)]


class _Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("ks", ctypes.c_void_p), ("vs", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page", ctypes.c_int), ("heads", ctypes.c_int), ("dim", ctypes.c_int),
                ("bits", ctypes.c_int)]


class _Batch(ctypes.Structure):
    _fields_ = [("cu", ctypes.c_void_p), ("start", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("seqs", ctypes.c_int64), ("tokens", ctypes.c_int64), ("max_pages", ctypes.c_int64)]


class _Pool(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("held", ctypes.c_void_p), ("stack", ctypes.c_void_p),
                ("top", ctypes.c_void_p), ("seqs", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("pages", ctypes.c_int64), ("page", ctypes.c_int)]


_i64, _p, _u = ctypes.c_int64, ctypes.c_void_p, ctypes.c_uint
_int, _f, _d = ctypes.c_int, ctypes.c_float, ctypes.c_double
_SIGS = {
    "w4_quantize_weights": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p]),
    "w8_quantize_weights": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p]),
    "act_quantize_i8": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p]),
    "w4a8_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "w4a8_gemv": (ctypes.c_int, [_p, _p, _i64, _i64, _p, _p, _i64, _p, _p, _p, ctypes.c_size_t, _u, _p]),
    "w4a8_linear": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _i64, _p, _p, _p, _p, _p, ctypes.c_size_t, _u, _p]),
    "w4a8_linear_prefetch": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _i64, _p, _p, ctypes.c_size_t, _u, _p, _p,
                                            ctypes.c_size_t]),
    "w4a8_linear_grouped_prefetch": (ctypes.c_int, [_p, _i64, _i64, ctypes.c_int, _p, _p, _p, _p, _p,
                                                    ctypes.c_size_t, _u, _p, _p, ctypes.c_size_t]),
    "w4a8_linear_noalloc": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _i64, _p, _u, _p]),
    "w4a8_linear_grouped": (ctypes.c_int, [_p, _i64, _i64, ctypes.c_int, _p, _p, _p, _p, _p,
                                           ctypes.c_size_t, _u, _p]),
    "w8a16_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "w8a16_gemv": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _i64, _p, _p, ctypes.c_size_t, _u, _p]),
    "w4a8_last_error": (ctypes.c_char_p, []),
    "w4a8_device_error": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint), _p]),
    "w4a8_set_tuning": (ctypes.c_int, [ctypes.POINTER(_Tuning)]),
    "w4a8_plan_info": (ctypes.c_int, [_i64, _i64, _i64, ctypes.c_int, ctypes.c_int,
                                      ctypes.POINTER(ctypes.c_int), ctypes.c_int]),
    "w4g_quantize_weights": (ctypes.c_int, [_p, _i64, _i64, _i64, _p, _p, _p]),
    "w4a8g_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64, _i64]),
    "w4a8g_gemv": (ctypes.c_int, [_p, _p, _i64, _i64, _i64, _p, _p, _i64, _p, _p, ctypes.c_size_t,
                                  _u, _p]),
    "w4a8g_linear": (ctypes.c_int, [_p, _i64, _i64, _i64, _p, _p, _i64, _p, _p, _p, _p,
                                    ctypes.c_size_t, _u, _p]),
    "w4a8g_linear_grouped": (ctypes.c_int, [_p, _i64, _i64, _i64, ctypes.c_int, _p, _p, _p, _p,
                                            _p, ctypes.c_size_t, _u, _p]),
    "w4a8g_plan_info": (ctypes.c_int, [_i64, _i64, _i64, _i64, ctypes.c_int,
                                       ctypes.POINTER(ctypes.c_int), ctypes.c_int]),
    "index_softmax_lut": (ctypes.c_int, [ctypes.c_int, ctypes.c_double, _p]),
    "index_softmax_c_int": (_i64, [ctypes.c_double, _i64, ctypes.c_float, ctypes.c_float]),
    "index_softmax_u8": (ctypes.c_int, [_p, _i64, _i64, _i64, ctypes.c_int, _p, _p, _p]),
    "w4_interleave_rows": (ctypes.c_int, [_p, _p, _p, _p, _i64, _i64, _p, _p, _p]),
    "w4a8_gate_up_silu_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "w4a8_gate_up_silu": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _i64, _p, _p, _p, ctypes.c_size_t, _u, _p]),
    "w4a8_silu_mul": (ctypes.c_int, [_p, _p, _i64, _i64, _p, _u, _p]),
    "add_norm": (ctypes.c_int, [_p, _int, _p, _int, _p, _p, _i64, _p, _i64, _i64, _f, _f, _f, _p, _p, _p, _p, _u, _p]),
    "rope_frequencies": (ctypes.c_int, [_int, _d, _int, _d, _d, _d, _d, _p, _p]),
    "rope_rotate": (ctypes.c_int, [_p, _int, _i64, _i64, _int, _int, _p, _p, _int, _int, _f, _p, _int, _i64, _u, _p]),
    "kvq_write": (ctypes.c_int, [_p, _p, _p, _i64, _p, _i64, _p, _i64, _int, _int, _p, _p, _int, _int, _f, _p, _u,
                                 _p]),
    "kvq_read": (ctypes.c_int, [_p, _p, _p, _p, _int, _u, _p]),
    "kvq_keep": (ctypes.c_int, [_p, _p, _p, _u, _p]),
    "kvq_attention_workspace_bytes": (ctypes.c_size_t, [_p, _p, _int]),
    "kvq_attention": (ctypes.c_int, [_p, _p, _p, _int, _p, _f, _p, _p, ctypes.c_size_t, _u, _p]),
    "rope_rotate_axes": (ctypes.c_int, [_p, _int, _i64, _i64, _int, _int, _p, _int, _p, _p, _int, _int, _f, _p, _int,
                                        _i64, _u, _p]),
    "kvq_write_axes": (ctypes.c_int, [_p, _p, _p, _i64, _p, _i64, _p, _i64, _int, _int, _p, _int, _p, _p, _int, _int, _f,
                                      _p, _u, _p]),
    "kvq_plan_workspace_bytes": (ctypes.c_size_t, [_p]),
    "kvq_plan": (ctypes.c_int, [_p, _p, _p, _p, _p, _i64, _p, _p, _p, _p, _p, ctypes.c_size_t, _u, _p]),
    "draft_verify_workspace_bytes": (ctypes.c_size_t, [_i64, _i64]),
    "draft_verify": (ctypes.c_int, [_p, _int, _i64, _i64, _p, _i64, _i64, _p, _p, _p, _int, _i64, _p, _p, _p, _p, _p, _p,
                                    ctypes.c_size_t, _u, _p]),
    "f8_quantize_weights": (ctypes.c_int, [_p, _i64, _i64, _p, _p, _p]),
    "f8_quantize_rows": (ctypes.c_int, [_p, _int, _i64, _i64, _p, _p, _u, _p]),
    "f8_gemm": (ctypes.c_int, [_p, _p, _i64, _i64, _p, _p, _i64, _p, _int, _u, _p]),
    "f8_linear_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64]),
    "f8_linear": (ctypes.c_int, [_p, _int, _i64, _i64, _p, _p, _i64, _p, _int, _p, ctypes.c_size_t, _u, _p]),
}

_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libw4a8.so not built: call __graft_entry__.build() or "
                              "python -m bit_weight_quantized_w4a8_gb300.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def _check(st: int):
    if st != OK:
        raise W4A8Error(st, lib().w4a8_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it (2 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor) -> int:
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _want(t, dtype, name, shape=None):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous() and \
            (shape is None or t.shape == shape):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


_ws_cache = {}


def _workspace(nbytes: int, device: torch.device, ws):
    """Caller-provided workspace, or a cached zero-filled one per device."""
    if nbytes == 0:
        return ws
    if ws is not None:
        return ws
    key = device.index if device.index is not None else torch.cuda.current_device()
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


# --------------------------------------------------------------------------
# entry points
# --------------------------------------------------------------------------

def w4_quantize_weights(W: torch.Tensor, Wq=None, sw=None):
    """W [N][K] fp32 -> (Wq [N][K/2] uint8, sw [N] fp32)."""
    _want(W, torch.float32, "W")
    N, K = W.shape
    Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device) if Wq is None else Wq
    sw = torch.empty((N,), dtype=torch.float32, device=W.device) if sw is None else sw
    _want(Wq, torch.uint8, "Wq", (N, K // 2))
    _want(sw, torch.float32, "sw", (N,))
    _check(lib().w4_quantize_weights(_ptr(W), N, K, _ptr(Wq), _ptr(sw), _stream(W)))
    return Wq, sw


def w8_quantize_weights(W: torch.Tensor, Wq8=None, sw16=None):
    """W [N][K] fp32 -> (Wq8 [N][K] int8, sw16 [N] fp16)."""
    _want(W, torch.float32, "W")
    N, K = W.shape
    Wq8 = torch.empty((N, K), dtype=torch.int8, device=W.device) if Wq8 is None else Wq8
    sw16 = torch.empty((N,), dtype=torch.float16, device=W.device) if sw16 is None else sw16
    _want(Wq8, torch.int8, "Wq8", (N, K))
    _want(sw16, torch.float16, "sw16", (N,))
    _check(lib().w8_quantize_weights(_ptr(W), N, K, _ptr(Wq8), _ptr(sw16), _stream(W)))
    return Wq8, sw16


def act_quantize_i8(X: torch.Tensor, Xq=None, sa=None):
    """X [M][K] fp16 -> (Xq [M][K] int8, sa [M] fp32)."""
    _want(X, torch.float16, "X")
    M, K = X.shape
    Xq = torch.empty((M, K), dtype=torch.int8, device=X.device) if Xq is None else Xq
    sa = torch.empty((M,), dtype=torch.float32, device=X.device) if sa is None else sa
    _want(Xq, torch.int8, "Xq", (M, K))
    _want(sa, torch.float32, "sa", (M,))
    _check(lib().act_quantize_i8(_ptr(X), M, K, _ptr(Xq), _ptr(sa), _stream(X)))
    return Xq, sa


def w4a8_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().w4a8_workspace_bytes(M, K, N))


def w8a16_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().w8a16_workspace_bytes(M, K, N))


def w4a8_gemv(Xq, sa, Wq, sw, Y=None, acc_out=None, ws=None, flags: int = 0):
    """Y[m][n] = ((float)sum_k Xq[m,k] q[n,k] * sw[n]) * sa[m]; returns Y."""
    _want(Xq, torch.int8, "Xq")
    M, K = Xq.shape
    N = Wq.shape[0]
    _want(sa, torch.float32, "sa", (M,))
    _want(Wq, torch.uint8, "Wq", (N, K // 2))
    _want(sw, torch.float32, "sw", (N,))
    Y = torch.empty((M, N), dtype=torch.float32, device=Xq.device) if Y is None else Y
    _want(Y, torch.float32, "Y", (M, N))
    if acc_out is not None:
        _want(acc_out, torch.int32, "acc_out", (M, N))
    nbytes = w4a8_workspace_bytes(M, K, N)
    ws = _workspace(nbytes, Xq.device, ws)
    _check(lib().w4a8_gemv(_ptr(Xq), _ptr(sa), M, K, _ptr(Wq), _ptr(sw), N, _ptr(Y), _ptr(acc_out),
                           _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), flags,
                           _stream(Xq)))
    return Y


def _prefetch_arg(prefetch, prefetch_bytes):
    if prefetch is None:
        return None, 0
    if not isinstance(prefetch, torch.Tensor) or not prefetch.is_cuda:
        raise TypeError("prefetch must be a CUDA tensor")
    nb = prefetch.numel() * prefetch.element_size()
    return prefetch.data_ptr(), min(nb, int(prefetch_bytes) if prefetch_bytes else nb)


def w4a8_linear(X, Wq, sw, Y=None, Xq_out=None, sa_out=None, acc_out=None, ws=None,
                flags: int = 0, prefetch=None, prefetch_bytes: int = 0):
    """Fused activation quantization + W4A8 product; returns Y.  `prefetch`
    (a CUDA tensor, e.g. the next launch's packed weights) and
    `prefetch_bytes` (0 = all of it): an L2 prefetch hint for the next
    launch (w4a8_linear_prefetch; the optional outputs are then not taken)."""
    _want(X, torch.float16, "X")
    M, K = X.shape
    N = Wq.shape[0]
    _want(Wq, torch.uint8, "Wq", (N, K // 2))
    _want(sw, torch.float32, "sw", (N,))
    Y = torch.empty((M, N), dtype=torch.float32, device=X.device) if Y is None else Y
    _want(Y, torch.float32, "Y", (M, N))
    if Xq_out is not None:
        _want(Xq_out, torch.int8, "Xq_out", (M, K))
    if sa_out is not None:
        _want(sa_out, torch.float32, "sa_out", (M,))
    if acc_out is not None:
        _want(acc_out, torch.int32, "acc_out", (M, N))
    nbytes = w4a8_workspace_bytes(M, K, N)
    ws = _workspace(nbytes, X.device, ws)
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    if prefetch is not None:
        if Xq_out is not None or sa_out is not None or acc_out is not None:
            raise ValueError("the prefetching call takes no optional outputs")
        pp, pb = _prefetch_arg(prefetch, prefetch_bytes)
        _check(lib().w4a8_linear_prefetch(_ptr(X), M, K, _ptr(Wq), _ptr(sw), N, _ptr(Y), _ptr(ws), wsb,
                                          flags, _stream(X), pp, pb))
        return Y
    _check(lib().w4a8_linear(_ptr(X), M, K, _ptr(Wq), _ptr(sw), N, _ptr(Y), _ptr(Xq_out),
                             _ptr(sa_out), _ptr(acc_out), _ptr(ws), wsb, flags, _stream(X)))
    return Y


def w4a8_linear_grouped(X, Wqs, sws, Ys=None, ws=None, flags: int = 0, prefetch=None,
                        prefetch_bytes: int = 0):
    """One launch for several weight matrices sharing X (e.g. q/k/v); returns
    the list of outputs, each bit-identical to w4a8_linear on its own.
    `prefetch`, `prefetch_bytes`: as in w4a8_linear."""
    _want(X, torch.float16, "X")
    M, K = X.shape
    G = len(Wqs)
    if G != len(sws) or not 1 <= G <= 4:
        raise ValueError("need 1..4 weight matrices with one scale vector each")
    Ns = [int(w.shape[0]) for w in Wqs]
    for g in range(G):
        _want(Wqs[g], torch.uint8, "Wq[%d]" % g, (Ns[g], K // 2))
        _want(sws[g], torch.float32, "sw[%d]" % g, (Ns[g],))
    if Ys is None:
        Ys = [torch.empty((M, n), dtype=torch.float32, device=X.device) for n in Ns]
    for g in range(G):
        _want(Ys[g], torch.float32, "Y[%d]" % g, (M, Ns[g]))
    arr_p = ctypes.c_void_p * G
    wq_a = arr_p(*[w.data_ptr() for w in Wqs])
    sw_a = arr_p(*[s.data_ptr() for s in sws])
    y_a = arr_p(*[y.data_ptr() for y in Ys])
    n_a = (ctypes.c_int64 * G)(*Ns)
    nbytes = w4a8_workspace_bytes(M, K, sum(Ns))
    ws = _workspace(nbytes, X.device, ws)
    wsb = 0 if ws is None else ws.numel() * ws.element_size()
    args = (_ptr(X), M, K, G, ctypes.cast(wq_a, ctypes.c_void_p), ctypes.cast(sw_a, ctypes.c_void_p),
            ctypes.cast(n_a, ctypes.c_void_p), ctypes.cast(y_a, ctypes.c_void_p), _ptr(ws), wsb, flags,
            _stream(X))
    if prefetch is not None:
        pp, pb = _prefetch_arg(prefetch, prefetch_bytes)
        _check(lib().w4a8_linear_grouped_prefetch(*args, pp, pb))
    else:
        _check(lib().w4a8_linear_grouped(*args))
    return Ys


def w4a8_linear_noalloc(X, Wq, sw, Y=None, flags: int = 0):
    """w4a8_linear for callers that cannot provide workspace memory: the
    split-K scratch is the library's static per-GPU array (see the C header
    for its limit and for why calls overlapping on the GPU must be avoided).
    Allocates nothing when Y is given."""
    _want(X, torch.float16, "X")
    M, K = X.shape
    N = Wq.shape[0]
    _want(Wq, torch.uint8, "Wq", (N, K // 2))
    _want(sw, torch.float32, "sw", (N,))
    Y = torch.empty((M, N), dtype=torch.float32, device=X.device) if Y is None else Y
    _want(Y, torch.float32, "Y", (M, N))
    _check(lib().w4a8_linear_noalloc(_ptr(X), M, K, _ptr(Wq), _ptr(sw), N, _ptr(Y), flags,
                                     _stream(X)))
    return Y


def w8a16_gemv(X, Wq8, sw16, Y=None, ws=None, flags: int = 0):
    """Y[m][n] = float(sw16[n]) * sum_k q[n,k] * x[m,k]; returns Y."""
    _want(X, torch.float16, "X")
    M, K = X.shape
    N = Wq8.shape[0]
    _want(Wq8, torch.int8, "Wq8", (N, K))
    _want(sw16, torch.float16, "sw16", (N,))
    Y = torch.empty((M, N), dtype=torch.float32, device=X.device) if Y is None else Y
    _want(Y, torch.float32, "Y", (M, N))
    nbytes = w8a16_workspace_bytes(M, K, N)
    ws = _workspace(nbytes, X.device, ws)
    _check(lib().w8a16_gemv(_ptr(X), M, K, _ptr(Wq8), _ptr(sw16), N, _ptr(Y), _ptr(ws),
                            0 if ws is None else ws.numel() * ws.element_size(), flags,
                            _stream(X)))
    return Y


# -- the MLP's gated product ---------------------------------------------------

def w4_interleave_rows(Wq_a, sw_a, Wq_b, sw_b, Wq_out=None, sw_out=None):
    """Rows of two packed matrices interleaved: (Wq [2N][K/2], sw [2N])."""
    N, half = Wq_a.shape
    for t, dt, nm, shp in ((Wq_a, torch.uint8, "Wq_a", (N, half)), (Wq_b, torch.uint8, "Wq_b", (N, half)),
                           (sw_a, torch.float32, "sw_a", (N,)), (sw_b, torch.float32, "sw_b", (N,))):
        _want(t, dt, nm, shp)
    Wq_out = torch.empty((2 * N, half), dtype=torch.uint8, device=Wq_a.device) if Wq_out is None else Wq_out
    sw_out = torch.empty((2 * N,), dtype=torch.float32, device=Wq_a.device) if sw_out is None else sw_out
    _want(Wq_out, torch.uint8, "Wq_out", (2 * N, half))
    _want(sw_out, torch.float32, "sw_out", (2 * N,))
    _check(lib().w4_interleave_rows(_ptr(Wq_a), _ptr(sw_a), _ptr(Wq_b), _ptr(sw_b), N, 2 * half,
                                    _ptr(Wq_out), _ptr(sw_out), _stream(Wq_a)))
    return Wq_out, sw_out


def w4a8_gate_up_silu_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().w4a8_gate_up_silu_workspace_bytes(M, K, N))


def w4a8_gate_up_silu(X, Wq_gu, sw_gu, H=None, Y_gu=None, ws=None, flags: int = 0):
    """Gate/up projections of interleaved weights with the gated product in
    the epilogue; returns (H [M][N] fp16, Y_gu [M][2N] fp32)."""
    _want(X, torch.float16, "X")
    M, K = X.shape
    N2 = Wq_gu.shape[0]
    if N2 % 2:
        raise ValueError("Wq_gu must have an even number of rows (gate/up pairs)")
    N = N2 // 2
    _want(Wq_gu, torch.uint8, "Wq_gu", (N2, K // 2))
    _want(sw_gu, torch.float32, "sw_gu", (N2,))
    H = torch.empty((M, N), dtype=torch.float16, device=X.device) if H is None else H
    Y_gu = torch.empty((M, N2), dtype=torch.float32, device=X.device) if Y_gu is None else Y_gu
    _want(H, torch.float16, "H", (M, N))
    _want(Y_gu, torch.float32, "Y_gu", (M, N2))
    ws = _workspace(w4a8_gate_up_silu_workspace_bytes(M, K, N), X.device, ws)
    _check(lib().w4a8_gate_up_silu(_ptr(X), M, K, _ptr(Wq_gu), _ptr(sw_gu), N, _ptr(Y_gu), _ptr(H), _ptr(ws),
                                   0 if ws is None else ws.numel() * ws.element_size(), flags, _stream(X)))
    return H, Y_gu


def w4a8_silu_mul(g, u, H=None, flags: int = 0):
    """H = fp16(silu(g) * u), g and u [M][N] fp32; returns H."""
    _want(g, torch.float32, "g")
    M, N = g.shape
    _want(u, torch.float32, "u", (M, N))
    H = torch.empty((M, N), dtype=torch.float16, device=g.device) if H is None else H
    _want(H, torch.float16, "H", (M, N))
    _check(lib().w4a8_silu_mul(_ptr(g), _ptr(u), M, N, _ptr(H), flags, _stream(g)))
    return H


# -- group-wise INT4 scales -------------------------------------------------

def w4g_scale_stride(K: int, group: int) -> int:
    """Floats per row of the group-scale matrix: K/group rounded up to a
    multiple of 4 (the W4G_SCALE_STRIDE layout of the C header)."""
    return (K // group + 3) // 4 * 4


def w4g_quantize_weights(W: torch.Tensor, group: int, Wq=None, sg=None):
    """W [N][K] fp32 -> (Wq [N][K/2] uint8, sg [N][stride] fp32)."""
    _want(W, torch.float32, "W")
    N, K = W.shape
    ld = w4g_scale_stride(K, group) if group > 0 else 0
    Wq = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device) if Wq is None else Wq
    sg = torch.empty((N, ld), dtype=torch.float32, device=W.device) if sg is None else sg
    _want(Wq, torch.uint8, "Wq", (N, K // 2))
    _want(sg, torch.float32, "sg", (N, ld))
    _check(lib().w4g_quantize_weights(_ptr(W), N, K, group, _ptr(Wq), _ptr(sg), _stream(W)))
    return Wq, sg


def w4a8g_workspace_bytes(M: int, K: int, N: int, group: int) -> int:
    return int(lib().w4a8g_workspace_bytes(M, K, N, group))


def _want_group(Wq, sg, N, K, group, name=""):
    _want(Wq, torch.uint8, "Wq" + name, (N, K // 2))
    _want(sg, torch.float32, "sg" + name, (N, w4g_scale_stride(K, group) if group > 0 else 0))


def w4a8g_gemv(Xq, sa, Wq, sg, group: int, Y=None, ws=None, flags: int = 0):
    """Y[m][n] = sa[m] * sum_g sg[n][g] * acc_g[m][n] (group-wise scales); returns Y."""
    _want(Xq, torch.int8, "Xq")
    M, K = Xq.shape
    N = Wq.shape[0]
    _want(sa, torch.float32, "sa", (M,))
    _want_group(Wq, sg, N, K, group)
    Y = torch.empty((M, N), dtype=torch.float32, device=Xq.device) if Y is None else Y
    _want(Y, torch.float32, "Y", (M, N))
    ws = _workspace(w4a8g_workspace_bytes(M, K, N, group), Xq.device, ws)
    _check(lib().w4a8g_gemv(_ptr(Xq), _ptr(sa), M, K, group, _ptr(Wq), _ptr(sg), N, _ptr(Y),
                            _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(), flags,
                            _stream(Xq)))
    return Y


def w4a8g_linear(X, Wq, sg, group: int, Y=None, Xq_out=None, sa_out=None, ws=None,
                 flags: int = 0):
    """Fused activation quantization + group-scale W4A8 product; returns Y."""
    _want(X, torch.float16, "X")
    M, K = X.shape
    N = Wq.shape[0]
    _want_group(Wq, sg, N, K, group)
    Y = torch.empty((M, N), dtype=torch.float32, device=X.device) if Y is None else Y
    _want(Y, torch.float32, "Y", (M, N))
    if Xq_out is not None:
        _want(Xq_out, torch.int8, "Xq_out", (M, K))
    if sa_out is not None:
        _want(sa_out, torch.float32, "sa_out", (M,))
    ws = _workspace(w4a8g_workspace_bytes(M, K, N, group), X.device, ws)
    _check(lib().w4a8g_linear(_ptr(X), M, K, group, _ptr(Wq), _ptr(sg), N, _ptr(Y),
                              _ptr(Xq_out), _ptr(sa_out), _ptr(ws),
                              0 if ws is None else ws.numel() * ws.element_size(), flags,
                              _stream(X)))
    return Y


def w4a8g_linear_grouped(X, Wqs, sgs, group: int, Ys=None, ws=None, flags: int = 0):
    """One launch for several group-scale weight matrices sharing X; returns
    the list of outputs."""
    _want(X, torch.float16, "X")
    M, K = X.shape
    G = len(Wqs)
    if G != len(sgs) or not 1 <= G <= 4:
        raise ValueError("need 1..4 weight matrices with one scale matrix each")
    Ns = [int(w.shape[0]) for w in Wqs]
    for g in range(G):
        _want_group(Wqs[g], sgs[g], Ns[g], K, group, "[%d]" % g)
    if Ys is None:
        Ys = [torch.empty((M, n), dtype=torch.float32, device=X.device) for n in Ns]
    for g in range(G):
        _want(Ys[g], torch.float32, "Y[%d]" % g, (M, Ns[g]))
    arr_p = ctypes.c_void_p * G
    wq_a = arr_p(*[w.data_ptr() for w in Wqs])
    sg_a = arr_p(*[t.data_ptr() for t in sgs])
    y_a = arr_p(*[y.data_ptr() for y in Ys])
    n_a = (ctypes.c_int64 * G)(*Ns)
    ws = _workspace(w4a8g_workspace_bytes(M, K, sum(Ns), group), X.device, ws)
    _check(lib().w4a8g_linear_grouped(_ptr(X), M, K, group, G, ctypes.cast(wq_a, ctypes.c_void_p),
                                      ctypes.cast(sg_a, ctypes.c_void_p),
                                      ctypes.cast(n_a, ctypes.c_void_p),
                                      ctypes.cast(y_a, ctypes.c_void_p), _ptr(ws),
                                      0 if ws is None else ws.numel() * ws.element_size(), flags,
                                      _stream(X)))
    return Ys


# -- IndexSoftmax -------------------------------------------------------------

ISX_DEFAULT_B = 5
ISX_DEFAULT_C = 6.6


def index_softmax_lut(b: int = ISX_DEFAULT_B, c: float = ISX_DEFAULT_C) -> bytes:
    """The 2^b-entry UINT8 exponent table (computed on the host)."""
    buf = (ctypes.c_uint8 * (1 << b))() if 1 <= b <= 8 else (ctypes.c_uint8 * 1)()
    _check(lib().index_softmax_lut(b, c, ctypes.cast(buf, ctypes.c_void_p)))
    return bytes(buf)


def index_softmax_c_int(c: float, d: int, s_q: float, s_k: float) -> int:
    v = int(lib().index_softmax_c_int(c, d, s_q, s_k))
    if v < 0:
        raise W4A8Error(ERR_SHAPE, "index_softmax_c_int: arguments out of range")
    return v


def index_softmax_u8(A, c_int: int, b: int = ISX_DEFAULT_B, lut: bytes = None, P=None):
    """int32 logits [rows][cols] (CUDA) -> UINT8 probabilities; returns P."""
    _want(A, torch.int32, "A")
    rows, cols = A.shape
    P = torch.empty((rows, cols), dtype=torch.uint8, device=A.device) if P is None else P
    _want(P, torch.uint8, "P", (rows, cols))
    lut = index_softmax_lut(b) if lut is None else bytes(lut)
    if len(lut) != (1 << b):
        raise ValueError("lut must have 2^b entries")
    lut_buf = (ctypes.c_uint8 * len(lut)).from_buffer_copy(lut)
    _check(lib().index_softmax_u8(_ptr(A), rows, cols, c_int, b,
                                  ctypes.cast(lut_buf, ctypes.c_void_p), _ptr(P), _stream(A)))
    return P


# -- the decoder layer around the linears --------------------------------------

_F32, _F16 = 0, 1
_TYPES = {torch.float32: _F32, torch.float16: _F16}


def _want_type(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if t.dtype not in _TYPES:
        raise TypeError("%s must be float32 or float16, got %s" % (name, t.dtype))
    return _TYPES[t.dtype]


def add_norm(r, w=None, y=None, post_w=None, gate=None, alpha: float = 1.0, beta: float = 1.0, eps: float = 1e-6,
             r_out=None, X=None, Xq=None, sa=None, codes: bool = False, flags: int = 0):
    """Residual update with the norms on both sides of it:
    r' = alpha * r + beta * gate * u, u = y or rmsnorm(y) * post_w;
    X = fp16(rmsnorm(r') * w).

    r [M][N] fp32 or fp16; y (a linear's output) alike, any of the two types;
    post_w, w [N] fp32; gate [N] or [M][N] fp32.  Returns (r', X), r' of r's
    type (r_out may be r); with codes=True (r', X, Xq, sa), the INT8
    activation of X as act_quantize_i8 gives it.  Without w: (r', None)."""
    rt = _want_type(r, "r")
    _want(r, r.dtype, "r")
    shape = r.shape
    if len(shape) != 2:
        raise ValueError("r must have two dimensions")
    M, N = shape
    yt = ld_gate = 0
    yp = pp = gp = wp = xp = qp = sp = None
    if y is not None:
        yt = _want_type(y, "y")
        _want(y, y.dtype, "y", shape)
        yp = y.data_ptr()
    elif post_w is not None or gate is not None:
        raise ValueError("post_w and gate need y")
    if post_w is not None:
        _want(post_w, torch.float32, "post_w", (N,))
        pp = post_w.data_ptr()
    if gate is not None:
        _want(gate, torch.float32, "gate", (N,) if gate.dim() == 1 else shape)
        ld_gate = N if gate.dim() == 2 else 0
        gp = gate.data_ptr()
    if r_out is None:
        r_out = torch.empty_like(r)
    else:
        _want(r_out, r.dtype, "r_out", shape)
    if w is not None:
        _want(w, torch.float32, "w", (N,))
        wp = w.data_ptr()
        if X is None:
            X = torch.empty_like(r, dtype=torch.float16)
        else:
            _want(X, torch.float16, "X", shape)
        xp = X.data_ptr()
        if codes or Xq is not None or sa is not None:
            Xq = torch.empty_like(r, dtype=torch.int8) if Xq is None else Xq
            sa = torch.empty((M,), dtype=torch.float32, device=r.device) if sa is None else sa
            _want(Xq, torch.int8, "Xq", shape)
            _want(sa, torch.float32, "sa", (M,))
            qp, sp = Xq.data_ptr(), sa.data_ptr()
    elif X is not None or codes or Xq is not None or sa is not None:
        raise ValueError("X and its codes need w")
    _check(lib().add_norm(r.data_ptr(), rt, yp, yt, pp, gp, ld_gate, wp, M, N, alpha, beta, eps, r_out.data_ptr(), xp,
                          qp, sp, flags, _stream(r)))
    return (r_out, X) if Xq is None else (r_out, X, Xq, sa)


ROPE_SCALINGS = {None: 0, "plain": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}


def rope_frequencies(rot: int, base: float = 10000.0, scaling=None, factor: float = 1.0, old_ctx: float = 0.0,
                     low: float = 1.0, high: float = 32.0, device=None):
    """(freqs [rot/2] float64 tensor, mscale): the rotary frequencies, plain or
    scaled for long contexts ("linear", "ntk", "yarn", "bands").  Computed on
    the host; `device` places the tensor."""
    if scaling not in ROPE_SCALINGS:
        raise ValueError("scaling must be one of %s" % ", ".join(str(k) for k in ROPE_SCALINGS))
    buf = (ctypes.c_double * 128)()
    ms = ctypes.c_float(1.0)
    _check(lib().rope_frequencies(rot, base, ROPE_SCALINGS[scaling], factor, old_ctx, low, high,
                                  ctypes.cast(buf, ctypes.c_void_p), ctypes.byref(ms)))
    return torch.tensor(buf[:rot // 2], dtype=torch.float64, device=device), float(ms.value)


def _want_heads(t, name, shape=None):
    """[tokens][heads][dim], the last two dimensions contiguous, rows at any
    distance (a slice of a fused projection); returns the row distance."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    have = t.shape
    if len(have) != 3:
        raise ValueError("%s must be [tokens][heads][dim]" % name)
    if shape is not None and have != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(have)))
    n, h, d = have
    if t.is_contiguous():
        return h * d
    st = t.stride()
    if st[2] != 1 or (st[1] != d and h > 1):
        raise ValueError("%s: the heads of a row must be contiguous" % name)
    return st[0] if n > 1 else max(st[0], h * d)


def _want_rope(pos, freqs, tokens, axis=None):
    """rot and, with `axis` (the axis of each pair), (axes, axis as bytes)"""
    _want(freqs, torch.float64, "freqs")
    if freqs.dim() != 1:
        raise ValueError("freqs must have one dimension")
    pairs = freqs.shape[0]
    if axis is None:
        _want(pos, torch.int32, "pos", (tokens,))
        return 2 * pairs, None
    if not isinstance(axis, bytes):
        axis = bytes(int(a) for a in axis)
    if len(axis) != pairs:
        raise ValueError("axis must have one entry for each of the %d pairs, got %d" % (pairs, len(axis)))
    _want(pos, torch.int32, "pos")
    if pos.dim() != 2 or pos.shape[1] != tokens:
        raise ValueError("pos must be [axes][%d]" % tokens)
    return 2 * pairs, (pos.shape[0], axis)


def rope_axes(sections, cycled: bool = False) -> bytes:
    """The axis of each pair for rotary positions with several axes: `sections`
    gives the pairs of each axis (time, height, width), in blocks one after the
    other, or, cycled, the axes in turn for as long as each has pairs left."""
    sections = [int(n) for n in sections]
    if not 1 <= len(sections) <= 4 or min(sections) < 0:
        raise ValueError("sections must be 1 to 4 counts of pairs")
    if not cycled:
        return bytes(a for a, n in enumerate(sections) for _ in range(n))
    return bytes(a for i in range(max(sections)) for a, n in enumerate(sections) if i < n)


def rope_rotate(X, pos, freqs, interleaved: bool = False, mscale: float = 1.0, Y=None, dtype=None, flags: int = 0,
                axis=None):
    """Rotary positions on X [tokens][heads][dim] (fp32 or fp16, rows at any
    distance): pairs (i, i + rot/2), or (2i, 2i + 1) when interleaved, turned by
    pos * freqs[i]; rot = 2 * len(freqs).  With axis (rope_axes, or any sequence
    of len(freqs) numbers) pos is [axes][tokens] and pair i turns by
    pos[axis[i]] * freqs[i].  Returns Y (Y may be X)."""
    xt = _want_type(X, "X")
    ld = _want_heads(X, "X")
    n, h, d = X.shape
    rot, axes = _want_rope(pos, freqs, n, axis)
    if Y is None:
        Y = torch.empty((n, h, d), dtype=dtype or X.dtype, device=X.device)
    yt = _want_type(Y, "Y")
    ld_y = _want_heads(Y, "Y", X.shape)
    if axes is not None:
        _check(lib().rope_rotate_axes(_ptr(X), xt, ld, n, h, d, _ptr(pos), *axes, _ptr(freqs), rot, int(interleaved),
                                      mscale, _ptr(Y), yt, ld_y, flags, _stream(X)))
        return Y
    _check(lib().rope_rotate(_ptr(X), xt, ld, n, h, d, _ptr(pos), _ptr(freqs), rot, int(interleaved), mscale,
                             _ptr(Y), yt, ld_y, flags, _stream(X)))
    return Y


# Pages of quantized keys and values: k, v int8 [pages][heads][page][dim] (8
# bits) or uint8 [pages][heads][page][dim/2] (4 bits), ks, vs fp32
# [pages][heads][page].
KVQCache = collections.namedtuple("KVQCache", "k v ks vs")
# The tokens of a call: cu int32 [seqs + 1], start int32 [seqs], table int32
# [seqs][max_pages] (kvq_batch_t in the C header).
KVQBatch = collections.namedtuple("KVQBatch", "cu start table")


def kvq_cache(pages: int, page: int, heads: int, dim: int, bits: int = 8, device="cuda") -> KVQCache:
    """An empty cache."""
    if bits not in (8, 4):
        raise ValueError("bits must be 8 or 4")
    dt, width = (torch.int8, dim) if bits == 8 else (torch.uint8, dim // 2)
    k, v = (torch.zeros((pages, heads, page, width), dtype=dt, device=device) for _ in range(2))
    ks, vs = (torch.zeros((pages, heads, page), dtype=torch.float32, device=device) for _ in range(2))
    return KVQCache(k, v, ks, vs)


_pack_cache = struct.Struct("@4Pq4i").pack   # kvq_cache_t
_pack_batch = struct.Struct("@3P3q").pack    # kvq_batch_t


def _cache_arg(c):
    """(kvq_cache_t as bytes, heads, dim)"""
    k, v, ks, vs = c
    if not isinstance(k, torch.Tensor) or k.dtype not in (torch.int8, torch.uint8):
        raise TypeError("the cache's codes must be int8 (8 bits) or uint8 (4 bits) tensors")
    if k.dim() != 4:
        raise ValueError("the cache's codes must be [pages][heads][page][dim]")
    shape = k.shape
    _want(k, k.dtype, "k")
    _want(v, k.dtype, "v", shape)
    _want(ks, torch.float32, "ks", shape[:3])
    _want(vs, torch.float32, "vs", shape[:3])
    pages, heads, page, width = shape
    bits = 8 if k.dtype is torch.int8 else 4
    dim = width * 8 // bits
    return _pack_cache(k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), pages, page, heads, dim, bits), heads, dim


def _batch_arg(b, tokens):
    """kvq_batch_t as bytes"""
    cu, start, table = b
    _want(cu, torch.int32, "cu")
    _want(start, torch.int32, "start")
    _want(table, torch.int32, "table")
    cs, ss, ts = cu.shape, start.shape, table.shape
    if len(cs) != 1 or len(ss) != 1 or len(ts) != 2 or cs[0] != ss[0] + 1 or ts[0] != ss[0]:
        raise ValueError("the batch must be cu [seqs + 1], start [seqs], table [seqs][max_pages]")
    return _pack_batch(cu.data_ptr(), start.data_ptr(), table.data_ptr(), ss[0], tokens, ts[1])


def kvq_write(cache, batch, K, V, Q=None, pos=None, freqs=None, interleaved: bool = False, mscale: float = 1.0,
              Q_out=None, flags: int = 0, axis=None):
    """Writes K, V [tokens][heads][dim] (fp32 or fp16, rows at any distance) into
    the cache, rotated first when freqs is given, and rotates Q
    [tokens][heads_q][dim] in the same launch; returns Q_out (fp16; None without Q).
    axis: positions with several axes, as in rope_rotate."""
    ca, heads, dim = _cache_arg(cache)
    xt = _want_type(K, "K")
    n = K.shape[0]
    shape = (n, heads, dim)
    ld_k, ld_v = _want_heads(K, "K", shape), _want_heads(V, "V", shape)
    if V.dtype != K.dtype or (Q is not None and Q.dtype != K.dtype):
        raise TypeError("Q, K and V must have one type")
    ba = _batch_arg(batch, n)
    if axis is not None and freqs is None:
        raise ValueError("axis needs freqs")
    rot, axes = _want_rope(pos, freqs, n, axis) if freqs is not None else (0, None)
    hq = ld_q = 0
    if Q is not None:
        hq = Q.shape[1]
        ld_q = _want_heads(Q, "Q", (n, hq, dim))
        Q_out = torch.empty((n, hq, dim), dtype=torch.float16, device=K.device) if Q_out is None else Q_out
        _want(Q_out, torch.float16, "Q_out", (n, hq, dim))
    elif Q_out is not None:
        raise ValueError("Q_out needs Q")
    if axes is not None:
        _check(lib().kvq_write_axes(ca, ba, _ptr(K), ld_k, _ptr(V), ld_v, _ptr(Q), ld_q, hq, xt, _ptr(pos), *axes,
                                    _ptr(freqs), rot, int(interleaved), mscale, _ptr(Q_out), flags, _stream(K)))
        return Q_out
    _check(lib().kvq_write(ca, ba, _ptr(K), ld_k, _ptr(V), ld_v, _ptr(Q), ld_q, hq, xt,
                           _ptr(pos), _ptr(freqs), rot, int(interleaved), mscale, _ptr(Q_out), flags, _stream(K)))
    return Q_out


def kvq_read(cache, batch, tokens: int, dtype=torch.float16, K=None, V=None, flags: int = 0):
    """The batch's keys and values (tokens = cu[-1]) as values:
    (K, V) [tokens][heads][dim], fp16 or fp32."""
    ca, heads, dim = _cache_arg(cache)
    ba = _batch_arg(batch, tokens)
    shape = (tokens, heads, dim)
    K = torch.empty(shape, dtype=dtype, device=cache[0].device) if K is None else K
    V = torch.empty(shape, dtype=K.dtype, device=cache[0].device) if V is None else V
    yt = _want_type(K, "K")
    _want(K, K.dtype, "K", shape)
    _want(V, K.dtype, "V", shape)
    _check(lib().kvq_read(ca, ba, _ptr(K), _ptr(V), yt, flags, _stream(K)))
    return K, V


def kvq_keep(cache, batch, keep, flags: int = 0):
    """Moves a drafted tree's accepted tokens together: slot start[b] + i takes
    what slot start[b] + keep[cu[b] + i] held, until an entry is negative."""
    ca, heads, dim = _cache_arg(cache)
    _want(keep, torch.int32, "keep")
    if keep.dim() != 1:
        raise ValueError("keep must have one dimension")
    ba = _batch_arg(batch, keep.shape[0])
    _check(lib().kvq_keep(ca, ba, _ptr(keep), flags, _stream(keep)))


def kvq_attention_workspace_bytes(cache, batch, tokens: int, heads_q: int) -> int:
    ca, ba = _cache_arg(cache)[0], _batch_arg(batch, tokens)
    return int(lib().kvq_attention_workspace_bytes(ca, ba, heads_q))


_attn_ws = {}
_TICKET_BYTES = 4096  # arrival counters at a workspace's start (w4a8_workspace_bytes)


def _stream_workspace(device, stream: int, nbytes: int = 0):
    """A stream's workspace (its arrival counters zeroed), made anew when
    `nbytes` asks for more; under graph capture one of the graph's own, so that
    replays share nothing with eager calls."""
    capturing = torch.cuda.is_current_stream_capturing()
    if nbytes == 0:
        return None if capturing else _attn_ws.get((device, stream))
    buf = torch.empty(nbytes if capturing else max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
    buf[:_TICKET_BYTES].zero_()
    if not capturing:
        _attn_ws[(device, stream)] = buf
    return buf


def kvq_attention(Q, cache, batch, mask=None, scale: float = None, out=None, ws=None, flags: int = 0):
    """Attention of Q [tokens][heads_q][dim] fp16 over the cache; returns out
    (same shape, fp16).  Every token sees its sequence's start[b] cached slots and
    of the call's own tokens those whose bit is set in mask [tokens] (int64 as 64
    bits; a tree's ancestors and itself), or without mask those up to itself.
    scale: 1 / sqrt(dim) by default."""
    ca, heads, dim = _cache_arg(cache)
    _want(Q, torch.float16, "Q")
    if Q.dim() != 3 or Q.shape[2] != dim:
        raise ValueError("Q must be [tokens][heads_q][%d]" % dim)
    n, hq, d = Q.shape
    ba = _batch_arg(batch, n)
    if mask is not None:
        _want(mask, torch.int64, "mask", (n,))
    if out is None:
        out = torch.empty_like(Q)
    else:
        _want(out, torch.float16, "out", Q.shape)
    L = lib()
    stream = _stream(Q)
    mine = ws is None
    if mine:
        ws = _stream_workspace(Q.device, stream)
    mp = None if mask is None else mask.data_ptr()
    scale = d ** -0.5 if scale is None else scale
    while True:
        st = L.kvq_attention(ca, ba, Q.data_ptr(), hq, mp, scale, out.data_ptr(), _ptr(ws),
                             0 if ws is None else ws.numel() * ws.element_size(), flags, stream)
        if st != ERR_WORKSPACE or not mine:
            break
        ws, mine = _stream_workspace(Q.device, stream, int(L.kvq_attention_workspace_bytes(ca, ba, hq))), False
    _check(st)
    return out


# --------------------------------------------------------------------------
# a serving step around the layers
# --------------------------------------------------------------------------

_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device_of(t, name):
    """The index of the tensor's device, which has to be the current one: the call runs
    on its current stream."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    d = t.get_device()
    if d < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    if d != _current_device():
        raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, d, _current_device()))
    return d


def _arg(t, dtype, shape, name, dev):
    """The address of a contiguous tensor of that type, shape and device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.shape == shape and \
            t.is_contiguous():
        return t.data_ptr()
    _want(t, dtype, name, shape)
    raise ValueError("all tensors must be on one device (%s is on %s)" % (name, t.device))


def _optional(t, dtype, shape, name, dev):
    return None if t is None else _arg(t, dtype, shape, name, dev)


def _out(t, dtype, shape, name, dev, like):
    """(tensor, address) of an output: the caller's, or a new one beside `like`."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=like.device)
        return t, t.data_ptr()
    return t, _arg(t, dtype, shape, name, dev)


def _scratch(ws, nbytes, like):
    """The caller's workspace as (tensor, bytes), or one of this call's own: the allocator
    hands it on in the stream's order (in a captured graph: within the graph)."""
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device), nbytes
    if not isinstance(ws, torch.Tensor) or ws.get_device() != like.get_device():
        raise ValueError("ws must be a tensor on the device of the others")
    return ws, ws.numel() * ws.element_size()


# The pages of a pool and who holds them: table int32 [seqs][max_pages], held
# int32 [seqs], stack int32 [pages], top int32 [1] (kvq_pool_t in the C header).
KVQPool = collections.namedtuple("KVQPool", "table held stack top")

_pack_pool = struct.Struct("@4P3qi").pack   # kvq_pool_t


def kvq_pool(seqs: int, max_pages: int, pages: int, device="cuda") -> KVQPool:
    """A pool whose pages are all free, for up to `seqs` requests of up to max_pages pages."""
    table = torch.full((seqs, max_pages), -1, dtype=torch.int32, device=device)
    held = torch.zeros((seqs,), dtype=torch.int32, device=device)
    stack = torch.arange(pages, dtype=torch.int32, device=device)
    return KVQPool(table, held, stack, torch.full((1,), pages, dtype=torch.int32, device=device))


def _pool_arg(p, page, dev):
    """(kvq_pool_t as bytes, seqs)"""
    table, held, stack, top = p
    if not isinstance(table, torch.Tensor) or not isinstance(stack, torch.Tensor):
        raise TypeError("the pool's arrays must be torch tensors")
    if table.dim() != 2 or stack.dim() != 1:
        raise ValueError("the pool must be table [seqs][max_pages], held [seqs], stack [pages], top [1]")
    (seqs, width), pages = table.shape, stack.shape[0]
    i32 = torch.int32
    return _pack_pool(_arg(table, i32, (seqs, width), "table", dev), _arg(held, i32, (seqs,), "held", dev),
                      _arg(stack, i32, (pages,), "stack", dev), _arg(top, i32, (1,), "top", dev), seqs, width, pages,
                      page), seqs


def kvq_plan_workspace_bytes(pool, page: int) -> int:
    return int(lib().kvq_plan_workspace_bytes(_pool_arg(pool, page, _device_of(pool[0], "table"))[0]))


def kvq_plan(pool, page: int, lens, add, tokens: int, grow=None, mask=None, cu=None, pos=None, slot=None, seq=None,
             ws=None, flags: int = 0):
    """Plans a step of up to `tokens` tokens: lens [seqs] int32 += grow, requests
    with add[b] < 0 end and give their pages back, those with add[b] > 0 take the
    pages they lack (or wait, if these or the tokens do not reach).  Returns
    (KVQBatch(cu, lens, pool.table), pos, slot, seq): positions int32 (with mask
    [tokens] int64: by depth in the drafted tree), rows of the pool int64 and
    rows of the batch int32 of the step's tokens.  mask lies as add asks, those
    that wait included; token t of row b is at[b] + t - cu[b] of such a layout, at =
    the sums of max(add, 0) before each row."""
    dev = _device_of(lens, "lens")
    pa, seqs = _pool_arg(pool, page, dev)
    i32, n = torch.int32, (seqs,)
    lp, ap, gp = _arg(lens, i32, n, "lens", dev), _arg(add, i32, n, "add", dev), _optional(grow, i32, n, "grow", dev)
    n = (tokens,)
    mp = _optional(mask, torch.int64, n, "mask", dev)
    cu, cp = _out(cu, i32, (seqs + 1,), "cu", dev, lens)
    pos, pp = _out(pos, i32, n, "pos", dev, lens)
    slot, tp = _out(slot, torch.int64, n, "slot", dev, lens)
    seq, qp = _out(seq, i32, n, "seq", dev, lens)
    L = lib()
    ws, wsb = _scratch(ws, L.kvq_plan_workspace_bytes(pa), lens)
    _check(L.kvq_plan(pa, lp, gp, ap, mp, tokens, cp, pp, tp, qp, ws.data_ptr(), wsb, flags, _stream(lens)))
    return KVQBatch(cu, lens, pool[0]), pos, slot, seq


def _want_rows(t, name, shape, dev):
    """[rows][cols] with contiguous columns, rows at any distance; returns the distance."""
    if t.get_device() != dev:
        raise ValueError("%s must be on the device of the others" % name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    n, v = shape
    if (v > 1 and t.stride(1) != 1) or (n > 1 and t.stride(0) < v):
        raise ValueError("%s: the values of a row must be contiguous, its rows apart" % name)
    return t.stride(0) if n > 1 else v


def draft_verify_workspace_bytes(tokens: int, vocab: int) -> int:
    return int(lib().draft_verify_workspace_bytes(tokens, vocab))


def draft_verify(logits, cu, ids, u, mask=None, q=None, temp=None, keep=None, out=None, count=None, ws=None,
                 flags: int = 0):
    """Which drafted tokens stay, and the next token of each sequence.

    logits [tokens][vocab] fp32 or fp16 (rows at any distance): the target's
    answers after each token of the batch, cu [seqs + 1] int32 its offsets; the
    first token of a sequence is certain, the others are drafts ids [tokens]
    int32, in a chain or, with mask [tokens] int64, a tree of ancestors' bits.
    q [tokens][vocab]: the probabilities that the children of each token were
    drawn from (None: the drafts are given).  u [tokens] fp32 in [0, 1): the
    random numbers of the tests, the root's that of the draw.  temp [seqs] fp32
    (None: 1; 0: greedy).  Returns (keep, out, count) int32: places kept (for
    kvq_keep), tokens said, how many of each (for kvq_plan's grow)."""
    lt = _want_type(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens][vocab]")
    dev = _device_of(logits, "logits")
    n, v = logits.shape
    ld = _want_rows(logits, "logits", (n, v), dev)
    if not isinstance(cu, torch.Tensor) or cu.dim() != 1 or cu.shape[0] < 2:
        raise ValueError("cu must be a tensor [seqs + 1]")
    seqs, i32, f32 = cu.shape[0] - 1, torch.int32, torch.float32
    cp, ip, up = _arg(cu, i32, (seqs + 1,), "cu", dev), _arg(ids, i32, (n,), "ids", dev), _arg(u, f32, (n,), "u", dev)
    mp, tp = _optional(mask, torch.int64, (n,), "mask", dev), _optional(temp, f32, (seqs,), "temp", dev)
    qt = ld_q = 0
    if q is not None:
        qt = _want_type(q, "q")
        ld_q = _want_rows(q, "q", (n, v), dev)
    keep, kp = _out(keep, i32, (n,), "keep", dev, ids)
    out, op = _out(out, i32, (n,), "out", dev, ids)
    count, np = _out(count, i32, (seqs,), "count", dev, ids)
    L = lib()
    ws, wsb = _scratch(ws, L.draft_verify_workspace_bytes(n, v), ids)
    _check(L.draft_verify(logits.data_ptr(), lt, ld, v, cp, seqs, n, ip, mp, _ptr(q), qt, ld_q, tp, up, kp, op, np,
                          ws.data_ptr(), wsb, flags, _stream(logits)))
    return keep, out, count


# --------------------------------------------------------------------------
# linear with 8-bit floating-point blocks of 128
# --------------------------------------------------------------------------

F8_BLOCK = 128


def _f8_blocks(n: int) -> int:
    return -(-n // F8_BLOCK)


def f8_quantize_weights(W, Wf=None, sw=None):
    """W [N][K] fp32 -> (Wf [N][K] uint8 (e4m3), sw [ceil(N/128)][ceil(K/128)] fp32)."""
    dev = _device_of(W, "W")
    if W.dim() != 2:
        raise ValueError("W must have two dimensions")
    N, K = W.shape
    wp = _arg(W, torch.float32, (N, K), "W", dev)
    blocks = (_f8_blocks(N), _f8_blocks(K))
    Wf, fp = _out(Wf, torch.uint8, (N, K), "Wf", dev, W)
    sw, sp = _out(sw, torch.float32, blocks, "sw", dev, W)
    _check(lib().f8_quantize_weights(wp, N, K, fp, sp, _stream(W)))
    return Wf, sw


def _f8_rows(X):
    """(type, M, K, address, device)"""
    xt = _want_type(X, "X")
    if X.dim() != 2:
        raise ValueError("X must have two dimensions")
    dev = _device_of(X, "X")
    M, K = X.shape
    return xt, M, K, _arg(X, X.dtype, (M, K), "X", dev), dev


def f8_quantize_rows(X, Xf=None, sa=None, flags: int = 0):
    """X [M][K] fp32 or fp16 -> (Xf [M][K] uint8 (e4m3), sa [ceil(K/128)][M] fp32)."""
    xt, M, K, xp, dev = _f8_rows(X)
    scales = (_f8_blocks(K), M)
    Xf, fp = _out(Xf, torch.uint8, (M, K), "Xf", dev, X)
    sa, sp = _out(sa, torch.float32, scales, "sa", dev, X)
    _check(lib().f8_quantize_rows(xp, xt, M, K, fp, sp, flags, _stream(X)))
    return Xf, sa


def _f8_weights(Wf, sw, K, dev):
    """(N, address of Wf, address of sw)"""
    if not isinstance(Wf, torch.Tensor) or Wf.dim() != 2 or Wf.shape[1] != K:
        raise ValueError("Wf must be a tensor [N][%d]" % K)
    N = Wf.shape[0]
    return N, _arg(Wf, torch.uint8, (N, K), "Wf", dev), _arg(sw, torch.float32, (_f8_blocks(N), _f8_blocks(K)), "sw", dev)


def _f8_out(Y, shape, dtype, like, dev):
    """(Y, type, address)"""
    if Y is not None:
        dtype = Y.dtype if isinstance(Y, torch.Tensor) else None
    if dtype not in _TYPES:
        raise TypeError("Y must be float32 or float16, got %s" % dtype)
    Y, yp = _out(Y, dtype, shape, "Y", dev, like)
    return Y, _TYPES[dtype], yp


def f8_linear_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib().f8_linear_workspace_bytes(M, K, N))


def f8_gemm(Xf, sa, Wf, sw, dtype=torch.float32, Y=None, flags: int = 0):
    """Y [M][N] (fp32 or fp16): the product of e4m3 codes with a scale for each row
    and 128 values of X and each 128 x 128 block of W."""
    dev = _device_of(Xf, "Xf")
    if Xf.dim() != 2:
        raise ValueError("Xf must have two dimensions")
    M, K = Xf.shape
    xp, ap = _arg(Xf, torch.uint8, (M, K), "Xf", dev), _arg(sa, torch.float32, (_f8_blocks(K), M), "sa", dev)
    N, wp, sp = _f8_weights(Wf, sw, K, dev)
    Y, yt, yp = _f8_out(Y, (M, N), dtype, Xf, dev)
    _check(lib().f8_gemm(xp, ap, M, K, wp, sp, N, yp, yt, flags, _stream(Xf)))
    return Y


def f8_linear(X, Wf, sw, dtype=torch.float32, Y=None, ws=None, flags: int = 0):
    """f8_quantize_rows and f8_gemm in one call: X [M][K] fp32 or fp16, any number
    of rows; Y [M][N] fp32 or fp16."""
    xt, M, K, xp, dev = _f8_rows(X)
    N, wp, sp = _f8_weights(Wf, sw, K, dev)
    Y, yt, yp = _f8_out(Y, (M, N), dtype, X, dev)
    L = lib()
    ws, wsb = _scratch(ws, L.f8_linear_workspace_bytes(M, K, N), X)
    _check(L.f8_linear(xp, xt, M, K, wp, sp, N, yp, yt, ws.data_ptr(), wsb, flags, _stream(X)))
    return Y


def w4a8_last_error() -> str:
    return lib().w4a8_last_error().decode(errors="replace")


def w4a8_device_error(device=None) -> int:
    """Reads and clears the device error word (synchronises the current stream)."""
    flags = ctypes.c_uint(0)
    stream = torch.cuda.current_stream(device).cuda_stream
    _check(lib().w4a8_device_error(ctypes.byref(flags), stream))
    return int(flags.value)


def w4a8_set_tuning(force_splits: int = 0, force_threads_per_row: int = 0,
                    ring_bytes: int = 0, ctas_per_sm: int = 0, mma_min_m: int = 0,
                    rowdot_max_m: int = 0, mma_e4m3: int = 0, qmma_max_m: int = 0,
                    qmma_tiles_per_warp: int = 0, stall_test_us: int = 0, qmma_operands: int = 0,
                    reset: bool = False):
    if reset:
        _check(lib().w4a8_set_tuning(None))
        return
    t = _Tuning(force_splits, force_threads_per_row, ring_bytes, ctas_per_sm, mma_min_m,
                rowdot_max_m, mma_e4m3, qmma_max_m, qmma_tiles_per_warp, stall_test_us, qmma_operands)
    _check(lib().w4a8_set_tuning(ctypes.byref(t)))


PLAN_FIELDS = ("splits", "threads_per_row", "cols_per_thread", "rows_per_stage", "ctas_per_split",
               "grid", "rows_per_cta", "stages", "stage_bytes", "smem_bytes", "ws_bytes",
               "kernel")


def w4a8_plan_info(M: int, K: int, N: int, w8a16: bool = False, num_sms: int = 0) -> dict:
    """Launch plan for a shape; num_sms > 0 plans without a GPU."""
    arr = (ctypes.c_int * len(PLAN_FIELDS))()
    _check(lib().w4a8_plan_info(M, K, N, int(w8a16), num_sms, arr, len(PLAN_FIELDS)))
    return dict(zip(PLAN_FIELDS, list(arr)))


# group scales: the fold chunks of the fixed-order contract (count, codes each)
GROUP_PLAN_FIELDS = PLAN_FIELDS + ("chunks", "chunk_codes")


def w4a8g_plan_info(M: int, K: int, N: int, group: int, num_sms: int = 0) -> dict:
    """Launch plan of the group-scale entry points; num_sms > 0 plans without a GPU."""
    arr = (ctypes.c_int * len(GROUP_PLAN_FIELDS))()
    _check(lib().w4a8g_plan_info(M, K, N, group, num_sms, arr, len(GROUP_PLAN_FIELDS)))
    return dict(zip(GROUP_PLAN_FIELDS, list(arr)))
