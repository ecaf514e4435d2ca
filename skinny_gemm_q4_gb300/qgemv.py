"""Thin ctypes binding of the qgemv C ABI (include/qgemv.h).

Argument marshalling only: every step of the product runs in the CUDA library
``_build/libqgemv.so``.  If the library is missing this module raises; there
is no CPU or PyTorch fallback.

The module-level functions carry the C names and take raw pointers/ints.
``QGemv`` is a convenience wrapper that takes torch CUDA tensors, keeps the
borrowed weight tensors alive and passes ``torch.cuda.current_stream()``.
"""
from __future__ import annotations

import ctypes
import os
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "_build", "libqgemv.so")

Q4_K = 12
Q5_K = 13
Q6_K = 14
NVFP4_W4A16 = 256
FP8_E4M3 = 257

OUT_F16 = 0
OUT_F32 = 1

FLAG_FORCE_REFERENCE = 1
FLAG_DEBUG_SYNC = 2
FLAG_NO_FALLBACK = 4
FLAG_MMA_SYNC_PREFILL = 8

OK = 0
EINVAL = -1
STATUS_NAMES = {0: "QG_OK", -1: "QG_EINVAL", -2: "QG_EUNSUPPORTED", -3: "QG_EALIGN",
                -4: "QG_ECUDA", -5: "QG_ENOMEM", -6: "QG_EFAULT_INJECTED"}

#: every symbol include/qgemv.h declares
EXPORTS = ["qgemv_create", "qgemv_run", "qgemv_run_add", "qgemv_pair_run", "qgemv_triple_run",
           "qgemv_run_host", "qgemv_dequantize", "qgemv_destroy", "qgemv_last_error",
           "qgemv_row_bytes", "qgemv_plan_info", "qgemv_describe", "qgemv_device_status",
           "qgemv_run_noalloc", "qgemv_pair_swiglu_run", "qgemv_chain_create",
           "qgemv_chain_run", "qgemv_chain_status", "qgemv_chain_destroy",
           "qgemv_chain_run_host",
           "qgemv_kv_page_bytes", "qgemv_kv_create", "qgemv_kv_write", "qgemv_kv_read",
           "qgemv_kv_status", "qgemv_kv_destroy", "qgemv_rope_freqs", "qgemv_rope_create",
           "qgemv_rope_run", "qgemv_rope_destroy", "qgemv_attn_create", "qgemv_attn_run",
           "qgemv_attn_status", "qgemv_attn_destroy"]

CHAIN_PERSISTENT = 1

CALL_RUN = 0
CALL_RUN_ADD = 1
CALL_PAIR = 2
CALL_TRIPLE = 3

KV_F16 = 0
KV_Q8 = 1
KV_Q4 = 2

ROPE_HALF = 0
ROPE_INTERLEAVED = 1

ROPE_SCALE_NONE = 0
ROPE_SCALE_LINEAR = 1
ROPE_SCALE_YARN = 2
ROPE_SCALE_BANDS = 3


class QgOpts(ctypes.Structure):
    _fields_ = [("flags", ctypes.c_uint32), ("max_tokens", ctypes.c_int32)]


class QgCall(ctypes.Structure):
    """struct qg_call (one call of a decode chain)."""
    _fields_ = [("kind", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("N", ctypes.c_int64),
                ("h", ctypes.c_void_p * 3), ("x", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("y", ctypes.c_void_p * 3)]


class QgRopeDesc(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_len", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double), ("mscale", ctypes.c_double)]


class QgRopeArgs(ctypes.Structure):
    """struct qg_rope_args (one norm + rotation call)."""
    _fields_ = [("N", ctypes.c_int64), ("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("q_out", ctypes.c_void_p), ("q_out_stride", ctypes.c_int64),
                ("k", ctypes.c_void_p), ("k_stride", ctypes.c_int64),
                ("k_out", ctypes.c_void_p), ("k_out_stride", ctypes.c_int64),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("positions", ctypes.c_void_p),
                ("cache", ctypes.c_void_p), ("slots", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("v_stride", ctypes.c_int64)]


class QgAttnDesc(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("max_batch", ctypes.c_int32), ("max_len", ctypes.c_int64)]


class QgAttnArgs(ctypes.Structure):
    """struct qg_attn_args (one attention call)."""
    _fields_ = [("cache", ctypes.c_void_p), ("q", ctypes.c_void_p), ("q_stride", ctypes.c_int64),
                ("out", ctypes.c_void_p), ("out_stride", ctypes.c_int64),
                ("lse", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int32),
                ("N", ctypes.c_int64), ("B", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
                ("window", ctypes.c_int32)]


class QgemvError(RuntimeError):
    def __init__(self, status: int, what: str, message: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libqgemv.so (built by ``skinny_gemm_q4_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"CUDA library {path} is not built; run "
                           "`python -m skinny_gemm_q4_gb300.build` first")
    lib = ctypes.CDLL(path)
    vp, i64, i32, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int
    lib.qgemv_create.argtypes = [ctypes.POINTER(vp), c_int, i64, i64, vp, vp, ctypes.c_float,
                                 ctypes.POINTER(QgOpts)]
    lib.qgemv_run.argtypes = [vp, vp, i64, vp, c_int, vp]
    lib.qgemv_run_add.argtypes = [vp, vp, i64, vp, vp, vp]
    lib.qgemv_pair_run.argtypes = [vp, vp, vp, i64, vp, vp, c_int, vp]
    lib.qgemv_triple_run.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp, c_int, vp]
    lib.qgemv_run_host.argtypes = [vp, vp, i64, vp, c_int, vp]
    lib.qgemv_dequantize.argtypes = [vp, vp, vp]
    lib.qgemv_destroy.argtypes = [vp]
    lib.qgemv_destroy.restype = None
    lib.qgemv_last_error.argtypes = []
    lib.qgemv_last_error.restype = ctypes.c_char_p
    lib.qgemv_row_bytes.argtypes = [c_int, i64]
    lib.qgemv_row_bytes.restype = i64
    lib.qgemv_plan_info.argtypes = [vp, i64, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                    ctypes.POINTER(i32)]
    lib.qgemv_device_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), c_int]
    lib.qgemv_describe.argtypes = []
    lib.qgemv_describe.restype = ctypes.c_char_p
    lib.qgemv_run_noalloc.argtypes = [c_int, i64, i64, vp, vp, ctypes.c_float, vp, i64, vp, c_int,
                                      vp]
    lib.qgemv_pair_swiglu_run.argtypes = [vp, vp, vp, i64, vp, c_int, vp]
    lib.qgemv_chain_create.argtypes = [ctypes.POINTER(vp), ctypes.c_uint32]
    lib.qgemv_chain_run.argtypes = [vp, ctypes.POINTER(QgCall), i32, vp]
    lib.qgemv_chain_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), c_int]
    sz = ctypes.c_size_t
    lib.qgemv_chain_run_host.argtypes = [vp, ctypes.POINTER(QgCall), i32, vp, vp, sz, vp, vp, sz,
                                         vp]
    lib.qgemv_chain_destroy.argtypes = [vp]
    lib.qgemv_chain_destroy.restype = None
    u32p = ctypes.POINTER(ctypes.c_uint32)
    lib.qgemv_kv_page_bytes.argtypes = [c_int, i32, i32, i32]
    lib.qgemv_kv_page_bytes.restype = i64
    lib.qgemv_kv_create.argtypes = [ctypes.POINTER(vp), c_int, i64, i32, i32, i32, vp]
    lib.qgemv_kv_write.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp]
    lib.qgemv_kv_read.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp]
    lib.qgemv_kv_status.argtypes = [vp, u32p, c_int]
    lib.qgemv_rope_freqs.argtypes = [ctypes.POINTER(QgRopeDesc), ctypes.POINTER(ctypes.c_double),
                                     ctypes.POINTER(ctypes.c_double)]
    lib.qgemv_rope_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(QgRopeDesc)]
    lib.qgemv_rope_run.argtypes = [vp, ctypes.POINTER(QgRopeArgs), vp]
    lib.qgemv_attn_create.argtypes = [ctypes.POINTER(vp), ctypes.POINTER(QgAttnDesc)]
    lib.qgemv_attn_run.argtypes = [vp, ctypes.POINTER(QgAttnArgs), vp]
    lib.qgemv_attn_status.argtypes = [vp, u32p, c_int]
    for name in ("qgemv_kv_destroy", "qgemv_rope_destroy", "qgemv_attn_destroy"):
        getattr(lib, name).argtypes = [vp]
        getattr(lib, name).restype = None
    for name in ("qgemv_create", "qgemv_run", "qgemv_run_add", "qgemv_pair_run",
                 "qgemv_triple_run", "qgemv_run_host", "qgemv_dequantize", "qgemv_plan_info",
                 "qgemv_device_status", "qgemv_run_noalloc", "qgemv_pair_swiglu_run",
                 "qgemv_chain_create", "qgemv_chain_run", "qgemv_chain_status",
                 "qgemv_chain_run_host", "qgemv_kv_create", "qgemv_kv_write", "qgemv_kv_read",
                 "qgemv_kv_status", "qgemv_rope_freqs", "qgemv_rope_create", "qgemv_rope_run",
                 "qgemv_attn_create", "qgemv_attn_run", "qgemv_attn_status"):
        getattr(lib, name).restype = c_int
    _lib = lib
    return lib


# ----------------------------------------------------------- C-named calls

def qgemv_last_error() -> str:
    return load().qgemv_last_error().decode()


def _check(status: int, what: str):
    if status != OK:
        raise QgemvError(status, what, qgemv_last_error())


def qgemv_row_bytes(qtype: int, K: int) -> int:
    return int(load().qgemv_row_bytes(qtype, K))


def qgemv_describe() -> str:
    return load().qgemv_describe().decode()


def qgemv_create(qtype: int, M: int, K: int, w_ptr: int, scales_ptr: int = 0,
                 global_scale: float = 1.0, flags: int = 0, max_tokens: int = 0) -> int:
    h = ctypes.c_void_p()
    opts = QgOpts(flags, max_tokens)
    _check(load().qgemv_create(ctypes.byref(h), qtype, M, K, w_ptr or None, scales_ptr or None,
                               global_scale, ctypes.byref(opts)), "qgemv_create")
    return h.value


def qgemv_destroy(h: int):
    if h:
        load().qgemv_destroy(h)


def qgemv_run(h, x_ptr, N, y_ptr, ydt, stream):
    _check(load().qgemv_run(h, x_ptr, N, y_ptr, ydt, stream), "qgemv_run")


def qgemv_run_add(h, x_ptr, N, res_ptr, y_ptr, stream):
    _check(load().qgemv_run_add(h, x_ptr, N, res_ptr, y_ptr, stream), "qgemv_run_add")


def qgemv_pair_run(a, b, x_ptr, N, ya, yb, ydt, stream):
    _check(load().qgemv_pair_run(a, b, x_ptr, N, ya, yb, ydt, stream), "qgemv_pair_run")


def qgemv_triple_run(a, b, c, x_ptr, N, ya, yb, yc, ydt, stream):
    _check(load().qgemv_triple_run(a, b, c, x_ptr, N, ya, yb, yc, ydt, stream),
           "qgemv_triple_run")


def qgemv_pair_swiglu_run(gate, up, x_ptr, N, h_ptr, hdt, stream):
    _check(load().qgemv_pair_swiglu_run(gate, up, x_ptr, N, h_ptr, hdt, stream),
           "qgemv_pair_swiglu_run")


def qgemv_run_host(h, x_host_ptr, N, y_host_ptr, ydt, stream):
    _check(load().qgemv_run_host(h, x_host_ptr, N, y_host_ptr, ydt, stream), "qgemv_run_host")


def qgemv_dequantize(h, w_out_ptr, stream):
    _check(load().qgemv_dequantize(h, w_out_ptr, stream), "qgemv_dequantize")


def qgemv_plan_info(h, N):
    ks, rows, launches = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    _check(load().qgemv_plan_info(h, N, ctypes.byref(ks), ctypes.byref(rows),
                                  ctypes.byref(launches)), "qgemv_plan_info")
    return ks.value, rows.value, launches.value


def qgemv_device_status(h, clear: bool = False) -> int:
    """The handle's device error word (h = None: qgemv_run_noalloc's, on the
    current device)."""
    w = ctypes.c_uint32()
    _check(load().qgemv_device_status(h, ctypes.byref(w), 1 if clear else 0),
           "qgemv_device_status")
    return w.value


def qgemv_run_noalloc(qtype, M, K, w_ptr, scales_ptr, global_scale, x_ptr, N, y_ptr, ydt,
                      stream):
    """Allocation-free product (no handle; scratch in a fixed device array)."""
    _check(load().qgemv_run_noalloc(qtype, M, K, w_ptr or None, scales_ptr or None, global_scale,
                                    x_ptr or None, N, y_ptr or None, ydt, stream),
           "qgemv_run_noalloc")


def qgemv_chain_create(flags: int = 0) -> int:
    c = ctypes.c_void_p()
    _check(load().qgemv_chain_create(ctypes.byref(c), flags), "qgemv_chain_create")
    return c.value


def qgemv_chain_run(c, calls, stream):
    """calls: a QgCall array (see make_calls)."""
    _check(load().qgemv_chain_run(c, calls, len(calls), stream), "qgemv_chain_run")


def qgemv_chain_run_host(c, calls, in_host, in_dev, in_bytes, out_dev, out_host, out_bytes,
                         stream):
    """One step with host inputs and outputs (raw pointers); synchronizes."""
    _check(load().qgemv_chain_run_host(c, calls, len(calls), in_host or None, in_dev or None,
                                       in_bytes, out_dev or None, out_host or None, out_bytes,
                                       stream), "qgemv_chain_run_host")


def qgemv_chain_status(c, clear: bool = False) -> int:
    w = ctypes.c_uint32()
    _check(load().qgemv_chain_status(c, ctypes.byref(w), 1 if clear else 0), "qgemv_chain_status")
    return w.value


def qgemv_chain_destroy(c):
    if c:
        load().qgemv_chain_destroy(c)


def make_calls(specs):
    """QgCall array from (kind, handles, x_ptr, N, ys, out_dtype, residual_ptr)
    tuples (raw pointers and handle values)."""
    arr = (QgCall * len(specs))()
    for i, (kind, hs, x, N, ys, odt, res) in enumerate(specs):
        c = arr[i]
        c.kind, c.out_dtype, c.N, c.x, c.residual = kind, odt, N, x, res or None
        for j, h in enumerate(hs):
            c.h[j] = h
        for j, y in enumerate(ys):
            c.y[j] = y
    return arr


def qgemv_kv_page_bytes(kind: int, page_size: int, kv_heads: int, head_dim: int) -> int:
    return int(load().qgemv_kv_page_bytes(kind, page_size, kv_heads, head_dim))


def qgemv_kv_create(kind: int, pages: int, page_size: int, kv_heads: int, head_dim: int,
                    pool_ptr: int) -> int:
    c = ctypes.c_void_p()
    _check(load().qgemv_kv_create(ctypes.byref(c), kind, pages, page_size, kv_heads, head_dim,
                                  pool_ptr or None), "qgemv_kv_create")
    return c.value


def qgemv_kv_write(c, k_ptr, k_stride, v_ptr, v_stride, slots_ptr, N, stream):
    _check(load().qgemv_kv_write(c, k_ptr or None, k_stride, v_ptr or None, v_stride,
                                 slots_ptr or None, N, stream), "qgemv_kv_write")


def qgemv_kv_read(c, slots_ptr, N, k_ptr, k_stride, v_ptr, v_stride, stream):
    _check(load().qgemv_kv_read(c, slots_ptr or None, N, k_ptr or None, k_stride, v_ptr or None,
                                v_stride, stream), "qgemv_kv_read")


def qgemv_kv_status(c, clear: bool = False) -> int:
    w = ctypes.c_uint32()
    _check(load().qgemv_kv_status(c, ctypes.byref(w), 1 if clear else 0), "qgemv_kv_status")
    return w.value


def qgemv_kv_destroy(c):
    if c:
        load().qgemv_kv_destroy(c)


def rope_desc(head_dim: int, rot_dim: int = 0, layout: int = ROPE_HALF, base: float = 10000.0,
              scaling: int = ROPE_SCALE_NONE, factor: float = 1.0, original_len: float = 0.0,
              low: float = 0.0, high: float = 0.0, mscale: float = 0.0) -> QgRopeDesc:
    return QgRopeDesc(head_dim, rot_dim or head_dim, layout, scaling, base, factor, original_len,
                      low, high, mscale)


def qgemv_rope_freqs(desc: QgRopeDesc):
    """(frequencies in radians per position, scale of cos and sin)."""
    f = (ctypes.c_double * 64)()
    m = ctypes.c_double()
    _check(load().qgemv_rope_freqs(ctypes.byref(desc), f, ctypes.byref(m)), "qgemv_rope_freqs")
    return list(f[:desc.rot_dim // 2]), m.value


def qgemv_rope_create(desc: QgRopeDesc) -> int:
    r = ctypes.c_void_p()
    _check(load().qgemv_rope_create(ctypes.byref(r), ctypes.byref(desc)), "qgemv_rope_create")
    return r.value


def qgemv_rope_run(r, args: QgRopeArgs, stream):
    _check(load().qgemv_rope_run(r, ctypes.byref(args), stream), "qgemv_rope_run")


def qgemv_rope_destroy(r):
    if r:
        load().qgemv_rope_destroy(r)


def qgemv_attn_create(desc: QgAttnDesc) -> int:
    a = ctypes.c_void_p()
    _check(load().qgemv_attn_create(ctypes.byref(a), ctypes.byref(desc)), "qgemv_attn_create")
    return a.value


def qgemv_attn_run(a, args: QgAttnArgs, stream):
    _check(load().qgemv_attn_run(a, ctypes.byref(args), stream), "qgemv_attn_run")


def qgemv_attn_status(a, clear: bool = False) -> int:
    w = ctypes.c_uint32()
    _check(load().qgemv_attn_status(a, ctypes.byref(w), 1 if clear else 0), "qgemv_attn_status")
    return w.value


def qgemv_attn_destroy(a):
    if a:
        load().qgemv_attn_destroy(a)


# ----------------------------------------------------- torch convenience

_raw_stream = None


def _stream_ptr(stream=None) -> int:
    """The handle of `stream`, or of torch's current stream.  (The raw query
    costs 0.2 us where torch.cuda.current_stream() makes an object in 3 us,
    half of a small call.)"""
    global _raw_stream
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        import torch
        torch.cuda.init()
        raw, dev = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream",
                                                         "_cuda_getDevice"))
        if raw and dev:
            _raw_stream = lambda: raw(dev())  # noqa: E731
        else:  # (they are not part of torch's public interface)
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _raw_stream()


class QGemv:
    """One weight matrix on the device (borrowed torch uint8 tensors)."""

    def __init__(self, qtype: int, M: int, K: int, w, scales=None, global_scale: float = 1.0,
                 flags: int = 0, max_tokens: int = 0):
        self.qtype, self.M, self.K = qtype, M, K
        self._w, self._scales = w, scales      # keep the borrowed buffers alive
        self.h = qgemv_create(qtype, M, K, w.data_ptr(),
                              scales.data_ptr() if scales is not None else 0,
                              global_scale, flags, max_tokens)

    def close(self):
        if getattr(self, "h", None):
            qgemv_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _y(self, N, out_f32, y):
        import torch
        if y is None:
            y = torch.empty((N, self.M), dtype=torch.float32 if out_f32 else torch.float16,
                            device=self._w.device)
        return y

    def run(self, x, y=None, out_f32: bool = False, stream=None):
        N = x.shape[0]
        y = self._y(N, out_f32, y)
        qgemv_run(self.h, x.data_ptr(), N, y.data_ptr(), OUT_F32 if out_f32 else OUT_F16,
                  _stream_ptr(stream))
        return y

    def run_add(self, x, residual, y=None, stream=None):
        N = x.shape[0]
        y = self._y(N, False, y)
        qgemv_run_add(self.h, x.data_ptr(), N, residual.data_ptr(), y.data_ptr(),
                      _stream_ptr(stream))
        return y

    def dequantize(self, stream=None):
        import torch
        w = torch.empty((self.M, self.K), dtype=torch.float32, device=self._w.device)
        qgemv_dequantize(self.h, w.data_ptr(), _stream_ptr(stream))
        return w

    def run_host(self, x_host, y_host, out_f32: bool = False, stream=None):
        qgemv_run_host(self.h, x_host.data_ptr(), x_host.shape[0], y_host.data_ptr(),
                       OUT_F32 if out_f32 else OUT_F16, _stream_ptr(stream))
        return y_host

    def plan_info(self, N: int):
        return qgemv_plan_info(self.h, N)

    def device_status(self, clear: bool = False) -> int:
        return qgemv_device_status(self.h, clear)


def pair_run(a: QGemv, b: QGemv, x, out_f32: bool = False, stream=None):
    N = x.shape[0]
    ya, yb = a._y(N, out_f32, None), b._y(N, out_f32, None)
    qgemv_pair_run(a.h, b.h, x.data_ptr(), N, ya.data_ptr(), yb.data_ptr(),
                   OUT_F32 if out_f32 else OUT_F16, _stream_ptr(stream))
    return ya, yb


def triple_run(a: QGemv, b: QGemv, c: QGemv, x, out_f32: bool = False, stream=None):
    N = x.shape[0]
    ya, yb, yc = a._y(N, out_f32, None), b._y(N, out_f32, None), c._y(N, out_f32, None)
    qgemv_triple_run(a.h, b.h, c.h, x.data_ptr(), N, ya.data_ptr(), yb.data_ptr(),
                     yc.data_ptr(), OUT_F32 if out_f32 else OUT_F16, _stream_ptr(stream))
    return ya, yb, yc


def pair_swiglu_run(gate: QGemv, up: QGemv, x, out_f32: bool = False, stream=None):
    """h = silu(x . gate^T) * (x . up^T), one launch."""
    N = x.shape[0]
    h = gate._y(N, out_f32, None)
    qgemv_pair_swiglu_run(gate.h, up.h, x.data_ptr(), N, h.data_ptr(),
                          OUT_F32 if out_f32 else OUT_F16, _stream_ptr(stream))
    return h


class Chain:
    """A decode chain: consecutive calls in one persistent launch where the
    library can, with the results of issuing them one by one."""

    def __init__(self, flags: int = 0):
        self.c = qgemv_chain_create(flags)

    def run(self, calls, stream=None):
        """calls: QgCall array from make_calls (reusable across runs)."""
        qgemv_chain_run(self.c, calls, _stream_ptr(stream))

    def status(self, clear: bool = False) -> int:
        return qgemv_chain_status(self.c, clear)

    def close(self):
        if getattr(self, "c", None):
            qgemv_chain_destroy(self.c)
            self.c = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------- the attention side of a layer

def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _heads(t, name: str, heads: int, dim: int, N: int):
    """(pointer, token stride) of an fp16 CUDA tensor [N][heads][dim] (or
    [N][heads * dim]) whose tokens may be strided.  (Tokens that all lie in one
    place, as expand() makes them, are refused: a stride of 0 means contiguous
    to the library.)"""
    if t.shape == (N, heads, dim):
        s, h, d = t.stride()
        ok = N == 0 or (d == 1 and (h == dim or heads == 1))
    else:
        ok = t.shape == (N, heads * dim) and (N == 0 or t.stride(1) == 1)
        s = t.stride(0) if ok else 0
    if not (ok and (s or N < 2) and t.is_cuda and t.dtype is sys.modules["torch"].float16):
        raise ValueError(f"{name}: a CUDA fp16 tensor [{N}][{heads}][{dim}] expected, tokens "
                         "contiguous")
    return t.data_ptr(), (s if N > 1 else 0)


def _ints(t, name: str, n, dtype):
    if not (t.is_cuda and t.dtype is dtype and t.numel() == n and t.is_contiguous()):
        raise ValueError(f"{name}: a contiguous CUDA {dtype} tensor of {n} expected")
    return t.data_ptr()


class _Call:
    """A prepared call: the C arguments and the tensors that they point to.
    It can be run any number of times (the tensors' contents may change), on
    handles of its q heads' number and size, `heads`: the library goes by the
    handle's and cannot see the tensors'."""

    def __init__(self, args, heads, cache, *keep):
        self.args, self.ref, self.heads, self.cache = args, ctypes.byref(args), heads, cache
        self.keep = keep


def _unfit(what: str, call: _Call, handle: str):
    """Refuse a call of other heads than the handle's, or of a cache that was
    closed after the call was made."""
    if call.cache is not None and call.cache.c is None:
        raise QgemvError(EINVAL, what, "the call's cache is closed")
    raise QgemvError(EINVAL, what, f"the call has heads {call.heads[0]} x {call.heads[1]}, "
                                   f"the handle is for {handle}")


class KVCache:
    """A paged key/value cache in `pool`, a uint8 CUDA tensor [pages][page
    bytes] (borrowed; ``KVCache.new`` allocates one)."""

    def __init__(self, kind: int, pool, page_size: int, kv_heads: int, head_dim: int):
        import torch
        nbytes = qgemv_kv_page_bytes(kind, page_size, kv_heads, head_dim)
        _need(nbytes < 0 or (pool.is_cuda and pool.dtype == torch.uint8 and pool.is_contiguous()
                             and pool.dim() == 2 and pool.shape[1] == nbytes),
              f"pool: a contiguous CUDA uint8 tensor [pages][{nbytes}]")
        self.kind, self.page_size, self.kv_heads, self.head_dim = (kind, page_size, kv_heads,
                                                                   head_dim)
        self.pool = pool
        with torch.cuda.device(pool.device):  # the handle's own memory goes there too
            self.c = qgemv_kv_create(kind, pool.shape[0], page_size, kv_heads, head_dim,
                                     pool.data_ptr())

    @classmethod
    def new(cls, kind: int, pages: int, page_size: int, kv_heads: int, head_dim: int,
            device="cuda"):
        import torch
        nbytes = qgemv_kv_page_bytes(kind, page_size, kv_heads, head_dim)
        _need(nbytes > 0, "KVCache: unsupported type or shape")
        return cls(kind, torch.empty((pages, nbytes), dtype=torch.uint8, device=device),
                   page_size, kv_heads, head_dim)

    def close(self):
        if getattr(self, "c", None):
            qgemv_kv_destroy(self.c)
            self.c = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def write(self, k, v, slots, stream=None):
        """k and v [N][kv_heads][head_dim] into slots [N] (int64; < 0: skipped)."""
        N = k.shape[0]
        kp, ks = _heads(k, "k", self.kv_heads, self.head_dim, N)
        vp, vs = _heads(v, "v", self.kv_heads, self.head_dim, N)
        sp = _ints(slots, "slots", N, sys.modules["torch"].int64)
        if N:
            st = _lib.qgemv_kv_write(self.c, kp, ks, vp, vs, sp, N, _stream_ptr(stream))
            if st:
                _check(st, "qgemv_kv_write")

    def read(self, slots, k_out=None, v_out=None, stream=None):
        """What the cache holds for slots: (k, v), fp16 [N][kv_heads][head_dim]."""
        torch = sys.modules["torch"]
        N = slots.shape[0]
        if k_out is None or v_out is None:
            with torch.cuda.stream(stream):  # outputs made here belong to the call's stream
                k_out, v_out = (torch.empty((N, self.kv_heads, self.head_dim),
                                            dtype=torch.float16, device=slots.device)
                                if t is None else t for t in (k_out, v_out))
        kp, ks = _heads(k_out, "k_out", self.kv_heads, self.head_dim, N)
        vp, vs = _heads(v_out, "v_out", self.kv_heads, self.head_dim, N)
        sp = _ints(slots, "slots", N, torch.int64)
        if N:
            st = _lib.qgemv_kv_read(self.c, sp, N, kp, ks, vp, vs, _stream_ptr(stream))
            if st:
                _check(st, "qgemv_kv_read")
        return k_out, v_out

    def status(self, clear: bool = False) -> int:
        return qgemv_kv_status(self.c, clear)


def make_rope_call(q, k, positions, q_out=None, k_out=None, q_weight=None, k_weight=None,
                   eps: float = 1e-6, cache: KVCache = None, slots=None, v=None) -> _Call:
    """Norm + rotation of q [N][q_heads][D] and k [N][kv_heads][D] (in place
    where no output is given; k only into the cache when one is); fp32 weights
    [D] or None; with a cache, k and v are written to slots."""
    import torch
    N, H, D = q.shape
    q_out = q if q_out is None else q_out
    a = QgRopeArgs()
    a.N, a.q_heads, a.eps = N, H, eps
    a.q, a.q_stride = _heads(q, "q", H, D, N)
    a.q_out, a.q_out_stride = _heads(q_out, "q_out", H, D, N)
    if k is not None:
        a.kv_heads = k.shape[1]
        a.k, a.k_stride = _heads(k, "k", a.kv_heads, D, N)
        if k_out is None and cache is None:
            k_out = k
        if k_out is not None:
            a.k_out, a.k_out_stride = _heads(k_out, "k_out", a.kv_heads, D, N)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _need(w.is_cuda and w.dtype == torch.float32 and w.is_contiguous() and w.numel() == D,
                  f"{name}: a contiguous CUDA fp32 tensor of {D}")
            setattr(a, name, w.data_ptr())
    a.positions = _ints(positions, "positions", N, torch.int32)
    if cache is not None:
        _need(slots is not None and v is not None, "a cache needs slots and v")
        a.cache = cache.c
        a.slots = _ints(slots, "slots", N, torch.int64)
        a.v, a.v_stride = _heads(v, "v", cache.kv_heads, D, N)
    return _Call(a, (H, D), cache, q, k, q_out, k_out, q_weight, k_weight, positions, slots, v)


class Rope:
    """The rotation of one description (see ``rope_desc``)."""

    def __init__(self, head_dim: int, **desc):
        self.desc = rope_desc(head_dim, **{n: v for n, v in desc.items() if v is not None})
        self.head_dim = head_dim  # (a field of desc costs 0.1 us a look)
        self.r = qgemv_rope_create(self.desc)

    def close(self):
        if getattr(self, "r", None):
            qgemv_rope_destroy(self.r)
            self.r = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def run(self, call: _Call, stream=None):
        if call.heads[1] != self.head_dim or call.cache is not None and call.cache.c is None:
            _unfit("qgemv_rope_run", call, f"heads of {self.head_dim}")
        st = _lib.qgemv_rope_run(self.r, call.ref, _stream_ptr(stream))
        if st:
            _check(st, "qgemv_rope_run")


def make_attn_call(cache: KVCache, q, out, q_start, kv_len, page_table, max_q: int,
                   scale: float = None, causal: bool = True, window: int = 0, lse=None) -> _Call:
    """Attention of q [N][q_heads][D] (request b's new tokens are rows
    q_start[b] .. q_start[b + 1] - 1) over cached contexts of kv_len[b] tokens
    whose pages are page_table[b]; out as q, lse fp32 [N][q_heads] or None."""
    import torch
    N, H, D = q.shape
    _need(D == cache.head_dim, f"q: heads of {D}, the cache's are of {cache.head_dim}")
    B = kv_len.shape[0]
    a = QgAttnArgs()
    a.cache, a.N, a.B, a.max_q = cache.c, N, B, max_q
    a.q, a.q_stride = _heads(q, "q", H, D, N)
    a.out, a.out_stride = _heads(out, "out", H, D, N)
    if lse is not None:
        _need(lse.is_cuda and lse.dtype == torch.float32 and lse.is_contiguous()
              and lse.numel() == N * H, f"lse: a contiguous CUDA fp32 tensor [{N}][{H}]")
        a.lse = lse.data_ptr()
    a.q_start = _ints(q_start, "q_start", B + 1, torch.int32)
    a.kv_len = _ints(kv_len, "kv_len", B, torch.int32)
    _need(page_table.is_cuda and page_table.dtype == torch.int32 and page_table.dim() == 2
          and page_table.shape[0] == B and (page_table.shape[1] < 2 or page_table.stride(1) == 1),
          f"page_table: a CUDA int32 tensor [{B}][pages]")
    _need(B < 2 or page_table.stride(0) >= page_table.shape[1], "page_table: overlapping rows")
    a.page_table = page_table.data_ptr()
    a.table_width = page_table.shape[1]
    a.table_stride = page_table.stride(0) if B > 1 else 0
    a.scale = D ** -0.5 if scale is None else scale
    a.causal, a.window = int(causal), window
    return _Call(a, (H, D), cache, q, out, q_start, kv_len, page_table, lse)


class Attn:
    """Attention of one head shape; layers share it on one stream.  Its workspace
    grows with max_len times the new tokens that requests of few rows can have
    in a call: max_batch (default: max_tokens) requests, max_tokens at most."""

    def __init__(self, q_heads: int, kv_heads: int, head_dim: int, max_tokens: int,
                 max_len: int, max_batch: int = None):
        self.heads = q_heads, head_dim
        self.a = qgemv_attn_create(QgAttnDesc(q_heads, kv_heads, head_dim, max_tokens,
                                              min(max_tokens, 65535) if max_batch is None
                                              else max_batch, max_len))

    def close(self):
        if getattr(self, "a", None):
            qgemv_attn_destroy(self.a)
            self.a = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def run(self, call: _Call, stream=None):
        if call.heads != self.heads or call.cache.c is None:
            _unfit("qgemv_attn_run", call, "%d x %d" % self.heads)
        st = _lib.qgemv_attn_run(self.a, call.ref, _stream_ptr(stream))
        if st:
            _check(st, "qgemv_attn_run")

    def status(self, clear: bool = False) -> int:
        return qgemv_attn_status(self.a, clear)
