"""ctypes binding of libqmm.so (include/qmm.h): argument marshalling only.

Every step of the product runs in the library's CUDA kernels; this module passes device
pointers (``tensor.data_ptr()``), sizes and the caller's current CUDA stream.  There is no
fallback: if the library is missing or cannot load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqmm.so")

QMM_QK = 256
QMM_BLOCK_BYTES = 144
QMM_MAX_M = 32
QMM_MAX_BATCH = 512

VARIANT_AUTO, VARIANT_FMA, VARIANT_TC = 0, 1, 2
VARIANT_NAMES = {VARIANT_FMA: "fma", VARIANT_TC: "tc"}

STATUS = {0: "QMM_OK", 1: "QMM_ERR_NULL", 2: "QMM_ERR_SHAPE", 3: "QMM_ERR_M_RANGE",
          4: "QMM_ERR_ALIGN", 5: "QMM_ERR_BUFSIZE", 6: "QMM_ERR_NONFINITE", 7: "QMM_ERR_CUDA",
          8: "QMM_ERR_COUNT", 9: "QMM_ERR_VARIANT", 10: "QMM_ERR_SCRATCH", 11: "QMM_ERR_FORMAT",
          12: "QMM_ERR_TYPE"}

FMT_Q4K, FMT_Q5K, FMT_NVFP4, FMT_INT4, FMT_Q6K = 0, 1, 2, 3, 4
F32, BF16, F16 = 0, 1, 2   # element types of the attention half (qmm_dtype)
FORMATS = {"q4k": FMT_Q4K, "q5k": FMT_Q5K, "q6k": FMT_Q6K, "nvfp4": FMT_NVFP4, "int4": FMT_INT4}

# Every symbol include/qmm.h declares.
EXPORTS = ["qmm_packed_bytes", "qmm_pack", "qmm_run", "qmm_run_batched", "qmm_dequant",
           "qmm_run_variant", "qmm_select_variant", "qmm_device_status", "qmm_strerror",
           "qmm_last_cuda_error", "qmm_run_noalloc", "qmm_select_variant_batched",
           "qmm_ffn_workspace_bytes", "qmm_run_ffn", "qmm_indexed_workspace_bytes", "qmm_run_indexed",
           "qmm_fmt_packed_bytes", "qmm_fmt_pack", "qmm_fmt_run", "qmm_fmt_dequant", "qmm_fmt_run_batched",
           "qmm_ffn_fused_workspace_bytes", "qmm_run_ffn_fused", "qmm_release", "qmm_workspace_bytes_held",
           "qmm_stream_read", "qmm_stream_read_sink_words", "qmm_set_wait_limit", "qmm_pack_dev",
           "qmm_norm_rope", "qmm_attn_workspace_bytes", "qmm_attn_shared", "qmm_lora_workspace_bytes",
           "qmm_run_lora"]
NOALLOC_SCRATCH_BYTES = 4 << 20


class QmmError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        lib = _lib
        text = lib.qmm_strerror(status).decode() if lib is not None else STATUS.get(status, "?")
        if status == 7 and lib is not None:
            text += ": " + lib.qmm_last_cuda_error().decode()
        super().__init__(f"{what}: {STATUS.get(status, status)} ({text})")


class _Entry(ctypes.Structure):
    _fields_ = [("Wq", ctypes.c_void_p), ("X", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class _FmtEntry(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("Wq", ctypes.c_void_p), ("X", ctypes.c_void_p), ("Y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


class _NormRopeArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("T", "Hq", "Hk", "D", "rot", "interleaved", "in_type", "out_type")] + [
        ("eps", ctypes.c_float), ("Q", ctypes.c_void_p), ("K", ctypes.c_void_p), ("V", ctypes.c_void_p),
        ("ldq", ctypes.c_int64), ("ldk", ctypes.c_int64), ("ldv", ctypes.c_int64),
        ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("cos_sin", ctypes.c_void_p),
        ("max_pos", ctypes.c_int64), ("positions", ctypes.c_void_p), ("slots", ctypes.c_void_p),
        ("Q_out", ctypes.c_void_p), ("ldqo", ctypes.c_int64), ("K_cache", ctypes.c_void_p),
        ("V_cache", ctypes.c_void_p), ("n_slots", ctypes.c_int64)]


class _AttnArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("T", "B", "Hq", "Hk", "D", "page_size", "type")] + [
        ("scale", ctypes.c_float), ("Q", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("K_cache", ctypes.c_void_p),
        ("V_cache", ctypes.c_void_p), ("n_slots", ctypes.c_int64), ("prefix_pages", ctypes.c_void_p),
        ("prefix_len", ctypes.c_int64), ("pages", ctypes.c_void_p), ("pages_per_stream", ctypes.c_int64),
        ("kv_lens", ctypes.c_void_p), ("row_starts", ctypes.c_void_p), ("O", ctypes.c_void_p),
        ("ldo", ctypes.c_int64), ("lse", ctypes.c_void_p)]


class _LoraAdapter(ctypes.Structure):
    _fields_ = [("A", ctypes.c_void_p), ("Bt", ctypes.c_void_p), ("scale", ctypes.c_float), ("rank", ctypes.c_int)]


class _LoraEntry(ctypes.Structure):
    _fields_ = [("adapters", ctypes.c_void_p), ("n_adapters", ctypes.c_int), ("X", ctypes.c_void_p),
                ("Y0", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


_lib = None


def load(path: str | None = None):
    """Load libqmm.so (raises if it is missing: build it with build_lib.build())."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libqmm.so not found at {p}: run bit_quantized_skinny_gb300.build_lib.build()")
    lib = ctypes.CDLL(p)
    vp, i64, i32, u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint
    lib.qmm_packed_bytes.argtypes = [i64, i64]
    lib.qmm_packed_bytes.restype = ctypes.c_size_t
    lib.qmm_pack.argtypes = [vp, i64, i64, vp, ctypes.c_size_t, i32]
    lib.qmm_pack.restype = i32
    lib.qmm_pack_dev.argtypes = [vp, i64, i64, vp, ctypes.c_size_t, vp]
    lib.qmm_pack_dev.restype = i32
    lib.qmm_run.argtypes = [vp, i64, i64, vp, vp, i32, vp]
    lib.qmm_run.restype = i32
    lib.qmm_run_variant.argtypes = [vp, i64, i64, vp, vp, i32, i32, vp]
    lib.qmm_run_variant.restype = i32
    lib.qmm_run_noalloc.argtypes = [vp, i64, i64, vp, vp, i32, vp]
    lib.qmm_run_noalloc.restype = i32
    lib.qmm_stream_read.argtypes = [vp, ctypes.c_size_t, vp, vp]
    lib.qmm_stream_read.restype = i32
    lib.qmm_stream_read_sink_words.argtypes = []
    lib.qmm_stream_read_sink_words.restype = ctypes.c_size_t
    lib.qmm_set_wait_limit.argtypes = [ctypes.c_uint32, ctypes.c_uint32]
    lib.qmm_set_wait_limit.restype = None
    lib.qmm_release.argtypes = []
    lib.qmm_release.restype = i32
    lib.qmm_workspace_bytes_held.argtypes = []
    lib.qmm_workspace_bytes_held.restype = ctypes.c_size_t
    lib.qmm_run_batched.argtypes = [ctypes.POINTER(_Entry), i32, i32, vp]
    lib.qmm_run_batched.restype = i32
    lib.qmm_dequant.argtypes = [vp, i64, i64, vp, vp]
    lib.qmm_dequant.restype = i32
    lib.qmm_select_variant.argtypes = [i32, i64, i64]
    lib.qmm_select_variant.restype = i32
    lib.qmm_select_variant_batched.argtypes = [ctypes.POINTER(_Entry), i32, i32]
    lib.qmm_select_variant_batched.restype = i32
    lib.qmm_ffn_workspace_bytes.argtypes = [i32, i64]
    lib.qmm_ffn_workspace_bytes.restype = ctypes.c_size_t
    lib.qmm_run_ffn.argtypes = [vp, vp, i64, i64, vp, vp, i32, vp, ctypes.c_size_t, vp]
    lib.qmm_run_ffn.restype = i32
    lib.qmm_ffn_fused_workspace_bytes.argtypes = [i32, i64]
    lib.qmm_ffn_fused_workspace_bytes.restype = ctypes.c_size_t
    lib.qmm_run_ffn_fused.argtypes = [vp, vp, i64, i64, vp, vp, i32, vp, ctypes.c_size_t, vp]
    lib.qmm_run_ffn_fused.restype = i32
    lib.qmm_indexed_workspace_bytes.argtypes = [i32, i64, i64]
    lib.qmm_indexed_workspace_bytes.restype = ctypes.c_size_t
    lib.qmm_run_indexed.argtypes = [ctypes.POINTER(vp), i32, i64, i64, ctypes.POINTER(ctypes.c_int32), vp, vp, i32,
                                    vp, ctypes.c_size_t, vp]
    lib.qmm_run_indexed.restype = i32
    lib.qmm_fmt_packed_bytes.argtypes = [i32, i64, i64]
    lib.qmm_fmt_packed_bytes.restype = ctypes.c_size_t
    lib.qmm_fmt_pack.argtypes = [i32, vp, i64, i64, vp, ctypes.c_size_t, i32]
    lib.qmm_fmt_pack.restype = i32
    lib.qmm_fmt_run.argtypes = [i32, vp, i64, i64, vp, vp, i32, vp]
    lib.qmm_fmt_run.restype = i32
    lib.qmm_fmt_run_batched.argtypes = [ctypes.POINTER(_FmtEntry), i32, i32, vp]
    lib.qmm_fmt_run_batched.restype = i32
    lib.qmm_fmt_dequant.argtypes = [i32, vp, i64, i64, vp, vp]
    lib.qmm_fmt_dequant.restype = i32
    lib.qmm_norm_rope.argtypes = [ctypes.POINTER(_NormRopeArgs), vp]
    lib.qmm_norm_rope.restype = i32
    lib.qmm_attn_workspace_bytes.argtypes = [ctypes.POINTER(_AttnArgs)]
    lib.qmm_attn_workspace_bytes.restype = ctypes.c_size_t
    lib.qmm_attn_shared.argtypes = [ctypes.POINTER(_AttnArgs), vp, ctypes.c_size_t, vp]
    lib.qmm_attn_shared.restype = i32
    lib.qmm_lora_workspace_bytes.argtypes = [ctypes.POINTER(_LoraEntry), i32, i32, i32]
    lib.qmm_lora_workspace_bytes.restype = ctypes.c_size_t
    lib.qmm_run_lora.argtypes = [ctypes.POINTER(_LoraEntry), i32, vp, i32, i32, vp, ctypes.c_size_t, vp]
    lib.qmm_run_lora.restype = i32
    lib.qmm_device_status.argtypes = [ctypes.POINTER(u32)]
    lib.qmm_device_status.restype = i32
    lib.qmm_strerror.argtypes = [i32]
    lib.qmm_strerror.restype = ctypes.c_char_p
    lib.qmm_last_cuda_error.argtypes = []
    lib.qmm_last_cuda_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int, what: str):
    if status != 0:
        raise QmmError(status, what)


def _current_stream() -> int:
    """Handle of torch's current stream on the current device.  (Without the Stream object that
    torch.cuda.current_stream() makes: 0.4 us a call, not 3.3.)"""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream


def _stream_handle(stream):
    if stream is None:
        return _current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def packed_bytes(N: int, K: int) -> int:
    return load().qmm_packed_bytes(N, K)


def pack(W: np.ndarray, threads: int = 0, out: np.ndarray | None = None) -> np.ndarray:
    """Pack an N x K fp32 host array into Q4K bytes (host, multi-threaded)."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    nbytes = packed_bytes(N, K)
    if nbytes == 0:
        raise QmmError(2, "qmm_pack")
    if out is None:
        out = np.empty(nbytes, dtype=np.uint8)
    _check(load().qmm_pack(W.ctypes.data_as(ctypes.c_void_p), N, K, out.ctypes.data_as(ctypes.c_void_p),
                           out.nbytes, threads), "qmm_pack")
    return out


def pack_dev(W, out=None, stream=None):
    """qmm_pack_dev: pack an N x K fp32 CUDA tensor into Q4K bytes on the GPU (a uint8 CUDA
    tensor of packed_bytes(N, K) bytes, allocated when `out` is None), asynchronous on `stream`
    (default: torch's current stream).  Non-finite super-blocks come out as zeros and set bit 1
    of device_status()."""
    import torch
    N, K = W.shape
    nbytes = packed_bytes(N, K)
    if nbytes == 0:
        raise QmmError(2, "qmm_pack_dev")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    _check(load().qmm_pack_dev(ctypes.c_void_p(W.data_ptr()), N, K, ctypes.c_void_p(out.data_ptr()),
                               out.numel() * out.element_size(), _stream_handle(stream)), "qmm_pack_dev")
    return out


def run(Wq, N: int, K: int, X, Y, M: int | None = None, variant: int = VARIANT_AUTO, stream=None):
    """Y[M x N] = X[M x K] * dequant(Wq)^T on the GPU (torch CUDA tensors: uint8/any Wq,
    bf16 or int16 X, fp32 Y).  Asynchronous on `stream` (default: torch's current stream)."""
    if M is None:
        M = X.shape[0]
    st = load().qmm_run_variant(ctypes.c_void_p(Wq.data_ptr()), N, K, ctypes.c_void_p(X.data_ptr()),
                                ctypes.c_void_p(Y.data_ptr()), M, variant, _stream_handle(stream))
    _check(st, "qmm_run")


def run_noalloc(Wq, N: int, K: int, X, Y, M: int | None = None, stream=None):
    """qmm_run_noalloc: the tensor-core product without any device allocation (fixed 4 MiB
    library buffer for the prepared activations; see include/qmm.h for its limits)."""
    if M is None:
        M = X.shape[0]
    st = load().qmm_run_noalloc(ctypes.c_void_p(Wq.data_ptr()), N, K, ctypes.c_void_p(X.data_ptr()),
                                ctypes.c_void_p(Y.data_ptr()), M, _stream_handle(stream))
    _check(st, "qmm_run_noalloc")


def run_raw(wq_ptr: int, N: int, K: int, x_ptr: int, y_ptr: int, M: int, variant: int = VARIANT_AUTO,
            stream_handle: int = 0) -> int:
    """Unchecked call on raw device pointers; returns the status code."""
    return load().qmm_run_variant(ctypes.c_void_p(wq_ptr), N, K, ctypes.c_void_p(x_ptr),
                                  ctypes.c_void_p(y_ptr), M, variant, ctypes.c_void_p(stream_handle))


def make_entries(items):
    """items: sequence of (Wq, X, Y, N, K) with torch tensors or raw int pointers."""
    arr = (_Entry * len(items))()
    for k, (Wq, X, Y, N, K) in enumerate(items):
        ptr = lambda t: t if isinstance(t, int) else t.data_ptr()
        arr[k] = _Entry(ptr(Wq), ptr(X), ptr(Y), N, K)
    return arr


def run_batched(entries, M: int, stream=None):
    """One call over independent products sharing M (one product launch per 160 products).
    `entries` from make_entries()."""
    st = load().qmm_run_batched(entries, len(entries), M, _stream_handle(stream))
    _check(st, "qmm_run_batched")


def ffn_workspace_bytes(M: int, F: int) -> int:
    return load().qmm_ffn_workspace_bytes(M, F)


def run_ffn(Wgu, Wdown, F: int, K: int, X, Y, workspace, M: int | None = None, stream=None):
    """One feed-forward block: Y = (silu(X Wg^T) * (X Wu^T) as bf16) Wdown^T, all on the GPU.
    `workspace`: a device tensor of >= ffn_workspace_bytes(M, F) bytes (holds G and H)."""
    if M is None:
        M = X.shape[0]
    nbytes = workspace.numel() * workspace.element_size()
    st = load().qmm_run_ffn(ctypes.c_void_p(Wgu.data_ptr()), ctypes.c_void_p(Wdown.data_ptr()), F, K,
                            ctypes.c_void_p(X.data_ptr()), ctypes.c_void_p(Y.data_ptr()), M,
                            ctypes.c_void_p(workspace.data_ptr()), nbytes, _stream_handle(stream))
    _check(st, "qmm_run_ffn")


def ffn_fused_workspace_bytes(M: int, F: int) -> int:
    return load().qmm_ffn_fused_workspace_bytes(M, F)


def run_ffn_fused(Wgu_interleaved, Wdown, F: int, K: int, X, Y, workspace, M: int | None = None, stream=None):
    """The feed-forward block with the gating in the gate/up product's epilogue.  Wgu_interleaved:
    packed (2F) x K weights with row 2f = gate row f and row 2f+1 = up row f.  `workspace`: a
    device tensor of >= ffn_fused_workspace_bytes(M, F) bytes (holds H)."""
    if M is None:
        M = X.shape[0]
    nbytes = workspace.numel() * workspace.element_size()
    st = load().qmm_run_ffn_fused(ctypes.c_void_p(Wgu_interleaved.data_ptr()), ctypes.c_void_p(Wdown.data_ptr()),
                                  F, K, ctypes.c_void_p(X.data_ptr()), ctypes.c_void_p(Y.data_ptr()), M,
                                  ctypes.c_void_p(workspace.data_ptr()), nbytes, _stream_handle(stream))
    _check(st, "qmm_run_ffn_fused")


def indexed_workspace_bytes(M: int, N: int, K: int) -> int:
    return load().qmm_indexed_workspace_bytes(M, N, K)


def run_indexed(experts, N: int, K: int, ids, X, Y, workspace, stream=None):
    """Y[i] = X[i] * dequant(experts[ids[i]])^T for every row i, on the GPU.  `experts`: device
    tensors (packed N x K each); `ids`: host sequence of M expert indices; `workspace`: a device
    tensor of >= indexed_workspace_bytes(M, N, K) bytes."""
    M = len(ids)
    ptrs = (ctypes.c_void_p * len(experts))(*[w.data_ptr() for w in experts])
    idv = (ctypes.c_int32 * M)(*[int(v) for v in ids])
    nbytes = workspace.numel() * workspace.element_size()
    st = load().qmm_run_indexed(ptrs, len(experts), N, K, idv, ctypes.c_void_p(X.data_ptr()),
                                ctypes.c_void_p(Y.data_ptr()), M, ctypes.c_void_p(workspace.data_ptr()), nbytes,
                                _stream_handle(stream))
    _check(st, "qmm_run_indexed")


def dequant(Wq, N: int, K: int, out, stream=None):
    _check(load().qmm_dequant(ctypes.c_void_p(Wq.data_ptr()), N, K, ctypes.c_void_p(out.data_ptr()),
                              _stream_handle(stream)), "qmm_dequant")


def fmt_packed_bytes(fmt: int, N: int, K: int) -> int:
    return load().qmm_fmt_packed_bytes(fmt, N, K)


def fmt_pack(fmt: int, W: np.ndarray, threads: int = 0) -> np.ndarray:
    """Pack an N x K fp32 host array into weight format `fmt` (host, multi-threaded)."""
    W = np.ascontiguousarray(W, dtype=np.float32)
    N, K = W.shape
    nbytes = fmt_packed_bytes(fmt, N, K)
    if nbytes == 0:
        raise QmmError(2, "qmm_fmt_pack")
    out = np.empty(nbytes, dtype=np.uint8)
    _check(load().qmm_fmt_pack(fmt, W.ctypes.data_as(ctypes.c_void_p), N, K, out.ctypes.data_as(ctypes.c_void_p),
                               out.nbytes, threads), "qmm_fmt_pack")
    return out


def fmt_run(fmt: int, Wq, N: int, K: int, X, Y, M: int | None = None, stream=None):
    """Y[M x N] = X[M x K] * dequant(Wq)^T for weights in format `fmt`, on the GPU."""
    if M is None:
        M = X.shape[0]
    st = load().qmm_fmt_run(fmt, ctypes.c_void_p(Wq.data_ptr()), N, K, ctypes.c_void_p(X.data_ptr()),
                            ctypes.c_void_p(Y.data_ptr()), M, _stream_handle(stream))
    _check(st, "qmm_fmt_run")


def make_fmt_entries(items):
    """items: sequence of (fmt, Wq, X, Y, N, K) with torch tensors or raw int pointers."""
    arr = (_FmtEntry * len(items))()
    for k, (fmt, Wq, X, Y, N, K) in enumerate(items):
        ptr = lambda t: t if isinstance(t, int) else t.data_ptr()
        arr[k] = _FmtEntry(fmt, ptr(Wq), ptr(X), ptr(Y), N, K)
    return arr


def fmt_run_batched(entries, M: int, stream=None):
    """Independent products sharing M, weights in any formats: each format's entries run as one
    batched call."""
    _check(load().qmm_fmt_run_batched(entries, len(entries), M, _stream_handle(stream)), "qmm_fmt_run_batched")


def fmt_dequant(fmt: int, Wq, N: int, K: int, out, stream=None):
    _check(load().qmm_fmt_dequant(fmt, ctypes.c_void_p(Wq.data_ptr()), N, K, ctypes.c_void_p(out.data_ptr()),
                                  _stream_handle(stream)), "qmm_fmt_dequant")


def _dtype_code(t) -> int:
    import torch
    code = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}.get(t.dtype)
    if code is None:
        raise QmmError(12, f"dtype {t.dtype}")
    return code


def _rows(t, what: str) -> int:
    """Elements between the rows of a T x H x D tensor whose rows are dense (H x D contiguous)."""
    if t.dim() != 3 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise QmmError(2, what)
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1] * t.shape[2])


def _dense(t, dtype, what: str) -> int:
    """Data pointer of a contiguous tensor of that dtype (0 for None)."""
    if t is None:
        return 0
    if t.dtype != dtype:
        raise QmmError(12, what)
    if not t.is_contiguous():
        raise QmmError(2, what)
    return t.data_ptr()


def make_norm_rope(Q, K, V, q_weight, k_weight, cos_sin, positions, slots, Q_out, K_cache, V_cache,
                   eps: float = 1e-6, interleaved: bool = False):
    """Arguments of norm_rope().  Q: T x Hq x D, K and V: T x Hk x D (rows may be strided), one of
    fp32, bf16 and fp16; Q_out: T x Hq x D and the caches n_slots x Hk x D, bf16 or fp16; weights
    fp32 D or None; cos_sin fp32 max_pos x rot or None (no rotation); positions int32 T, slots int64
    T.  K, V, slots and the caches may be None together, and V with V_cache.  The tensors are kept
    alive by what is returned."""
    import torch
    T, Hq, D = Q.shape
    a = _NormRopeArgs(T=T, Hq=Hq, Hk=0 if K is None else K.shape[1], D=D, rot=0 if cos_sin is None else cos_sin.shape[1],
                      interleaved=int(interleaved), in_type=_dtype_code(Q), out_type=_dtype_code(Q_out), eps=eps)
    a.Q, a.ldq, a.Q_out, a.ldqo = Q.data_ptr(), _rows(Q, "Q"), Q_out.data_ptr(), _rows(Q_out, "Q_out")
    if tuple(Q_out.shape) != (T, Hq, D):
        raise QmmError(2, "Q_out")
    for t, cache, name in ((K, K_cache, "K"), (V, V_cache, "V")):
        if t is None:
            continue
        if cache is None:
            raise QmmError(1, name + "_cache")
        if tuple(t.shape) != (T, a.Hk, D) or cache.shape[1:] != (a.Hk, D):
            raise QmmError(2, name)
        if t.dtype != Q.dtype:
            raise QmmError(12, name)
        setattr(a, name, t.data_ptr())
        setattr(a, "ldk" if name == "K" else "ldv", _rows(t, name))
        setattr(a, name + "_cache", _dense(cache, Q_out.dtype, name + "_cache"))
    if K is not None:
        a.n_slots = K_cache.shape[0]
        if V is not None and V_cache.shape[0] != a.n_slots:
            raise QmmError(2, "V_cache")
        a.slots = _dense(slots, torch.int64, "slots")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None and w.numel() != D:
            raise QmmError(2, name)
        setattr(a, name, _dense(w, torch.float32, name))
    if cos_sin is not None:
        a.cos_sin, a.max_pos = _dense(cos_sin, torch.float32, "cos_sin"), cos_sin.shape[0]
        a.positions = _dense(positions, torch.int32, "positions")
    for t, name in ((positions if cos_sin is not None else None, "positions"), (slots if K is not None else None, "slots")):
        if t is not None and t.numel() != T:
            raise QmmError(2, name)
    a._keep = (Q, K, V, q_weight, k_weight, cos_sin, positions, slots, Q_out, K_cache, V_cache)
    return a


def norm_rope(args, stream=None) -> None:
    """qmm_norm_rope: norm and rotation of every query and key head, keys and values to their cache
    slots.  `args` from make_norm_rope()."""
    _check(load().qmm_norm_rope(args, _stream_handle(stream)), "qmm_norm_rope")


def make_attn(Q, K_cache, V_cache, page_size: int, prefix_pages, prefix_len: int, pages, kv_lens, row_starts, O,
              scale: float, lse=None):
    """Arguments of attn_shared().  Q, O: T x Hq x D (rows may be strided), caches n_slots x Hk x D, all
    bf16 or all fp16; prefix_pages int32 (None without a prefix), pages int32 B x pages_per_stream,
    kv_lens int32 B, row_starts int32 B + 1; lse fp32 T x Hq or None.  The tensors are kept alive by
    what is returned."""
    import torch
    if any(t is None for t in (K_cache, V_cache, pages, kv_lens, row_starts, O)):
        raise QmmError(1, "make_attn")
    T, Hq, D = Q.shape
    n_slots, Hk, Dk = K_cache.shape
    B, per_stream = pages.shape
    if Dk != D or V_cache.shape != K_cache.shape or O.shape != Q.shape:
        raise QmmError(2, "make_attn")
    if kv_lens.numel() != B or row_starts.numel() != B + 1 or (lse is not None and tuple(lse.shape) != (T, Hq)):
        raise QmmError(2, "make_attn")
    if prefix_len > 0 and (prefix_pages is None or prefix_pages.numel() * page_size < prefix_len):
        raise QmmError(2, "prefix_pages")
    if O.dtype != Q.dtype:
        raise QmmError(12, "O")
    a = _AttnArgs(T=T, B=B, Hq=Hq, Hk=Hk, D=D, page_size=page_size, type=_dtype_code(Q), scale=scale,
                  n_slots=n_slots, prefix_len=prefix_len, pages_per_stream=per_stream)
    a.Q, a.ldq, a.O, a.ldo = Q.data_ptr(), _rows(Q, "Q"), O.data_ptr(), _rows(O, "O")
    a.K_cache, a.V_cache = _dense(K_cache, Q.dtype, "K_cache"), _dense(V_cache, Q.dtype, "V_cache")
    a.prefix_pages = _dense(prefix_pages, torch.int32, "prefix_pages")
    a.pages, a.kv_lens = _dense(pages, torch.int32, "pages"), _dense(kv_lens, torch.int32, "kv_lens")
    a.row_starts, a.lse = _dense(row_starts, torch.int32, "row_starts"), _dense(lse, torch.float32, "lse")
    a._keep = (Q, K_cache, V_cache, prefix_pages, pages, kv_lens, row_starts, O, lse)
    return a


def attn_workspace_bytes(args) -> int:
    return load().qmm_attn_workspace_bytes(args)


def attn_shared(args, workspace, stream=None) -> None:
    """qmm_attn_shared: attention of every stream's rows over the shared prefix and the stream's own
    keys.  `args` from make_attn(); `workspace`: a device tensor of >= attn_workspace_bytes(args)
    bytes."""
    _check(load().qmm_attn_shared(args, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream)), "qmm_attn_shared")


def make_lora_adapters(items):
    """Device table of one projection's adapters.  items: sequence of (A, Bt, scale) with bf16 CUDA
    tensors A rank x K and Bt rank x N (B transposed), both contiguous, K and N those of the projection.
    The tensors are kept alive by what is returned."""
    import torch
    if not items:
        raise QmmError(8, "make_lora_adapters")
    arr = (_LoraAdapter * len(items))()
    first = items[0][0], items[0][1]
    for k, (A, Bt, scale) in enumerate(items):
        if A.dim() != 2 or Bt.dim() != 2 or A.shape[0] != Bt.shape[0]:
            raise QmmError(2, "make_lora_adapters")
        if A.shape[1] != first[0].shape[1] or Bt.shape[1] != first[1].shape[1]:
            raise QmmError(2, "make_lora_adapters: adapters of different projections")
        arr[k] = _LoraAdapter(_dense(A, torch.bfloat16, "A"), _dense(Bt, torch.bfloat16, "Bt"), scale, A.shape[0])
        if (arr[k].A or 0) % 16:
            raise QmmError(4, "make_lora_adapters")
    table = torch.frombuffer(bytearray(bytes(arr)), dtype=torch.uint8).to(first[0].device)
    table.lora_shape = first[1].shape[1], first[0].shape[1]   # N, K, for make_lora_entries()
    table._keep = tuple(items)
    return table


def make_lora_entries(items):
    """items: sequence of (adapters, X, Y0, Y, N, K): the table of make_lora_adapters(), X bf16 M x K, Y0
    and Y fp32 M x N (they may be one tensor), all contiguous.  The tensors are kept alive by what is
    returned."""
    import torch
    arr = (_LoraEntry * len(items))()
    for k, (table, X, Y0, Y, N, K) in enumerate(items):
        if getattr(table, "lora_shape", (N, K)) != (N, K):
            raise QmmError(2, "make_lora_entries: adapters of another projection")
        if X.dim() != 2 or X.shape[1] != K:
            raise QmmError(2, "X")
        for t, name in ((Y0, "Y0"), (Y, "Y")):
            if t.dim() != 2 or t.shape[0] != X.shape[0] or t.shape[1] != N:
                raise QmmError(2, name)
        arr[k] = _LoraEntry(_dense(table, torch.uint8, "adapters"), table.numel() // ctypes.sizeof(_LoraAdapter),
                            _dense(X, torch.bfloat16, "X"), _dense(Y0, torch.float32, "Y0"), _dense(Y, torch.float32, "Y"),
                            N, K)
    arr._keep = tuple(items)
    arr._rows, arr._ids_type = min((item[1].shape[0] for item in items), default=0), torch.int32   # for run_lora()
    return arr


def lora_workspace_bytes(entries, M: int, rank_max: int) -> int:
    return load().qmm_lora_workspace_bytes(entries, len(entries), M, rank_max)


def run_lora(entries, ids, M: int, rank_max: int, workspace, stream=None) -> None:
    """qmm_run_lora: Y[i] = Y0[i] + scale * B (A x_i) with the adapter ids[i] (int32 device tensor, -1:
    none) for each projection of `entries` (make_lora_entries()).  rank_max: at least every rank in
    use; `workspace`: a device tensor of >= lora_workspace_bytes(entries, M, rank_max) bytes."""
    if ids.dtype is not entries._ids_type:
        raise QmmError(12, "ids")
    if M > entries._rows or ids.numel() < M or not ids.is_contiguous():
        raise QmmError(2, "run_lora: M rows, M dense ids")
    _check(load().qmm_run_lora(entries, len(entries), ids.data_ptr(), M, rank_max, workspace.data_ptr(),
                               workspace.numel() * workspace.element_size(), _stream_handle(stream)), "qmm_run_lora")


def select_variant(M: int, N: int, K: int) -> int:
    return load().qmm_select_variant(M, N, K)


def select_variant_batched(entries, M: int) -> int:
    return load().qmm_select_variant_batched(entries, len(entries), M)


def stream_read(buf, sink, stream=None) -> None:
    """qmm_stream_read: read every byte of the device tensor `buf` once (the read-bandwidth probe);
    `sink` is a device uint32 tensor of at least qmm_stream_read_sink_words() words."""
    st = load().qmm_stream_read(ctypes.c_void_p(buf.data_ptr()), buf.numel() * buf.element_size(),
                                ctypes.c_void_p(sink.data_ptr()), _stream_handle(stream))
    _check(st, "qmm_stream_read")


def stream_read_sink_words() -> int:
    return int(load().qmm_stream_read_sink_words())


def set_wait_limit(polls: int = 0, suspend_ns: int = 0) -> None:
    """qmm_set_wait_limit: the tensor-core kernel's wait bound for later launches (0, 0: default)."""
    load().qmm_set_wait_limit(polls, suspend_ns)


def release() -> None:
    """qmm_release: free every tensor-core workspace the library holds (synchronous)."""
    _check(load().qmm_release(), "qmm_release")


def workspace_bytes_held() -> int:
    """qmm_workspace_bytes_held: device bytes the tensor-core workspaces hold now."""
    return int(load().qmm_workspace_bytes_held())


def device_status() -> int:
    v = ctypes.c_uint(0)
    _check(load().qmm_device_status(ctypes.byref(v)), "qmm_device_status")
    return v.value
