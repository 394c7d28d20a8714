"""MI355X (gfx950) microscaled FP8 matrix multiply -- Python binding.

Thin ctypes binding of ``libmxgemm.so`` (C ABI in include/mxgemm.h), with
the same entry-point names.  It only marshals arguments: every step of the
multiply runs in the library's HIP kernels.  PyTorch supplies device memory
and streams; it is imported before the library is loaded so that both use
the one HIP runtime already in the process.

If the library has not been built this module raises on use; there is no
fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch  # noqa: F401  (loads the process's HIP runtime first)

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmxgemm.so")

MXGEMM_FMT_E4M3 = 0
MXGEMM_FMT_E5M2 = 1
MXGEMM_FMT_E2M3 = 2
MXGEMM_FMT_E3M2 = 3
MXGEMM_FMT_E2M1 = 4
MXGEMM_OUT_F32 = 0
MXGEMM_OUT_BF16 = 1
MXGEMM_X_F32 = 0
MXGEMM_X_BF16 = 1
MXGEMM_VARIANT_AUTO = 0
MXGEMM_VARIANT_LARGE = 1
MXGEMM_VARIANT_SKINNY = 2
MXGEMM_VARIANT_LARGE_NATIVE = 3
MXGEMM_VARIANT_SKINNY_NATIVE = 4
MXGEMM_WORKSPACE_BYTES = 4096 + 256 * 64 * 112 * 4
MXGEMM_WORKSPACE_BYTES_LARGE = 4096 + 256 * 256 * 256 * 4
MXGEMM_NOALLOC_SCRATCH_BYTES = MXGEMM_WORKSPACE_BYTES
MXGEMM_SCALES_ROW_MAJOR = 0
MXGEMM_SCALES_PRESHUFFLED = 1

STATUS = {0: "MXGEMM_OK", 1: "MXGEMM_ERR_NULL", 2: "MXGEMM_ERR_FMT", 3: "MXGEMM_ERR_DTYPE",
          4: "MXGEMM_ERR_SHAPE", 5: "MXGEMM_ERR_ALIGN", 6: "MXGEMM_ERR_DEVICE",
          7: "MXGEMM_ERR_HIP", 8: "MXGEMM_ERR_HANDLE", 9: "MXGEMM_ERR_ALIAS",
          10: "MXGEMM_ERR_VARIANT", 11: "MXGEMM_ERR_WORKSPACE"}
STATUS_CODE = {v: k for k, v in STATUS.items()}

# name -> (restype, argtypes), in the order of include/mxgemm.h
_vp, _i32, _i64, _u8p = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
SIGNATURES = {
    "mxgemm_version": (_i32, []),
    "mxgemm_create": (_i32, [ctypes.POINTER(ctypes.c_void_p)]),
    "mxgemm_destroy": (_i32, [_vp]),
    "mxgemm_set_variant": (_i32, [_vp, _i32]),
    "mxgemm_set_workspace": (_i32, [_vp, _vp, ctypes.c_size_t, _vp]),
    "mxgemm_operand_buffer_bytes": (_i64, [_i32, _i32, _i64, _i64, _i64]),
    "mxgemm_set_operand_buffer": (_i32, [_vp, _vp, ctypes.c_size_t]),
    "mxgemm_widen": (_i32, [_vp, _vp, _i32, _i64, _i64, _u8p, _vp]),
    "mxgemm_set_splits": (_i32, [_vp, _i32]),
    "mxgemm_set_scale_layout": (_i32, [_vp, _i32]),
    "mxgemm_scale_bytes": (_i64, [_i32, _i64, _i64]),
    "mxgemm_preshuffle_scales": (_i32, [_vp, _u8p, _u8p, _i64, _i64, _vp]),
    "mxgemm_validate_args": (_i32, [_vp, _u8p, _i32, _vp, _u8p, _i32, _vp, _i64, _i64, _i64,
                                    _i32, _i32]),
    "mxgemm_run": (_i32, [_vp, _vp, _u8p, _i32, _vp, _u8p, _i32, _vp, _i64, _i64, _i64, _i32,
                          _i32, _vp]),
    "mxgemm_run_noalloc": (_i32, [_vp, _vp, _u8p, _i32, _vp, _u8p, _i32, _vp, _i64, _i64, _i64,
                                  _i32, _i32, _vp]),
    "mxgemm_validate_quantize": (_i32, [_vp, _i32, _i64, _i64, _i32, _u8p, _u8p]),
    "mxgemm_quantize": (_i32, [_vp, _vp, _i32, _i64, _i64, _i32, _u8p, _u8p, _vp]),
    "mxgemm_validate_block128": (_i32, [_vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _i64, _i64, _i64,
                                        _i32, _i32]),
    "mxgemm_run_block128": (_i32, [_vp, _vp, _vp, _i32, _vp, _vp, _i32, _i32, _vp, _i64, _i64, _i64,
                                   _i32, _i32, _vp]),
    "mxgemm_validate_quantize_block128": (_i32, [_vp, _i32, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp]),
    "mxgemm_quantize_block128": (_i32, [_vp, _vp, _i32, _i64, _i64, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "mxgemm_validate_cache_append": (_i32, [_vp, _vp, _vp, _vp, _i32, _i64]),
    "mxgemm_cache_append": (_i32, [_vp, _vp, _vp, _vp, _vp, _i32, _i64, _vp]),
    "mxgemm_cache_attention_workspace": (_i64, [_vp, _vp, _i32, _i64]),
    "mxgemm_validate_cache_attention": (_i32, [_vp, _vp, _vp, _i32, _i64, ctypes.c_float, _i64, _i64, _vp,
                                               _i64, _vp, _vp, ctypes.c_size_t]),
    "mxgemm_cache_attention": (_i32, [_vp, _vp, _vp, _vp, _i32, _i64, ctypes.c_float, _i64, _i64, _vp,
                                      _i64, _vp, _vp, ctypes.c_size_t, _vp]),
    "mxgemm_validate_copy": (_i32, [_vp, _vp, ctypes.c_uint64]),
    "mxgemm_copy": (_i32, [_vp, _vp, _vp, ctypes.c_uint64, _vp]),
    "mxgemm_status_string": (ctypes.c_char_p, [_i32]),
}

_lib = None


class CacheStruct(ctypes.Structure):
    """mxgemm_cache."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int), ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int)]


class BatchStruct(ctypes.Structure):
    """mxgemm_batch."""
    _fields_ = [("page_table", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("ctx_len", ctypes.c_void_p), ("seqs", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("max_q", ctypes.c_int64), ("max_ctx", ctypes.c_int64)]


class MxgemmError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)} ({status_string(code)})")


def load_library(path: str = LIB_PATH):
    """Load libmxgemm.so; raises if it has not been built."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it first "
                           "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(code: int) -> str:
    return load_library().mxgemm_status_string(int(code)).decode()


def _check(code: int, where: str):
    if code != 0:
        raise MxgemmError(code, where)


def mxgemm_version() -> int:
    return load_library().mxgemm_version()


def mxgemm_create() -> int:
    h = ctypes.c_void_p()
    _check(load_library().mxgemm_create(ctypes.byref(h)), "mxgemm_create")
    return h.value


def mxgemm_destroy(h: int) -> None:
    _check(load_library().mxgemm_destroy(h), "mxgemm_destroy")


def mxgemm_set_variant(h: int, variant: int) -> None:
    _check(load_library().mxgemm_set_variant(h, int(variant)), "mxgemm_set_variant")


# the current stream's handle without a Stream object around it (2.7 us less
# a call), where this torch has it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is None or _current_device is None or not torch.cuda.is_initialized():
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(_current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def mxgemm_set_workspace(h, ws, nbytes: int, stream=None) -> None:
    """Attach a device buffer of at least MXGEMM_WORKSPACE_BYTES (256-byte
    aligned) for split-K, or detach with ws=None; zeroes its counters on
    `stream`."""
    _check(load_library().mxgemm_set_workspace(h, _ptr(ws), int(nbytes),
                                               _stream(stream) if ws is not None else None),
           "mxgemm_set_workspace")


def mxgemm_operand_buffer_bytes(fmtA: int, fmtB: int, M: int, N: int, K: int) -> int:
    """Bytes of the operand buffer a widened format pair needs (0: the pair
    runs as it is, -1: invalid arguments)."""
    return int(load_library().mxgemm_operand_buffer_bytes(int(fmtA), int(fmtB), int(M), int(N),
                                                          int(K)))


def mxgemm_set_operand_buffer(h, buf, nbytes: int) -> None:
    """Attach a device buffer (256-byte aligned) for widened operands, or
    detach with buf=None."""
    _check(load_library().mxgemm_set_operand_buffer(h, _ptr(buf), int(nbytes) if buf is not None else 0),
           "mxgemm_set_operand_buffer")


def mxgemm_widen(h, src, fmt: int, rows: int, K: int, dst, stream=None) -> None:
    """rows x K sub-byte codes (e2m1 / e2m3 / e3m2) -> rows x K e4m3 bytes
    of the same values, on `stream` (default: torch's current stream)."""
    _check(load_library().mxgemm_widen(h, _ptr(src), int(fmt), int(rows), int(K), _ptr(dst),
                                       _stream(stream)),
           "mxgemm_widen")


def row_bytes(fmt: int, K: int) -> int:
    """Bytes of an operand row of K codes: e2m1 K/2, e2m3 and e3m2 3K/4,
    e4m3 / e5m2 K."""
    if fmt == MXGEMM_FMT_E2M1:
        return K // 2
    if fmt in (MXGEMM_FMT_E2M3, MXGEMM_FMT_E3M2):
        return 3 * K // 4
    return K


def codes_per_row(fmt: int, nbytes: int) -> int:
    """K of an operand row of `nbytes` bytes (the inverse of row_bytes)."""
    if fmt == MXGEMM_FMT_E2M1:
        return 2 * nbytes
    if fmt in (MXGEMM_FMT_E2M3, MXGEMM_FMT_E3M2):
        return 4 * nbytes // 3
    return nbytes


def mxgemm_set_splits(h, splits: int) -> None:
    """K splits of later calls: 0 automatic, 1 never, S >= 2 forced."""
    _check(load_library().mxgemm_set_splits(h, int(splits)), "mxgemm_set_splits")


def mxgemm_set_scale_layout(h, layout: int) -> None:
    """Scale layout of later multiplies and quantizations through h:
    MXGEMM_SCALES_ROW_MAJOR (default) or MXGEMM_SCALES_PRESHUFFLED."""
    _check(load_library().mxgemm_set_scale_layout(h, int(layout)), "mxgemm_set_scale_layout")


def mxgemm_scale_bytes(layout: int, rows: int, K: int) -> int:
    """Bytes of a rows x K operand's scale buffer in `layout` (0: invalid)."""
    return int(load_library().mxgemm_scale_bytes(int(layout), int(rows), int(K)))


def mxgemm_preshuffle_scales(h, src, dst, rows: int, K: int, stream=None) -> None:
    """Row-major scale bytes (rows x K/32) to the preshuffled layout, on
    `stream` (default: torch's current stream)."""
    _check(load_library().mxgemm_preshuffle_scales(h, _ptr(src), _ptr(dst), int(rows), int(K),
                                                   _stream(stream)),
           "mxgemm_preshuffle_scales")


def _ptr(x) -> int:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def mxgemm_validate_args(A, A_scale, fmtA, B, B_scale, fmtB, C, M, N, K, use_acc,
                         out_dtype) -> int:
    """Returns the status code (0 = valid); pure host check."""
    return load_library().mxgemm_validate_args(
        _ptr(A), _ptr(A_scale), int(fmtA), _ptr(B), _ptr(B_scale), int(fmtB), _ptr(C),
        int(M), int(N), int(K), int(use_acc), int(out_dtype))


def mxgemm_run(h, A, A_scale, fmtA, B, B_scale, fmtB, C, M, N, K, use_acc, out_dtype,
               stream=None) -> None:
    """C (+)= (A*2^(As-127)) @ (B*2^(Bs-127)) on `stream` (default: torch's
    current stream).  Tensors are passed by device pointer; shapes and dtypes
    are the caller's responsibility, as in the C ABI."""
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    _check(load_library().mxgemm_run(
        h, _ptr(A), _ptr(A_scale), int(fmtA), _ptr(B), _ptr(B_scale), int(fmtB), _ptr(C),
        int(M), int(N), int(K), int(use_acc), int(out_dtype), stream), "mxgemm_run")


def mxgemm_run_noalloc(h, A, A_scale, fmtA, B, B_scale, fmtB, C, M, N, K, use_acc, out_dtype,
                       stream=None) -> None:
    """mxgemm_run with the library's fixed split-K scratch instead of an
    attached workspace: allocates nothing (calls on one GPU must not overlap)."""
    _check(load_library().mxgemm_run_noalloc(
        h, _ptr(A), _ptr(A_scale), int(fmtA), _ptr(B), _ptr(B_scale), int(fmtB), _ptr(C),
        int(M), int(N), int(K), int(use_acc), int(out_dtype), _stream(stream)), "mxgemm_run_noalloc")


def mxgemm_validate_quantize(X, x_dtype, R, K, fmt, codes, scales) -> int:
    """Returns the status code (0 = valid); pure host check."""
    return load_library().mxgemm_validate_quantize(
        _ptr(X), int(x_dtype), int(R), int(K), int(fmt), _ptr(codes), _ptr(scales))


def mxgemm_quantize(h, X, x_dtype, R, K, fmt, codes, scales, stream=None) -> None:
    """MX block quantization of the R x K matrix X into codes (R x K) and
    scales (R x K/32) on `stream` (default: torch's current stream)."""
    if stream is None:
        stream = torch.cuda.current_stream().cuda_stream
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    _check(load_library().mxgemm_quantize(
        h, _ptr(X), int(x_dtype), int(R), int(K), int(fmt), _ptr(codes), _ptr(scales), stream),
        "mxgemm_quantize")


def mxgemm_validate_block128(A, A_scale, fmtA, B, B_scale, fmtB, b_rows, C, M, N, K, use_acc,
                             out_dtype) -> int:
    """Returns the status code (0 = valid); pure host check."""
    return load_library().mxgemm_validate_block128(
        _ptr(A), _ptr(A_scale), int(fmtA), _ptr(B), _ptr(B_scale), int(fmtB), int(b_rows), _ptr(C),
        int(M), int(N), int(K), int(use_acc), int(out_dtype))


def mxgemm_run_block128(h, A, A_scale, fmtA, B, B_scale, fmtB, b_rows, C, M, N, K, use_acc, out_dtype,
                        stream=None) -> None:
    """C (+)= the product of codes with one fp32 scale per 128 K (B: per
    b_rows x 128) on `stream` (default: torch's current stream)."""
    _check(load_library().mxgemm_run_block128(
        h, _ptr(A), _ptr(A_scale), int(fmtA), _ptr(B), _ptr(B_scale), int(fmtB), int(b_rows), _ptr(C),
        int(M), int(N), int(K), int(use_acc), int(out_dtype), _stream(stream)), "mxgemm_run_block128")


def mxgemm_validate_quantize_block128(X, x_dtype, R, K, rows, fmt, codes, scales, codes_t, scales_t) -> int:
    """Returns the status code (0 = valid); pure host check."""
    return load_library().mxgemm_validate_quantize_block128(
        _ptr(X), int(x_dtype), int(R), int(K), int(rows), int(fmt), _ptr(codes), _ptr(scales),
        _ptr(codes_t), _ptr(scales_t))


def mxgemm_quantize_block128(h, X, x_dtype, R, K, rows, fmt, codes, scales, codes_t, scales_t,
                             stream=None) -> None:
    """Quantization of the R x K matrix X in blocks of `rows` x 128, and of
    its transpose, on `stream` (default: torch's current stream); either
    pair of outputs may be None."""
    _check(load_library().mxgemm_quantize_block128(
        h, _ptr(X), int(x_dtype), int(R), int(K), int(rows), int(fmt), _ptr(codes), _ptr(scales),
        _ptr(codes_t), _ptr(scales_t), _stream(stream)), "mxgemm_quantize_block128")


def _ref(x):
    return None if x is None else ctypes.addressof(x)


def mxgemm_validate_cache_append(cache, batch, K, V, x_dtype, kv_stride) -> int:
    """Returns the status code (0 = valid); pure host check.  `cache` and
    `batch` are a CacheStruct and a BatchStruct."""
    return load_library().mxgemm_validate_cache_append(_ref(cache), _ref(batch), _ptr(K), _ptr(V),
                                                       int(x_dtype), int(kv_stride))


def mxgemm_cache_append(h, cache, batch, K, V, x_dtype, kv_stride, stream=None) -> None:
    """Stores the batch's new tokens in the cache on `stream` (default:
    torch's current stream)."""
    _check(load_library().mxgemm_cache_append(h, _ref(cache), _ref(batch), _ptr(K), _ptr(V), int(x_dtype),
                                              int(kv_stride), _stream(stream)), "mxgemm_cache_append")


def mxgemm_cache_attention_workspace(cache, batch, q_heads, window=0) -> int:
    """Bytes of the workspace that lets this call split its keys (0: it would
    not split, -1: invalid arguments)."""
    return int(load_library().mxgemm_cache_attention_workspace(_ref(cache), _ref(batch), int(q_heads),
                                                               int(window)))


def mxgemm_validate_cache_attention(cache, batch, Q, q_heads, q_stride, softmax_scale, window, sinks, O,
                                    o_stride, lse, ws, ws_bytes) -> int:
    """Returns the status code (0 = valid); pure host check."""
    return load_library().mxgemm_validate_cache_attention(
        _ref(cache), _ref(batch), _ptr(Q), int(q_heads), int(q_stride), float(softmax_scale), int(window),
        int(sinks), _ptr(O), int(o_stride), _ptr(lse), _ptr(ws), int(ws_bytes))


def mxgemm_cache_attention(h, cache, batch, Q, q_heads, q_stride, softmax_scale, window, sinks, O,
                           o_stride, lse, ws, ws_bytes, stream=None) -> None:
    """Attention of the batch's new tokens over the cache on `stream`
    (default: torch's current stream)."""
    _check(load_library().mxgemm_cache_attention(
        h, _ref(cache), _ref(batch), _ptr(Q), int(q_heads), int(q_stride), float(softmax_scale),
        int(window), int(sinks), _ptr(O), int(o_stride), _ptr(lse), _ptr(ws), int(ws_bytes),
        _stream(stream)), "mxgemm_cache_attention")


def mxgemm_validate_copy(dst, src, nbytes) -> int:
    """Returns the status code (0 = valid); pure host check."""
    return load_library().mxgemm_validate_copy(_ptr(dst), _ptr(src), int(nbytes))


def mxgemm_copy(h, dst, src, nbytes, stream=None) -> None:
    """Streaming copy of nbytes from src to dst on `stream` (default: torch's
    current stream); the achievable-bandwidth reference of the benchmark."""
    _check(load_library().mxgemm_copy(h, _ptr(dst), _ptr(src), int(nbytes), _stream(stream)),
           "mxgemm_copy")


class Gemm:
    """Owns one handle; call(...) checks tensor shapes and runs."""

    def __init__(self):
        self.h = mxgemm_create()
        self.lib = load_library()
        self.device = torch.cuda.current_device()   # the handle's
        self.scale_layout = MXGEMM_SCALES_ROW_MAJOR

    def close(self):
        if self.h:
            mxgemm_destroy(self.h)
            self.h = None

    def __del__(self):  # pragma: no cover
        try:
            self.close()
        except Exception:
            pass

    def set_variant(self, variant: int):
        mxgemm_set_variant(self.h, variant)

    def enable_split_k(self, device="cuda:0", stream=None, nbytes=MXGEMM_WORKSPACE_BYTES_LARGE):
        """Give the handle its own split-K workspace (a torch allocation that
        this object keeps alive); calls through this handle must then be
        ordered on one stream.  The default size never limits a split."""
        if getattr(self, "workspace", None) is None:
            self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
            mxgemm_set_workspace(self.h, self.workspace, nbytes, stream)

    def disable_split_k(self):
        if getattr(self, "workspace", None) is not None:
            mxgemm_set_workspace(self.h, None, 0)
            self.workspace = None

    def set_splits(self, splits: int):
        mxgemm_set_splits(self.h, splits)

    def ensure_operand_buffer(self, fmtA, fmtB, M, N, K, device="cuda:0"):
        """Attach an operand buffer large enough for a widened pair (a torch
        allocation this object keeps, grown as needed); calls through this
        handle must then be ordered on one stream."""
        need = mxgemm_operand_buffer_bytes(fmtA, fmtB, M, N, K)
        if need <= 0:
            return
        device = torch.device(device)
        cur = getattr(self, "opbuf", None)
        if cur is None or cur.numel() < need or cur.device != device:
            torch.cuda.synchronize(device)  # a call on any stream may still read the old buffer
            self.opbuf = torch.empty(need, dtype=torch.uint8, device=device)
            mxgemm_set_operand_buffer(self.h, self.opbuf, need)

    def set_scale_layout(self, layout: int):
        """Scales of later calls are row-major (R, K/32) tensors, or with
        MXGEMM_SCALES_PRESHUFFLED (ceil(R/32)*32, K/32) tensors holding the
        preshuffled bytes."""
        mxgemm_set_scale_layout(self.h, layout)
        self.scale_layout = layout

    def _scale_shape(self, rows: int, K: int):
        if self.scale_layout == MXGEMM_SCALES_PRESHUFFLED:
            return ((rows + 31) // 32 * 32, K // 32)
        return (rows, K // 32)

    def preshuffle_scales(self, S, stream=None):
        """A contiguous (R, K/32) uint8 device tensor of row-major scale
        bytes -> a new (ceil(R/32)*32, K/32) tensor in the preshuffled
        layout (padding rows zero)."""
        if S.dim() != 2 or S.dtype != torch.uint8 or not S.is_contiguous() or S.device.type != "cuda":
            raise ValueError("S must be a contiguous 2-D uint8 device tensor")
        R, kb = S.shape
        out = torch.empty(((R + 31) // 32 * 32, kb), dtype=torch.uint8, device=S.device)
        mxgemm_preshuffle_scales(self.h, S, out, R, 32 * kb, stream)
        return out

    def __call__(self, A, A_scale, fmtA, B, B_scale, fmtB, C, use_acc=False,
                 out_dtype=MXGEMM_OUT_F32, stream=None):
        # sub-byte operands are packed along K: e2m1 two codes per byte,
        # e2m3 / e3m2 four codes per three bytes
        M, ka = A.shape
        N = B.shape[0]
        K = codes_per_row(fmtA, ka)
        if B.shape[1] != row_bytes(fmtB, K) or A_scale.shape != self._scale_shape(M, K) or \
                B_scale.shape != self._scale_shape(N, K):
            raise ValueError("operand shapes do not match (A MxK, B NxK, scales K/32 per row, "
                             "preshuffled: rows padded to 32; e2m1: K/2 bytes per row, "
                             "e2m3 / e3m2: 3K/4)")
        want = torch.float32 if out_dtype == MXGEMM_OUT_F32 else torch.bfloat16
        if C.shape != (M, N) or C.dtype != want:
            raise ValueError(f"C must be ({M}, {N}) {want}")
        for t in (A, A_scale, B, B_scale, C):
            if not t.is_contiguous() or t.device.type != "cuda":
                raise ValueError("all operands must be contiguous device tensors")
        self.ensure_operand_buffer(fmtA, fmtB, M, N, K, A.device)
        mxgemm_run(self.h, A, A_scale, fmtA, B, B_scale, fmtB, C, M, N, K, int(bool(use_acc)),
                   out_dtype, stream)
        return C

    def quantize(self, X, fmt, codes=None, scales=None, stream=None):
        """MX block quantization of a contiguous (R, K) fp32 or bf16 device
        tensor; returns (codes (R, K) uint8, scales (R, K/32) uint8)."""
        if X.dim() != 2 or not X.is_contiguous() or X.device.type != "cuda":
            raise ValueError("X must be a contiguous 2-D device tensor")
        if X.dtype == torch.float32:
            xd = MXGEMM_X_F32
        elif X.dtype == torch.bfloat16:
            xd = MXGEMM_X_BF16
        else:
            raise ValueError("X must be float32 or bfloat16")
        R, K = X.shape
        kc = row_bytes(fmt, K)  # e2m1: two codes per byte; e2m3 / e3m2: four per three bytes
        if codes is None:
            codes = torch.empty((R, kc), dtype=torch.uint8, device=X.device)
        if scales is None:
            # preshuffled: the padding rows, which the quantizer does not
            # write, start as zeros
            scales = torch.zeros(self._scale_shape(R, K), dtype=torch.uint8, device=X.device)
        if codes.shape != (R, kc) or scales.shape != self._scale_shape(R, K) or \
                codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise ValueError("codes must be (R, K) (e2m1: (R, K/2), e2m3 / e3m2: (R, 3K/4)) and "
                             "scales (R, K/32) (preshuffled: rows padded to 32), uint8")
        mxgemm_quantize(self.h, X, xd, R, K, fmt, codes, scales, stream)
        return codes, scales

    def block128(self, A, A_scale, fmtA, B, B_scale, fmtB, C, use_acc=False, stream=None):
        """C (+)= (A * A_scale) @ (B * B_scale)^T for uint8 e4m3 / e5m2 codes A
        (M, K) and B (N, K) with fp32 scales A_scale (M, ceil(K / 128)) and
        B_scale (ceil(N / 128), ceil(K / 128)), or (N, ceil(K / 128)) for one
        scale per row; C (M, N) float32 or bfloat16."""
        if A.dim() != 2 or B.dim() != 2:
            raise ValueError("A must be (M, K) and B (N, K)")
        (M, K), (N, kB) = A.shape, B.shape
        kb, nb = (K + 127) // 128, (N + 127) // 128
        sb = B_scale.shape
        if kB != K or A_scale.shape != (M, kb) or (sb != (nb, kb) and sb != (N, kb)):
            raise ValueError("A must be (M, K), B (N, K), A_scale (M, ceil(K / 128)) and B_scale "
                             "(ceil(N / 128), ceil(K / 128)) or (N, ceil(K / 128))")
        f32 = C.dtype == torch.float32
        if C.shape != (M, N) or not (f32 or C.dtype == torch.bfloat16):
            raise ValueError(f"C must be ({M}, {N}) float32 or bfloat16")
        if A.dtype != torch.uint8 or B.dtype != torch.uint8 or A_scale.dtype != torch.float32 or \
                B_scale.dtype != torch.float32:
            raise ValueError("codes must be uint8 and scales float32")
        _on_device(self.device, A, A_scale, B, B_scale, C)
        if not (A.is_contiguous() and B.is_contiguous() and A_scale.is_contiguous() and
                B_scale.is_contiguous() and C.is_contiguous()):
            raise ValueError("all operands must be contiguous")
        # the library at once: a call of the wrapper costs a microsecond more
        rc = self.lib.mxgemm_run_block128(
            self.h, A.data_ptr(), A_scale.data_ptr(), fmtA, B.data_ptr(), B_scale.data_ptr(), fmtB,
            128 if sb[0] == nb else 1, C.data_ptr(), M, N, K, 1 if use_acc else 0,
            MXGEMM_OUT_F32 if f32 else MXGEMM_OUT_BF16, _stream_on(stream, self.device))
        if rc:
            _check(rc, "mxgemm_run_block128")
        return C

    def quantize_block128(self, X, fmt, rows=1, normal=True, transposed=False, stream=None):
        """Quantization of a contiguous (R, K) fp32 or bf16 device tensor in
        blocks of `rows` (1 or 128) x 128: (codes (R, K), scales) if `normal`,
        then (codes of the transpose (K, R rounded up to 16), their scales) if
        `transposed`."""
        if X.dim() != 2 or not X.is_contiguous():
            raise ValueError("X must be a contiguous 2-D device tensor")
        _on_device(self.device, X)
        if X.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("X must be float32 or bfloat16")
        if rows not in (1, 128):
            raise ValueError("rows must be 1 or 128")
        if not (normal or transposed):
            raise ValueError("nothing to compute: normal and transposed are both off")
        R, K = X.shape
        kb, rb = (K + 127) // 128, (R + 127) // 128
        with _on_stream(stream):
            if normal:
                c = X.new_empty((R, K), dtype=torch.uint8)
                sc = X.new_empty((R if rows == 1 else rb, kb), dtype=torch.float32)
            if transposed:
                ct = X.new_empty((K, (R + 15) // 16 * 16), dtype=torch.uint8)
                st = X.new_empty((K if rows == 1 else kb, rb), dtype=torch.float32)
        rc = self.lib.mxgemm_quantize_block128(
            self.h, X.data_ptr(), MXGEMM_X_F32 if X.dtype == torch.float32 else MXGEMM_X_BF16, R, K, rows, fmt,
            c.data_ptr() if normal else None, sc.data_ptr() if normal else None,
            ct.data_ptr() if transposed else None, st.data_ptr() if transposed else None,
            _stream_on(stream, self.device))
        if rc:
            _check(rc, "mxgemm_quantize_block128")
        return (c, sc) if not transposed else (c, sc, ct, st) if normal else (ct, st)


def _on_device(device, *tensors):
    for t in tensors:
        if t.get_device() != device:     # -1 on the host
            raise ValueError(f"all tensors must be on the handle's GPU (cuda:{device})")


def _stream_on(stream, device) -> int:
    """_stream for a call whose tensors are on `device`."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream(stream)


def _same_device(*tensors):
    d = tensors[0].get_device()     # -1 on the host
    for t in tensors:
        if t.get_device() != d or d < 0:
            raise ValueError("all tensors must be on one GPU")


_NOTHING = contextlib.nullcontext()


def _on_stream(stream):
    """The context in which a call on `stream` allocates, so that the memory
    is not handed out again before that stream is done with it."""
    if stream is None:
        return _NOTHING
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)


def _token_stride(t, heads: int, dim: int, what: str) -> int:
    """Elements between the tokens of a (tokens, heads, dim) tensor whose
    tokens are contiguous."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or t.stride(2) != 1 or \
            (heads > 1 and t.stride(1) != dim):
        raise ValueError(f"{what} must be (tokens, {heads}, {dim}) with contiguous tokens")
    return t.stride(0) if t.shape[0] > 1 else heads * dim


class Batch:
    """The sequences of one step: page_table (S, max_pages), q_start (S + 1)
    and ctx_len (S), int32 device tensors that the calls read when they run
    (mxgemm_batch).  max_q bounds the new tokens of a sequence; max_ctx is
    the longest context expected and only shapes the launch (default: the
    page table's reach, given the cache)."""

    def __init__(self, page_table, q_start, ctx_len, max_q: int, max_ctx: int = None):
        if page_table.dim() != 2 or q_start.shape != (page_table.shape[0] + 1,) or \
                ctx_len.shape != (page_table.shape[0],):
            raise ValueError("page_table must be (S, max_pages), q_start (S + 1,), ctx_len (S,)")
        _same_device(page_table, q_start, ctx_len)
        for t in (page_table, q_start, ctx_len):
            if t.dtype != torch.int32 or not t.is_contiguous():
                raise ValueError("page_table, q_start and ctx_len must be contiguous int32")
        self.tensors = (page_table, q_start, ctx_len)   # kept alive
        self.max_q, self.max_ctx = int(max_q), None if max_ctx is None else int(max_ctx)
        self.device = page_table.get_device()
        self._structs = {}

    def struct(self, cache, rows: int) -> BatchStruct:
        """The mxgemm_batch of a call on `rows` tokens over `cache`."""
        key = (rows, cache.page_size, self.max_q, self.max_ctx)
        got = self._structs.get(key)
        if got is None:
            t, q, c = self.tensors
            reach = t.shape[1] * cache.page_size
            got = BatchStruct(t.data_ptr(), q.data_ptr(), c.data_ptr(), t.shape[0], t.shape[1], rows,
                              self.max_q, reach if self.max_ctx is None else self.max_ctx)
            if len(self._structs) < 64:
                self._structs[key] = got
        if self.device != cache.device:
            raise ValueError("the batch and the cache must be on one GPU")
        return got


class KVCache:
    """Keys and values of one attention layer as e4m3 codes in pages, one
    e8m0 scale byte per page and kv head (mxgemm_cache).  The tensors are the
    caller's: k_codes (pages, kv_heads, page_size, head_dim), v_codes (pages,
    kv_heads, head_dim, page_size), k_scales and v_scales (pages, kv_heads),
    all uint8."""

    def __init__(self, gemm: Gemm, k_codes, k_scales, v_codes, v_scales):
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be (pages, kv_heads, page_size, head_dim)")
        pages, heads, page, dim = k_codes.shape
        if v_codes.shape != (pages, heads, dim, page) or k_scales.shape != (pages, heads) or \
                v_scales.shape != (pages, heads):
            raise ValueError("v_codes must be (pages, kv_heads, head_dim, page_size), the scales "
                             "(pages, kv_heads)")
        _on_device(gemm.device, k_codes, k_scales, v_codes, v_scales)
        self.tensors = (k_codes, k_scales, v_codes, v_scales)
        for t in self.tensors:
            if t.dtype != torch.uint8 or not t.is_contiguous():
                raise ValueError("codes and scales must be contiguous uint8")
        self.gemm, self.device = gemm, gemm.device
        self.page_size, self.kv_heads, self.head_dim = page, heads, dim
        self.struct = CacheStruct(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                                  v_scales.data_ptr(), pages, page, heads, dim)

    @classmethod
    def empty(cls, gemm: Gemm, pages: int, page_size: int, kv_heads: int, head_dim: int):
        """A cache of new tensors (zeros) on the handle's GPU."""
        z = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=f"cuda:{gemm.device}")
        return cls(gemm, z(pages, kv_heads, page_size, head_dim), z(pages, kv_heads),
                   z(pages, kv_heads, head_dim, page_size), z(pages, kv_heads))

    def append(self, batch: Batch, K, V, stream=None):
        """Stores the batch's new tokens: K and V (tokens, kv_heads, head_dim),
        float32 or bfloat16; tokens may lie further apart (views of a fused
        projection)."""
        stride = _token_stride(K, self.kv_heads, self.head_dim, "K")
        if V.shape != K.shape or V.dtype != K.dtype or \
                _token_stride(V, self.kv_heads, self.head_dim, "V") != stride:
            raise ValueError("V must match K in shape, type and stride")
        if K.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("K and V must be float32 or bfloat16")
        if K.get_device() != self.device or V.get_device() != self.device:
            raise ValueError("K, V and the cache must be on one GPU")
        if K.shape[0] == 0:
            return
        b = batch.struct(self, K.shape[0])
        rc = self.gemm.lib.mxgemm_cache_append(
            self.gemm.h, ctypes.addressof(self.struct), ctypes.addressof(b), K.data_ptr(), V.data_ptr(),
            MXGEMM_X_F32 if K.dtype == torch.float32 else MXGEMM_X_BF16, stride,
            _stream_on(stream, self.device))
        if rc:
            _check(rc, "mxgemm_cache_append")

    def attend(self, batch: Batch, Q, scale: float = None, window: int = 0, sinks: int = 0, out=None,
               lse=None, stream=None):
        """Causal softmax attention of the batch's new tokens (appended
        before) over the cache: Q (tokens, q_heads, head_dim) bfloat16 ->
        (out like Q, lse (tokens, q_heads) float32).  scale defaults to
        head_dim ** -0.5; window > 0 hides keys that far back or further,
        except the first `sinks`.  Rows of out outside every sequence are not
        written."""
        if Q.dim() != 3 or Q.dtype != torch.bfloat16 or Q.get_device() != self.device:
            raise ValueError("Q must be a (tokens, q_heads, head_dim) bfloat16 tensor on the cache's GPU")
        T, heads, dim = Q.shape
        q_stride = _token_stride(Q, heads, self.head_dim, "Q")
        with _on_stream(stream):
            if out is None:
                out = Q.new_empty((T, heads, dim))
                o_stride = heads * dim
            else:
                if out.shape != Q.shape or out.dtype != torch.bfloat16 or out.get_device() != self.device:
                    raise ValueError("out must be bfloat16 like Q")
                o_stride = _token_stride(out, heads, dim, "out")
            if lse is None:
                lse = Q.new_empty((T, heads), dtype=torch.float32)
            elif lse.shape != (T, heads) or lse.dtype != torch.float32 or lse.get_device() != self.device or \
                    not lse.is_contiguous():
                raise ValueError("lse must be a contiguous (tokens, q_heads) float32")
            if T == 0:
                return out, lse
            b = batch.struct(self, T)
            # a workspace of its own for each call: calls on several streams and
            # captured graphs share none
            lib, at, b_at = self.gemm.lib, ctypes.addressof(self.struct), ctypes.addressof(b)
            n = max(lib.mxgemm_cache_attention_workspace(at, b_at, heads, window), 0)
            ws = Q.new_empty((n,), dtype=torch.uint8) if n else None
            rc = lib.mxgemm_cache_attention(
                self.gemm.h, at, b_at, Q.data_ptr(), heads, q_stride,
                self.head_dim ** -0.5 if scale is None else scale, window, sinks, out.data_ptr(), o_stride,
                lse.data_ptr(), ws.data_ptr() if n else None, n, _stream_on(stream, self.device))
            if rc:
                _check(rc, "mxgemm_cache_attention")
        return out, lse
