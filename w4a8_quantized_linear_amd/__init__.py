"""Python binding of libcider.so, the MI355X (gfx950) fused quantized linear
layer: per-token INT8 activation quantization, INT8 x INT8 -> INT32 product on
the matrix cores, fused dequantization to fp16 (W8A8 per channel, W8A8 per
group of 64 / 128, W4A8 with packed int4 weights), and of its 4-bit paged
key/value cache with attention over it (the cider_kv4_ functions).

This module only marshals arguments: every function has the name and the
argument order of the C function declared in include/cider.h, takes device
tensors (or raw integer device pointers) and a stream, and returns the
cider_status.  With ``check=True`` (the default) a non-zero status raises
CiderError.  All computation happens in the HIP kernels of libcider.so;
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY = os.path.join(_PKG, "libcider.so")

CIDER_OK = 0
CIDER_ERR_INVALID_ARG = 1
CIDER_ERR_UNSUPPORTED_SHAPE = 2
CIDER_ERR_MISALIGNED = 3
CIDER_ERR_NO_DEVICE = 4
CIDER_ERR_HIP = 5
CIDER_ERR_WORKSPACE = 6
CIDER_ERR_SCRATCH_LIMIT = 7
CIDER_NOALLOC_SCRATCH_BYTES = 64 << 20

PATH_AUTO, PATH_GEMV, PATH_GEMM = 0, 1, 2

EXPORTS = (
    "cider_is_available", "cider_status_str", "cider_quantize_weight", "cider_quantize_act",
    "cider_w8a8_gemm", "cider_w4a8_gemm", "cider_w8a8_gemm_i32", "cider_w4a8_gemm_i32",
    "cider_linear_workspace_bytes", "cider_linear_workspace_bytes_ex", "cider_w8a8_linear", "cider_w4a8_linear", "cider_set_path",
    "cider_quantize_weight_clipped", "cider_quantize_weight_ex", "cider_smooth_fold_weight",
    "cider_quantize_act_ex", "cider_gemm_ex", "cider_linear_ex", "cider_decode_linear",
    "cider_linear_ex_noalloc",
    "cider_kv4_cache_bytes", "cider_kv4_append", "cider_kv4_read", "cider_kv4_attention",
    "cider_kv4_attention_workspace_bytes", "cider_kv4_set_tiles", "cider_kv4_append_rotated",
    "cider_kv4_attention_shared", "cider_kv4_attention_shared_workspace_bytes",
    "cider_lora_add", "cider_lora_workspace_bytes",
)

KV4_PAGE_TOKENS = 64
LORA_MAX_SLICES = 8

CIDER_DTYPE_F16 = 0
CIDER_DTYPE_BF16 = 1


class CiderError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s failed: %s (status %d)" % (what, cider_status_str(status), status))


_KV4_BATCH = struct.Struct("4Q8qi4x")  # cider_kv4_batch's fields


class cider_kv4_batch(ctypes.Structure):
    """The batch of a cider_kv4_* call (the struct of include/cider.h): a paged
    4-bit key/value cache, its page table, and the rows and lengths of each
    sequence.  Tensors are kept alive as long as the object is."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("cache", "pages", "row_start", "kv_len")] +
                [(n, ctypes.c_int64) for n in ("batch", "rows", "max_rows", "max_kv_len", "max_pages",
                                               "num_pages", "kv_heads", "head_dim")] +
                [("group_size", ctypes.c_int)])

    def __init__(self, cache, pages, row_start, kv_len, batch, rows, max_rows, max_kv_len, max_pages,
                 num_pages, kv_heads, head_dim, group_size):
        # written in one piece: 13 assignments cost 0.35 us more, a tenth of a launch
        _KV4_BATCH.pack_into(self, 0, _ptr(cache) or 0, _ptr(pages) or 0, _ptr(row_start) or 0, _ptr(kv_len) or 0,
                             batch, rows, max_rows, max_kv_len, max_pages, num_pages, kv_heads, head_dim,
                             group_size)
        self._tensors = (cache, pages, row_start, kv_len)


_KV4_RUNS = struct.Struct("2Q3q")  # cider_kv4_runs' fields


class cider_kv4_runs(ctypes.Structure):
    """Runs of sequences that hold the same first pages (the struct of
    include/cider.h), for cider_kv4_attention_shared.  Tensors are kept alive as
    long as the object is."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("group_start", "shared_len")] +
                [(n, ctypes.c_int64) for n in ("groups", "max_rows", "max_shared_len")])

    def __init__(self, group_start, shared_len, groups, max_rows, max_shared_len):
        _KV4_RUNS.pack_into(self, 0, _ptr(group_start) or 0, _ptr(shared_len) or 0, groups, max_rows, max_shared_len)
        self._tensors = (group_start, shared_len)


_ROTATION = struct.Struct("5Q3qif")  # cider_rotation's fields


class cider_rotation(ctypes.Structure):
    """Norm weights and rotation of cider_kv4_append_rotated (the struct of
    include/cider.h).  pair_axis: bytes, or any row of whole numbers, one
    below `axes` for each pair; None with one axis.  Tensors and pair_axis are kept
    alive as long as the object is, so a program makes one for each step's
    positions, or one for all where the cache's positions serve."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("cos_sin", "positions", "q_weight", "k_weight", "pair_axis")] +
                [(n, ctypes.c_int64) for n in ("table_len", "rot_dim", "axes")] +
                [("interleaved", ctypes.c_int), ("eps", ctypes.c_float)])

    def __init__(self, cos_sin, table_len, rot_dim, interleaved=False, positions=None, axes=1, pair_axis=None,
                 q_weight=None, k_weight=None, eps=1e-6):
        axis = 0
        if pair_axis is not None and axes > 1:
            if not isinstance(pair_axis, bytes):
                pair_axis = bytes(int(i) for i in pair_axis)
            if len(pair_axis) != rot_dim // 2:
                raise ValueError("pair_axis has %d entries, rot_dim / 2 is %d" % (len(pair_axis), rot_dim // 2))
            axis = ctypes.cast(pair_axis, ctypes.c_void_p).value or 0
        _ROTATION.pack_into(self, 0, _ptr(cos_sin) or 0, _ptr(positions) or 0, _ptr(q_weight) or 0,
                            _ptr(k_weight) or 0, axis, table_len, rot_dim, axes, bool(interleaved), eps)
        self._kept = (cos_sin, positions, q_weight, k_weight, pair_axis)


_LORA = struct.Struct("3Q4q%dq" % LORA_MAX_SLICES)  # cider_lora's fields


class cider_lora(ctypes.Structure):
    """The adapters of cider_lora_add (the struct of include/cider.h).
    slice_end: a row of numbers, where the outputs of each slice end; of one
    number for a plain product.  Tensors are kept alive as long as the object is."""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("a", "b", "scale")] +
                [(n, ctypes.c_int64) for n in ("slots", "rank", "in_features", "slices")] +
                [("slice_end", ctypes.c_int64 * LORA_MAX_SLICES)])

    def __init__(self, a, b, scale, slots, rank, in_features, slice_end):
        ends = tuple(slice_end)
        _LORA.pack_into(self, 0, _ptr(a) or 0, _ptr(b) or 0, _ptr(scale) or 0, slots, rank, in_features, len(ends),
                        *(ends + (0,) * LORA_MAX_SLICES)[:LORA_MAX_SLICES])
        self._tensors = (a, b, scale)


_lib: ctypes.CDLL | None = None


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libcider.so.  When it has never been built, build it first (hipcc
    for gfx950); a load failure raises, there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY):
        if not build_if_missing:
            raise ImportError("libcider.so is not built (run __graft_entry__.build())")
        from . import build as _build
        _build.build(force=True)
    lib = ctypes.CDLL(LIBRARY)
    P, I64, I, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sig = {
        "cider_is_available": ([], I),
        "cider_status_str": ([I], ctypes.c_char_p),
        "cider_quantize_weight": ([P, I64, I64, I, I, P, P, P], I),
        "cider_quantize_act": ([P, I64, I64, I64, P, P, P], I),
        "cider_quantize_weight_clipped": ([P, I64, I64, I, I, ctypes.c_double, P, P, P], I),
        "cider_quantize_weight_ex": ([P, I, I64, I64, I, I, ctypes.c_double, P, P, P], I),
        "cider_smooth_fold_weight": ([P, I, I64, I64, P, P, P], I),
        "cider_quantize_act_ex": ([P, I, I64, I64, I64, P, P, P, P], I),
        "cider_gemm_ex": ([P, P, P, P, I64, I64, I64, I, I, I, P, P], I),
        "cider_linear_ex": ([P, I, I64, I64, I64, P, P, P, I64, I, I, I, P, SZ, P, P], I),
        "cider_linear_ex_noalloc": ([P, I, I64, I64, I64, P, P, P, I64, I, I, I, P, P], I),
        "cider_decode_linear": ([P, I64, P, P, I64, I, I, I, P, P], I),
        "cider_w8a8_gemm": ([P, P, P, P, I64, I64, I64, I, P, P], I),
        "cider_w4a8_gemm": ([P, P, P, P, I64, I64, I64, I, P, P], I),
        "cider_w8a8_gemm_i32": ([P, P, I64, I64, I64, I, P, P], I),
        "cider_w4a8_gemm_i32": ([P, P, I64, I64, I64, I, P, P], I),
        "cider_linear_workspace_bytes": ([I64, I64], SZ),
        "cider_linear_workspace_bytes_ex": ([I64, I64, I64, I, I], SZ),
        "cider_w8a8_linear": ([P, I64, I64, I64, P, P, I64, I, P, SZ, P, P], I),
        "cider_w4a8_linear": ([P, I64, I64, I64, P, P, I64, I, P, SZ, P, P], I),
        "cider_set_path": ([I], I),
        "cider_lora_add": ([P, P, P, I64, I64, I64, P, I, I64, P, I64, P, SZ, P, I64, P], I),
        "cider_lora_workspace_bytes": ([P, I64, I64, I64], SZ),
        "cider_kv4_cache_bytes": ([I64, I64, I64, I], SZ),
        "cider_kv4_append": ([P, P, P, I, I64, I64, P], I),
        "cider_kv4_read": ([P, P, P, I, I64, I64, P], I),
        "cider_kv4_append_rotated": ([P, P, P, P, P, I, I64, I64, I64, I64, P, I64, P], I),
        "cider_kv4_attention": ([P, P, I, I64, I64, ctypes.c_float, I64, I64, P, SZ, P, I, I64, P], I),
        "cider_kv4_attention_workspace_bytes": ([P, I64, I64, I64], SZ),
        "cider_kv4_attention_shared": ([P, P, P, I, I64, I64, ctypes.c_float, P, SZ, P, I, I64, P], I),
        "cider_kv4_attention_shared_workspace_bytes": ([P, P, I64], SZ),
        "cider_kv4_set_tiles": ([I], I),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _ptr(t) -> int | None:
    try:
        return t.data_ptr()
    except AttributeError:
        if t is None or isinstance(t, int):
            return t
        raise


_raw_stream = None


def _current_stream() -> int | None:
    """torch's current stream as a raw handle.  The Stream object that
    torch.cuda.current_stream() builds costs 2.7 us a call, as much as a
    launch, so the handle is asked for directly where torch offers that."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        if not torch.cuda.is_available():
            return None
        get, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        torch.cuda.init()
        _raw_stream = ((lambda: get(device())) if get and device
                       else (lambda: torch.cuda.current_stream().cuda_stream))
    return _raw_stream()


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ret(status: int, what: str, check: bool) -> int:
    if check and status != CIDER_OK:
        raise CiderError(status, what)
    return status


def _struct(b):
    """The address of a call's struct."""
    return None if b is None else ctypes.addressof(b)


def cider_is_available() -> bool:
    return bool(load().cider_is_available())


def cider_status_str(status: int) -> str:
    return load().cider_status_str(int(status)).decode()


def cider_quantize_weight(w_f16, N, K, bits, group_size, wq, s_w, stream=None, check=True):
    st = load().cider_quantize_weight(_ptr(w_f16), N, K, bits, group_size, _ptr(wq), _ptr(s_w),
                                      _stream(stream))
    return _ret(st, "cider_quantize_weight", check)


def cider_quantize_weight_clipped(w_f16, N, K, bits, group_size, clip_percentile, wq, s_w,
                                  stream=None, check=True):
    st = load().cider_quantize_weight_clipped(_ptr(w_f16), N, K, bits, group_size,
                                              float(clip_percentile), _ptr(wq), _ptr(s_w),
                                              _stream(stream))
    return _ret(st, "cider_quantize_weight_clipped", check)


def cider_quantize_weight_ex(w, w_dtype, N, K, bits, group_size, clip_percentile, wq, s_w,
                             stream=None, check=True):
    st = load().cider_quantize_weight_ex(_ptr(w), w_dtype, N, K, bits, group_size,
                                         float(clip_percentile), _ptr(wq), _ptr(s_w),
                                         _stream(stream))
    return _ret(st, "cider_quantize_weight_ex", check)


def cider_smooth_fold_weight(w, w_dtype, N, K, smooth, w_out, stream=None, check=True):
    st = load().cider_smooth_fold_weight(_ptr(w), w_dtype, N, K, _ptr(smooth), _ptr(w_out),
                                         _stream(stream))
    return _ret(st, "cider_smooth_fold_weight", check)


def cider_quantize_act_ex(x, x_dtype, M, K, ldx, smooth, xq, s_tok, stream=None, check=True):
    st = load().cider_quantize_act_ex(_ptr(x), x_dtype, M, K, ldx, _ptr(smooth), _ptr(xq),
                                      _ptr(s_tok), _stream(stream))
    return _ret(st, "cider_quantize_act_ex", check)


def cider_gemm_ex(xq, s_tok, wq, s_w, M, N, K, bits, group_size, y_dtype, y, stream=None,
                  check=True):
    st = load().cider_gemm_ex(_ptr(xq), _ptr(s_tok), _ptr(wq), _ptr(s_w), M, N, K, bits,
                              group_size, y_dtype, _ptr(y), _stream(stream))
    return _ret(st, "cider_gemm_ex", check)


def cider_linear_ex(x, x_dtype, M, K, ldx, smooth, wq, s_w, N, bits, group_size, y_dtype,
                    workspace, workspace_bytes, y, stream=None, check=True):
    st = load().cider_linear_ex(_ptr(x), x_dtype, M, K, ldx, _ptr(smooth), _ptr(wq), _ptr(s_w),
                                N, bits, group_size, y_dtype, _ptr(workspace), workspace_bytes,
                                _ptr(y), _stream(stream))
    return _ret(st, "cider_linear_ex", check)


def cider_linear_ex_noalloc(x, x_dtype, M, K, ldx, smooth, wq, s_w, N, bits, group_size, y_dtype,
                            y, stream=None, check=True):
    st = load().cider_linear_ex_noalloc(_ptr(x), x_dtype, M, K, ldx, _ptr(smooth), _ptr(wq),
                                        _ptr(s_w), N, bits, group_size, y_dtype, _ptr(y),
                                        _stream(stream))
    return _ret(st, "cider_linear_ex_noalloc", check)


def cider_decode_linear(x_f16, K, wq, s_w, N, bits, group_size, y_dtype, y, stream=None,
                        check=True):
    st = load().cider_decode_linear(_ptr(x_f16), K, _ptr(wq), _ptr(s_w), N, bits, group_size,
                                    y_dtype, _ptr(y), _stream(stream))
    return _ret(st, "cider_decode_linear", check)


def cider_quantize_act(x_f16, M, K, ldx, xq, s_tok, stream=None, check=True):
    st = load().cider_quantize_act(_ptr(x_f16), M, K, ldx, _ptr(xq), _ptr(s_tok), _stream(stream))
    return _ret(st, "cider_quantize_act", check)


def cider_w8a8_gemm(xq, s_tok, wq, s_w, M, N, K, group_size, y_f16, stream=None, check=True):
    st = load().cider_w8a8_gemm(_ptr(xq), _ptr(s_tok), _ptr(wq), _ptr(s_w), M, N, K, group_size,
                                _ptr(y_f16), _stream(stream))
    return _ret(st, "cider_w8a8_gemm", check)


def cider_w4a8_gemm(xq, s_tok, wq4, s_w, M, N, K, group_size, y_f16, stream=None, check=True):
    st = load().cider_w4a8_gemm(_ptr(xq), _ptr(s_tok), _ptr(wq4), _ptr(s_w), M, N, K, group_size,
                                _ptr(y_f16), _stream(stream))
    return _ret(st, "cider_w4a8_gemm", check)


def cider_w8a8_gemm_i32(xq, wq, M, N, K, group_size, acc, stream=None, check=True):
    st = load().cider_w8a8_gemm_i32(_ptr(xq), _ptr(wq), M, N, K, group_size, _ptr(acc),
                                    _stream(stream))
    return _ret(st, "cider_w8a8_gemm_i32", check)


def cider_w4a8_gemm_i32(xq, wq4, M, N, K, group_size, acc, stream=None, check=True):
    st = load().cider_w4a8_gemm_i32(_ptr(xq), _ptr(wq4), M, N, K, group_size, _ptr(acc),
                                    _stream(stream))
    return _ret(st, "cider_w4a8_gemm_i32", check)


def cider_linear_workspace_bytes(M, K) -> int:
    return int(load().cider_linear_workspace_bytes(M, K))


def cider_linear_workspace_bytes_ex(M, N, K, bits, group_size) -> int:
    return int(load().cider_linear_workspace_bytes_ex(M, N, K, bits, group_size))


def cider_w8a8_linear(x_f16, M, K, ldx, wq, s_w, N, group_size, workspace, workspace_bytes,
                      y_f16, stream=None, check=True):
    st = load().cider_w8a8_linear(_ptr(x_f16), M, K, ldx, _ptr(wq), _ptr(s_w), N, group_size,
                                  _ptr(workspace), workspace_bytes, _ptr(y_f16), _stream(stream))
    return _ret(st, "cider_w8a8_linear", check)


def cider_w4a8_linear(x_f16, M, K, ldx, wq4, s_w, N, group_size, workspace, workspace_bytes,
                      y_f16, stream=None, check=True):
    st = load().cider_w4a8_linear(_ptr(x_f16), M, K, ldx, _ptr(wq4), _ptr(s_w), N, group_size,
                                  _ptr(workspace), workspace_bytes, _ptr(y_f16), _stream(stream))
    return _ret(st, "cider_w4a8_linear", check)


def cider_lora_add(lora, seg_start, slot, segments, rows, max_rows, x, dtype, ldx, y_in, ldy_in, workspace,
                   workspace_bytes, y, ldy, stream=None, check=True):
    st = load().cider_lora_add(_struct(lora), _ptr(seg_start), _ptr(slot), segments, rows, max_rows, _ptr(x), dtype,
                               ldx, _ptr(y_in), ldy_in, _ptr(workspace), workspace_bytes, _ptr(y), ldy,
                               _stream(stream))
    return _ret(st, "cider_lora_add", check)


def cider_lora_workspace_bytes(lora, segments, rows, max_rows) -> int:
    return int(load().cider_lora_workspace_bytes(_struct(lora), segments, rows, max_rows))


def cider_kv4_cache_bytes(num_pages, kv_heads, head_dim, group_size) -> int:
    return int(load().cider_kv4_cache_bytes(num_pages, kv_heads, head_dim, group_size))


def cider_kv4_append(b, k, v, dtype, ldk, ldv, stream=None, check=True):
    st = load().cider_kv4_append(_struct(b), _ptr(k), _ptr(v), dtype, ldk, ldv, _stream(stream))
    return _ret(st, "cider_kv4_append", check)


def cider_kv4_append_rotated(b, rotation, q, k, v, dtype, ldq, ldk, ldv, q_heads, q_out, ldq_out, stream=None,
                             check=True):
    st = load().cider_kv4_append_rotated(_struct(b), _struct(rotation), _ptr(q), _ptr(k), _ptr(v), dtype, ldq, ldk,
                                         ldv, q_heads, _ptr(q_out), ldq_out, _stream(stream))
    return _ret(st, "cider_kv4_append_rotated", check)


def cider_kv4_read(b, k, v, dtype, ldk, ldv, stream=None, check=True):
    st = load().cider_kv4_read(_struct(b), _ptr(k), _ptr(v), dtype, ldk, ldv, _stream(stream))
    return _ret(st, "cider_kv4_read", check)


def cider_kv4_attention(b, q, q_dtype, ldq, q_heads, scale, window, sinks, workspace,
                        workspace_bytes, y, y_dtype, ldy, stream=None, check=True):
    st = load().cider_kv4_attention(_struct(b), _ptr(q), q_dtype, ldq, q_heads, scale, window, sinks,
                                    _ptr(workspace), workspace_bytes, _ptr(y), y_dtype, ldy,
                                    _stream(stream))
    return _ret(st, "cider_kv4_attention", check)


def cider_kv4_attention_workspace_bytes(b, q_heads, window, sinks) -> int:
    return int(load().cider_kv4_attention_workspace_bytes(_struct(b), q_heads, window, sinks))


def cider_kv4_attention_shared(b, runs, q, q_dtype, ldq, q_heads, scale, workspace, workspace_bytes, y, y_dtype, ldy,
                               stream=None, check=True):
    st = load().cider_kv4_attention_shared(_struct(b), _struct(runs), _ptr(q), q_dtype, ldq, q_heads, scale,
                                           _ptr(workspace), workspace_bytes, _ptr(y), y_dtype, ldy, _stream(stream))
    return _ret(st, "cider_kv4_attention_shared", check)


def cider_kv4_attention_shared_workspace_bytes(b, runs, q_heads) -> int:
    return int(load().cider_kv4_attention_shared_workspace_bytes(_struct(b), _struct(runs), q_heads))


def cider_kv4_set_tiles(columns: int) -> int:
    return int(load().cider_kv4_set_tiles(int(columns)))


def cider_set_path(path: int) -> int:
    return int(load().cider_set_path(int(path)))
