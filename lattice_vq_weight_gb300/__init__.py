"""Thin Python binding of liblq (include/lq.h): argument marshalling only.

Every step of quantization and of the code-based products runs in the CUDA
kernels of ``liblq.so``; this module only turns torch tensors into pointers,
sizes and the current CUDA stream, and raises :class:`LQError` on a non-OK
status.  There is no fallback: if the library is missing, importing the
binding's entry points raises ImportError.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblq.so")

LQ_OK, LQ_ERR_ARG, LQ_ERR_SHAPE, LQ_ERR_DTYPE, LQ_ERR_CUDA, LQ_ERR_UNSUPPORTED = range(6)
LQ_DEV_NONFINITE, LQ_DEV_RANGE, LQ_DEV_TIMEOUT, LQ_DEV_FORMAT = 1, 2, 4, 8
LQ_Z1, LQ_A2, LQ_D4, LQ_E8 = 1, 2, 4, 8
LQ_F32, LQ_BF16 = 0, 1
LATTICE_IDS = {"z1": LQ_Z1, "a2": LQ_A2, "d4": LQ_D4, "e8": LQ_E8}
LATTICE_DIM = {"z1": 1, "a2": 2, "d4": 4, "e8": 8}

# (name, restype, argtypes) of every entry point declared in include/lq.h
_P, _I64, _U64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int, ctypes.c_float
SIGNATURES = {
    "lq_status_string": (ctypes.c_char_p, [_I32]),
    "lq_version": (_I32, []),
    "lq_pick_tile": (_I32, [_I64, _I32]),
    "lq_make_signs": (_I32, [_U64, _I64, _P, _P]),
    "lq_quantize": (_I32, [_I32, _P, _I32, _I64, _I64, _I64, _I32, _U64, _F32, _P, _P, _P, _P, _P]),
    "lq_quantize_grouped": (_I32, [_I32, _I32, _P, _I32, _P, _P, _P, _I32, _P, _F32, _P, _P, _P, _P, _P]),
    "lq_dequantize": (_I32, [_I32, _P, _P, _P, _I64, _I64, _I32, _P, _I32, _P]),
    "lq_quantize_ex": (_I32, [_I32, _P, _I32, _I64, _I64, _I64, _I32, _U64, _F32, _I32, _P, _P, _P, _P, _P]),
    "lq_dequantize_ex": (_I32, [_I32, _P, _P, _I32, _P, _I64, _I64, _I32, _P, _I32, _P]),
    "lq_gemv_ex": (_I32, [_I32, _P, _P, _I32, _P, _I64, _I64, _I32, _P, _I32, _I32, _P, _P, _P, _P]),
    "lq_gemm_ex": (_I32, [_I32, _P, _P, _I32, _P, _I64, _I64, _I32, _P, _I64, _P, _I32, _P, _P, _P]),
    "lq_attention_decode_ex": (_I32, [_I32, _P, _P, _P, _P, _P, _P, _I32, _I64, _I32, _I32, _I32, _P, _I32, _P,
                                      _P, ctypes.c_size_t, _P]),
    "lq_quantize_dithered": (_I32, [_I32, _P, _I32, _I64, _I64, _I64, _I32, _U64, _U64, _F32, _I32, _P, _P, _P,
                                    _P, _P]),
    "lq_dequantize_dithered": (_I32, [_I32, _P, _P, _I32, _P, _U64, _I64, _I64, _I32, _P, _I32, _P]),
    "lq_attention_decode_rice": (_I32, [_I32, _P, ctypes.c_size_t, _P, _P, _P, _P, ctypes.c_size_t, _P, _P, _P,
                                        _I32, _I64, _I32, _I32, _I32, _P, _I32, _P, _P, ctypes.c_size_t, _P]),
    "lq_attention_decode_dithered": (_I32, [_I32, _P, _P, _P, _U64, _P, _P, _P, _U64, _I32, _I64, _I32, _I32, _I32,
                                            _P, _I32, _P, _P, ctypes.c_size_t, _P]),
    "lq_gemv_workspace_size": (ctypes.c_size_t, [_I32, _I64, _I32]),
    "lq_gemv": (_I32, [_I32, _P, _P, _P, _I64, _I64, _I32, _P, _I32, _I32, _P, _P, _P, _P]),
    "lq_gemv_noalloc": (_I32, [_I32, _P, _P, _P, _I64, _I64, _I32, _P, _I32, _I32, _P, _P, _P]),
    "lq_gemv_grouped_workspace_size": (ctypes.c_size_t, [_I32, _I32, _I64, _I32]),
    "lq_gemv_grouped": (_I32, [_I32, _I32, _P, _P, _P, _P, _I64, _I32, _P, _I32, _I32, _P, _P, _P, _P]),
    "lq_gemm_workspace_size": (ctypes.c_size_t, [_I64, _I64, _I64, _I32]),
    "lq_gemm": (_I32, [_I32, _P, _P, _P, _I64, _I64, _I32, _P, _I64, _P, _I32, _P, _P, _P]),
    "lq_gemm_wait_expiry_test": (_I32, [_I32, _P, _P, _P, _I64, _I64, _I32, _P, _I64, _P, _I32, _P, _P, _P]),
    "lq_rice_stream_bound": (ctypes.c_size_t, [_I32, _I64, _I64, _I32]),
    "lq_rice_workspace_size": (ctypes.c_size_t, [_I64, _I64, _I32]),
    "lq_rice_encode": (_I32, [_I32, _P, _I64, _I64, _I32, _P, ctypes.c_size_t, _P, _P, _P, _P, _P]),
    "lq_rice_decode": (_I32, [_I32, _P, ctypes.c_size_t, _P, _I64, _I64, _I32, _P, _P]),
    "lq_gemv_rice": (_I32, [_I32, _P, ctypes.c_size_t, _P, _P, _P, _I64, _I64, _I32, _P, _I32, _I32, _P, _P,
                            _P, _P]),
    "lq_beta_for_snr": (ctypes.c_double, [_I32, ctypes.c_double]),
    "lq_error_sums": (_I32, [_P, _I32, _I64, _I64, _I64, _P, _P, _P]),
    "lq_calibrate_workspace_size": (ctypes.c_size_t, [_I32, _I64, _I64, _I32]),
    "lq_calibrate_bps": (_I32, [_I32, _I32, ctypes.c_double, _P, _I32, _I64, _I64, _I64, _U64, _P, ctypes.c_size_t,
                                _P, _P]),
    "lq_attention_workspace_size": (ctypes.c_size_t, [_I64, _I32, _I32, _I32]),
    "lq_attention_decode": (_I32, [_I32, _P, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _P, _I32, _P, _P,
                                   ctypes.c_size_t, _P]),
    "lq_rotate_blocks": (_I32, [_P, _I32, _I32, _P, _I32, _I64, _I64, _I64, _P, _I64, _P]),
    "lq_kv_plan": (_I32, [_P, _P, _I32, _I32, _P, _I64, _P, _I64, _I32, _P, _P, _P, _P, _I64, _P, _P, _P]),
    "lq_qk_norm_rope": (_I32, [_P, _I64, _I32, _P, _I64, _I32, _I32, _I64, _I32, _P, _P, _F32, _P, _P, _I64, _I32,
                               _I32, _P, _I64, _P, _I64, _P, _P]),
    "lq_kv_append": (_I32, [_P, _I64, _P, _I64, _I32, _I64, _P, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _P, _P]),
    "lq_kv_gather": (_I32, [_P, _I64, _P, _P, _P, _P, _I64, _I32, _I32, _I32, _P, _P, _I32, _P, _P]),
    "lq_attention_paged_workspace_size": (ctypes.c_size_t, [_I32, _I64, _I32, _I32, _I32]),
    "lq_attention_paged": (_I32, [_P, _I64, _I32, _I64, _P, _P, _I32, _P, _I64, _I32, _P, _P, _P, _P, _I64, _I32,
                                  _I32, _I32, _I32, _F32, _P, _I64, _P, ctypes.c_size_t, _P, _P]),
    "lq_verify_draft": (_I32, [_P, _P, _I32, _I32, _I64, _P, _I64, _I64, _P, _I64, _I64, _I32, _P, _P, _P, _P, _P,
                               _P]),
}


class LQError(RuntimeError):
    """A liblq entry point returned a status other than LQ_OK."""

    def __init__(self, name: str, status: int):
        super().__init__(f"{name} failed: status {status} ({status_string(status)})")
        self.status = status


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"liblq.so is not built ({LIB_PATH}); run `python -m lattice_vq_weight_gb300.build` "
            "or __graft_entry__.build()")
    dll = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(dll, name)
        fn.restype = res
        fn.argtypes = args
    return dll


_LIB = None


def _get_lib():
    global _LIB
    if _LIB is None:
        _LIB = _load()
    return _LIB


def __getattr__(name):
    if name == "lib":
        return _get_lib()
    raise AttributeError(name)


def status_string(status: int) -> str:
    return _get_lib().lq_status_string(int(status)).decode()


def _check(name: str, status: int) -> None:
    if status != LQ_OK:
        raise LQError(name, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is not None:
        return ctypes.c_void_p(int(stream))
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _lattice_id(lattice) -> int:
    return LATTICE_IDS[lattice] if isinstance(lattice, str) else int(lattice)


def _row_stride(W) -> int:
    """Row stride in elements; an empty matrix (whose stride torch may report as 0) passes its width."""
    return int(W.stride(0)) if W.shape[0] > 0 else int(W.shape[1])


def _dtype_id(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return LQ_BF16
    if t.dtype == torch.float32:
        return LQ_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


# ------------------------------------------------------------------ C-ABI calls
def lq_version() -> int:
    return _get_lib().lq_version()


def lq_pick_tile(cols: int, requested: int) -> int:
    return _get_lib().lq_pick_tile(int(cols), int(requested))


def lq_make_signs(seed: int, signs, stream=None) -> None:
    _check("lq_make_signs", _get_lib().lq_make_signs(int(seed), signs.numel(), _ptr(signs), _stream(stream)))


def lq_quantize(lattice, W, tile: int, seed: int, beta: float, codes, scales, signs,
                dev_status=None, stream=None) -> None:
    """W [rows x cols] (row stride W.stride(0)) -> codes, scales, signs (all preallocated)."""
    rows, cols = W.shape
    assert W.stride(1) == 1
    _check("lq_quantize", _get_lib().lq_quantize(
        _lattice_id(lattice), _ptr(W), _dtype_id(W), rows, cols, _row_stride(W), int(tile), int(seed),
        float(beta), _ptr(codes), _ptr(scales), _ptr(signs), _ptr(dev_status), _stream(stream)))


def lq_dequantize(lattice, codes, scales, signs, tile: int, W_hat, stream=None) -> None:
    rows, cols = codes.shape
    _check("lq_dequantize", _get_lib().lq_dequantize(
        _lattice_id(lattice), _ptr(codes), _ptr(scales), _ptr(signs), rows, cols, int(tile),
        _ptr(W_hat), _dtype_id(W_hat), _stream(stream)))


def lq_gemv_workspace_size(batch: int, cols: int, tile: int) -> int:
    return int(_get_lib().lq_gemv_workspace_size(int(batch), int(cols), int(tile)))


def lq_gemv(lattice, codes, scales, signs, tile: int, x, y, workspace, dev_status=None,
            stream=None) -> None:
    """y[b, r] = sum_t s[r,t] p[r,t,:] . x~[b,t,:]; x [batch x cols], y float32 [batch x rows]."""
    rows, cols = codes.shape
    batch = x.shape[0]
    _check("lq_gemv", _get_lib().lq_gemv(
        _lattice_id(lattice), _ptr(codes), _ptr(scales), _ptr(signs), rows, cols, int(tile),
        _ptr(x), _dtype_id(x), batch, _ptr(y), _ptr(workspace), _ptr(dev_status), _stream(stream)))


# Largest workspace lq_gemv_noalloc can serve (LQ_GEMV_NOALLOC_MAX_WORKSPACE in lq.h)
LQ_GEMV_NOALLOC_MAX_WORKSPACE = 4 * 1024 * 1024 + 64 * 1024


def lq_gemv_noalloc(lattice, codes, scales, signs, tile: int, x, y, dev_status=None, stream=None) -> None:
    """lq_gemv using the library's fixed device scratch instead of a caller workspace."""
    rows, cols = codes.shape
    batch = x.shape[0]
    _check("lq_gemv_noalloc", _get_lib().lq_gemv_noalloc(
        _lattice_id(lattice), _ptr(codes), _ptr(scales), _ptr(signs), rows, cols, int(tile),
        _ptr(x), _dtype_id(x), batch, _ptr(y), _ptr(dev_status), _stream(stream)))


# Largest group lq_quantize_grouped takes (LQ_QUANTIZE_MAX_GROUP in lq.h)
LQ_QUANTIZE_MAX_GROUP = 8


def lq_quantize_grouped(lattice, Ws, tile: int, seeds, beta: float, codes, scales, signs, dev_status=None,
                        stream=None) -> None:
    """lq_quantize for n matrices in one launch pair: lists Ws[m], seeds[m], codes[m], scales[m], signs[m].

    Every W has the same dtype; rows, cols and the row stride are taken per matrix."""
    n = len(Ws)
    if any(W.dtype != Ws[0].dtype for W in Ws):
        raise TypeError("lq_quantize_grouped: every matrix of a group has the same dtype")
    rows = (ctypes.c_int64 * n)(*[int(W.shape[0]) for W in Ws])
    cols = (ctypes.c_int64 * n)(*[int(W.shape[1]) for W in Ws])
    ldw = (ctypes.c_int64 * n)(*[_row_stride(W) for W in Ws])
    sd = (ctypes.c_uint64 * n)(*[int(x) & 0xFFFFFFFFFFFFFFFF for x in seeds])
    keep = [_ptr_array(Ws), _ptr_array(codes), _ptr_array(scales), _ptr_array(signs)]
    _check("lq_quantize_grouped", _get_lib().lq_quantize_grouped(
        _lattice_id(lattice), n, keep[0][1], _dtype_id(Ws[0]), ctypes.cast(rows, ctypes.c_void_p),
        ctypes.cast(cols, ctypes.c_void_p), ctypes.cast(ldw, ctypes.c_void_p), int(tile),
        ctypes.cast(sd, ctypes.c_void_p), float(beta), keep[1][1], keep[2][1], keep[3][1], _ptr(dev_status),
        _stream(stream)))


# Largest group lq_gemv_grouped takes (LQ_GEMV_MAX_GROUP in lq.h)
LQ_GEMV_MAX_GROUP = 8


def lq_gemv_grouped_workspace_size(n: int, batch: int, cols: int, tile: int) -> int:
    return int(_get_lib().lq_gemv_grouped_workspace_size(int(n), int(batch), int(cols), int(tile)))


def _ptr_array(tensors):
    arr = (ctypes.c_void_p * len(tensors))(*[None if t is None else t.data_ptr() for t in tensors])
    return arr, ctypes.cast(arr, ctypes.c_void_p)


def lq_gemv_grouped(lattice, codes, scales, signs, tile: int, x, ys, workspace, dev_status=None,
                    stream=None) -> None:
    """lq_gemv for n matrices sharing x: lists codes[m], scales[m], signs[m], ys[m]."""
    n = len(codes)
    cols = codes[0].shape[1]
    rows = (ctypes.c_int64 * n)(*[int(c.shape[0]) for c in codes])
    keep = [_ptr_array(codes), _ptr_array(scales), _ptr_array(signs), _ptr_array(ys)]
    _check("lq_gemv_grouped", _get_lib().lq_gemv_grouped(
        _lattice_id(lattice), n, keep[0][1], keep[1][1], keep[2][1], ctypes.cast(rows, ctypes.c_void_p),
        cols, int(tile), _ptr(x), _dtype_id(x), x.shape[0], keep[3][1], _ptr(workspace), _ptr(dev_status),
        _stream(stream)))


def lq_gemm_workspace_size(M: int, N: int, K: int, ydtype=LQ_F32) -> int:
    yd = ydtype if isinstance(ydtype, int) else _dtype_id(ydtype)
    return int(_get_lib().lq_gemm_workspace_size(int(M), int(N), int(K), yd))


def lq_gemm(lattice, codes, scales, signs, tile: int, X, Y, workspace, dev_status=None,
            stream=None) -> None:
    """Y [M x N] (float32 or bf16, Y's dtype) = X~ . (s p)^T from the codes [N x K]; X bf16 [M x K]."""
    N, K = codes.shape
    M = X.shape[0]
    _check("lq_gemm", _get_lib().lq_gemm(
        _lattice_id(lattice), _ptr(codes), _ptr(scales), _ptr(signs), N, K, int(tile), _ptr(X), M,
        _ptr(Y), _dtype_id(Y), _ptr(workspace), _ptr(dev_status), _stream(stream)))


def lq_gemm_wait_expiry_test(lattice, codes, scales, signs, tile: int, X, Y, workspace, dev_status,
                             stream=None) -> None:
    """The GEMM's wait-expiry self-test (lq.h): raises LQ_DEV_TIMEOUT in dev_status."""
    N, K = codes.shape
    _check("lq_gemm_wait_expiry_test", _get_lib().lq_gemm_wait_expiry_test(
        _lattice_id(lattice), _ptr(codes), _ptr(scales), _ptr(signs), N, K, int(tile), _ptr(X), X.shape[0],
        _ptr(Y), _dtype_id(Y), _ptr(workspace), _ptr(dev_status), _stream(stream)))


def lq_rice_stream_bound(lattice, rows: int, cols: int, tile: int) -> int:
    return int(_get_lib().lq_rice_stream_bound(_lattice_id(lattice), int(rows), int(cols), int(tile)))


def lq_rice_workspace_size(rows: int, cols: int, tile: int) -> int:
    return int(_get_lib().lq_rice_workspace_size(int(rows), int(cols), int(tile)))


def lq_rice_encode(lattice, codes, tile: int, stream_words, tile_offsets, total_bits, workspace,
                   dev_status=None, stream=None) -> None:
    """codes int8 [rows x cols] -> Rice stream (uint32 words, as int32 tensor), offsets, total bits."""
    rows, cols = codes.shape
    _check("lq_rice_encode", _get_lib().lq_rice_encode(
        _lattice_id(lattice), _ptr(codes), rows, cols, int(tile), _ptr(stream_words),
        stream_words.numel() * stream_words.element_size(), _ptr(tile_offsets), _ptr(total_bits),
        _ptr(workspace), _ptr(dev_status), _stream(stream)))


def lq_rice_decode(lattice, stream_words, tile_offsets, tile: int, codes, stream=None) -> None:
    rows, cols = codes.shape
    _check("lq_rice_decode", _get_lib().lq_rice_decode(
        _lattice_id(lattice), _ptr(stream_words), stream_words.numel() * stream_words.element_size(),
        _ptr(tile_offsets), rows, cols, int(tile), _ptr(codes), _stream(stream)))


def lq_gemv_rice(lattice, stream_words, tile_offsets, scales, signs, tile: int, x, y, workspace,
                 dev_status=None, stream=None) -> None:
    """lq_gemv from the Rice stream; y float32 [batch x rows]."""
    rows = tile_offsets.shape[0]
    cols = signs.numel()
    batch = x.shape[0]
    _check("lq_gemv_rice", _get_lib().lq_gemv_rice(
        _lattice_id(lattice), _ptr(stream_words), stream_words.numel() * stream_words.element_size(),
        _ptr(tile_offsets), _ptr(scales), _ptr(signs), rows, cols, int(tile), _ptr(x), _dtype_id(x), batch,
        _ptr(y), _ptr(workspace), _ptr(dev_status), _stream(stream)))


def lq_beta_for_snr(lattice, snr_db: float) -> float:
    return float(_get_lib().lq_beta_for_snr(_lattice_id(lattice), float(snr_db)))


def lq_error_sums(W, W_hat, sums, stream=None) -> None:
    """sums (float64 device tensor of 2) = (sum w^2, sum (w - w^)^2)."""
    rows, cols = W.shape
    _check("lq_error_sums", _get_lib().lq_error_sums(
        _ptr(W), _dtype_id(W), rows, cols, _row_stride(W), _ptr(W_hat), _ptr(sums), _stream(stream)))


def lq_calibrate_workspace_size(lattice, rows: int, cols: int, tile: int) -> int:
    return int(_get_lib().lq_calibrate_workspace_size(_lattice_id(lattice), int(rows), int(cols), int(tile)))


def lq_calibrate_bps(lattice, tile: int, target_bps: float, W, seed: int, workspace, stream=None):
    """(beta, bits per weight, SNR dB) of the scale that meets target_bps on the sample W (synchronous)."""
    rows, cols = W.shape
    out = (ctypes.c_double * 3)()
    _check("lq_calibrate_bps", _get_lib().lq_calibrate_bps(
        _lattice_id(lattice), int(tile), float(target_bps), _ptr(W), _dtype_id(W), rows, cols, _row_stride(W),
        int(seed), _ptr(workspace), workspace.numel(), ctypes.cast(out, ctypes.c_void_p), _stream(stream)))
    return float(out[0]), float(out[1]), float(out[2])


def lq_attention_workspace_size(tokens: int, kv_heads: int, q_heads: int, head_dim: int) -> int:
    return int(_get_lib().lq_attention_workspace_size(int(tokens), int(kv_heads), int(q_heads), int(head_dim)))


def lq_attention_decode(lattice, k_codes, k_scales, k_signs, v_codes, v_scales, v_signs, q, out, workspace,
                        stream=None) -> None:
    """out [q_heads x d] = softmax(K^ q / sqrt d) V^ from quantized caches [tokens x kv_heads*d]."""
    tokens = k_codes.shape[0]
    kv_heads = k_scales.shape[1]
    q_heads, head_dim = q.shape
    _check("lq_attention_decode", _get_lib().lq_attention_decode(
        _lattice_id(lattice), _ptr(k_codes), _ptr(k_scales), _ptr(k_signs), _ptr(v_codes), _ptr(v_scales),
        _ptr(v_signs), tokens, kv_heads, q_heads, head_dim, _ptr(q), _dtype_id(q), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))


# Scale formats (LQ_SCALE_* in lq.h)
LQ_SCALE_TILE_F32, LQ_SCALE_ROW_BF16, LQ_SCALE_TILE_F16 = 0, 1, 2
_SCALE_FORMATS = {"tile_f32": 0, "row_bf16": 1, "tile_f16": 2}


def _scale_format_id(fmt) -> int:
    return int(_SCALE_FORMATS.get(fmt, fmt))


def scales_tensor(rows: int, cols: int, tile: int, scale_format, device):
    """Empty scale tensor of the shape and dtype `scale_format` stores."""
    import torch
    f = _scale_format_id(scale_format)
    if f == LQ_SCALE_ROW_BF16:
        return torch.empty((rows,), dtype=torch.bfloat16, device=device)
    dt = torch.float16 if f == LQ_SCALE_TILE_F16 else torch.float32
    return torch.empty((rows, cols // tile), dtype=dt, device=device)


def lq_quantize_ex(lattice, W, tile: int, seed: int, beta: float, scale_format, codes, scales, signs,
                   dev_status=None, stream=None) -> None:
    """lq_quantize storing the scales in `scale_format` ("tile_f32", "row_bf16", "tile_f16")."""
    rows, cols = W.shape
    _check("lq_quantize_ex", _get_lib().lq_quantize_ex(
        _lattice_id(lattice), _ptr(W), _dtype_id(W), rows, cols, _row_stride(W), int(tile),
        int(seed) & 0xFFFFFFFFFFFFFFFF, float(beta), _scale_format_id(scale_format), _ptr(codes), _ptr(scales),
        _ptr(signs), _ptr(dev_status), _stream(stream)))


def quantize_ex(W, lattice: str = "e8", tile: int = 256, seed: int = 0, beta: float = 0.25,
                scale_format="tile_f32", dev_status=None, stream=None):
    """Allocate outputs and call :func:`lq_quantize_ex`; returns (codes, scales, signs)."""
    import torch
    rows, cols = W.shape
    codes = torch.empty((rows, cols), dtype=torch.int8, device=W.device)
    scales = scales_tensor(rows, cols, tile, scale_format, W.device)
    signs = torch.empty((cols,), dtype=torch.int8, device=W.device)
    lq_quantize_ex(lattice, W, tile, seed, beta, scale_format, codes, scales, signs, dev_status, stream)
    return codes, scales, signs


def lq_dequantize_ex(lattice, codes, scales, scale_format, signs, tile: int, W_hat, stream=None) -> None:
    rows, cols = codes.shape
    _check("lq_dequantize_ex", _get_lib().lq_dequantize_ex(
        _lattice_id(lattice), _ptr(codes), _ptr(scales), _scale_format_id(scale_format), _ptr(signs), rows, cols,
        int(tile), _ptr(W_hat), _dtype_id(W_hat), _stream(stream)))


def lq_gemv_ex(lattice, codes, scales, scale_format, signs, tile: int, x, y, workspace, dev_status=None,
               stream=None) -> None:
    rows, cols = codes.shape
    _check("lq_gemv_ex", _get_lib().lq_gemv_ex(
        _lattice_id(lattice), _ptr(codes), _ptr(scales), _scale_format_id(scale_format), _ptr(signs), rows, cols,
        int(tile), _ptr(x), _dtype_id(x), x.shape[0], _ptr(y), _ptr(workspace), _ptr(dev_status),
        _stream(stream)))


def lq_gemm_ex(lattice, codes, scales, scale_format, signs, tile: int, X, Y, workspace, dev_status=None,
               stream=None) -> None:
    N, K = codes.shape
    _check("lq_gemm_ex", _get_lib().lq_gemm_ex(
        _lattice_id(lattice), _ptr(codes), _ptr(scales), _scale_format_id(scale_format), _ptr(signs), N, K,
        int(tile), _ptr(X), X.shape[0], _ptr(Y), _dtype_id(Y), _ptr(workspace), _ptr(dev_status),
        _stream(stream)))


def lq_attention_decode_ex(lattice, k_codes, k_scales, k_signs, v_codes, v_scales, v_signs, scale_format, q, out,
                           workspace, stream=None) -> None:
    tokens = k_codes.shape[0]
    kv_heads = k_scales.shape[1]
    q_heads, head_dim = q.shape
    _check("lq_attention_decode_ex", _get_lib().lq_attention_decode_ex(
        _lattice_id(lattice), _ptr(k_codes), _ptr(k_scales), _ptr(k_signs), _ptr(v_codes), _ptr(v_scales),
        _ptr(v_signs), _scale_format_id(scale_format), tokens, kv_heads, q_heads, head_dim, _ptr(q), _dtype_id(q),
        _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def lq_quantize_dithered(lattice, W, tile: int, seed: int, dither_seed: int, beta: float, scale_format, codes,
                         scales, signs, dev_status=None, stream=None) -> None:
    """lq_quantize with the subtractive Voronoi dither of seed `dither_seed`."""
    rows, cols = W.shape
    _check("lq_quantize_dithered", _get_lib().lq_quantize_dithered(
        _lattice_id(lattice), _ptr(W), _dtype_id(W), rows, cols, _row_stride(W), int(tile),
        int(seed) & 0xFFFFFFFFFFFFFFFF, int(dither_seed) & 0xFFFFFFFFFFFFFFFF, float(beta),
        _scale_format_id(scale_format), _ptr(codes), _ptr(scales), _ptr(signs), _ptr(dev_status), _stream(stream)))


def quantize_dithered(W, lattice: str = "e8", tile: int = 128, seed: int = 0, dither_seed: int = 1,
                      beta: float = 0.25, scale_format="tile_f32", dev_status=None, stream=None):
    """Allocate outputs and call :func:`lq_quantize_dithered`; returns (codes, scales, signs)."""
    import torch
    rows, cols = W.shape
    codes = torch.empty((rows, cols), dtype=torch.int8, device=W.device)
    scales = scales_tensor(rows, cols, tile, scale_format, W.device)
    signs = torch.empty((cols,), dtype=torch.int8, device=W.device)
    lq_quantize_dithered(lattice, W, tile, seed, dither_seed, beta, scale_format, codes, scales, signs, dev_status,
                         stream)
    return codes, scales, signs


def lq_dequantize_dithered(lattice, codes, scales, scale_format, signs, dither_seed: int, tile: int, W_hat,
                           stream=None) -> None:
    rows, cols = codes.shape
    _check("lq_dequantize_dithered", _get_lib().lq_dequantize_dithered(
        _lattice_id(lattice), _ptr(codes), _ptr(scales), _scale_format_id(scale_format), _ptr(signs),
        int(dither_seed) & 0xFFFFFFFFFFFFFFFF, rows, cols, int(tile), _ptr(W_hat), _dtype_id(W_hat),
        _stream(stream)))


def lq_attention_decode_dithered(lattice, k_codes, k_scales, k_signs, k_dither_seed: int, v_codes, v_scales,
                                 v_signs, v_dither_seed: int, scale_format, q, out, workspace, stream=None) -> None:
    tokens = k_codes.shape[0]
    kv_heads = k_scales.shape[1]
    q_heads, head_dim = q.shape
    _check("lq_attention_decode_dithered", _get_lib().lq_attention_decode_dithered(
        _lattice_id(lattice), _ptr(k_codes), _ptr(k_scales), _ptr(k_signs), int(k_dither_seed) & 0xFFFFFFFFFFFFFFFF,
        _ptr(v_codes), _ptr(v_scales), _ptr(v_signs), int(v_dither_seed) & 0xFFFFFFFFFFFFFFFF,
        _scale_format_id(scale_format), tokens, kv_heads, q_heads, head_dim, _ptr(q), _dtype_id(q), _ptr(out),
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def lq_attention_decode_rice(lattice, k_stream, k_offsets, k_scales, k_signs, v_stream, v_offsets, v_scales,
                             v_signs, scale_format, q, out, workspace, stream=None) -> None:
    """Decode attention over Rice-coded caches (streams and offsets from lq_rice_encode, tile = head_dim)."""
    tokens, kv_heads = k_offsets.shape
    q_heads, head_dim = q.shape
    _check("lq_attention_decode_rice", _get_lib().lq_attention_decode_rice(
        _lattice_id(lattice), _ptr(k_stream), k_stream.numel() * k_stream.element_size(), _ptr(k_offsets),
        _ptr(k_scales), _ptr(k_signs), _ptr(v_stream), v_stream.numel() * v_stream.element_size(), _ptr(v_offsets),
        _ptr(v_scales), _ptr(v_signs), _scale_format_id(scale_format), tokens, kv_heads, q_heads, head_dim, _ptr(q),
        _dtype_id(q), _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def lq_rotate_blocks(R, X, Y, transpose: bool = False, stream=None) -> None:
    """Y (float32) = every 128-column block of X rotated by R (or R^T)."""
    rows, cols = X.shape
    _check("lq_rotate_blocks", _get_lib().lq_rotate_blocks(
        _ptr(R), int(bool(transpose)), R.shape[0], _ptr(X), _dtype_id(X), rows, cols, X.stride(0), _ptr(Y),
        Y.stride(0), _stream(stream)))


# ------------------------------------------------------------------ serving from a paged 8-bit KV cache
# Largest batch of the paged calls (LQ_MAX_REQUESTS in lq.h)
LQ_MAX_REQUESTS = 8192


def _addr(t):
    """Device address of a tensor (or None) as the plain number a call of every step passes quickest."""
    return None if t is None else t.data_ptr()


def _want(name: str, t, shape, *dtypes) -> None:
    """Raise unless t is contiguous with this shape and one of these dtypes: the kernels trust both."""
    if tuple(t.shape) != tuple(shape) or t.dtype not in dtypes or not t.is_contiguous():
        raise ValueError(f"{name}: want a contiguous {tuple(shape)} tensor of {' or '.join(map(str, dtypes))}, "
                         f"got {tuple(t.shape)} {t.dtype} with strides {tuple(t.stride())}")


def _heads(name: str, t) -> int:
    """Token stride of a [tokens x heads x head_dim] tensor whose heads are packed."""
    if t.dim() != 3 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
        raise ValueError(f"{name}: want [tokens x heads x head_dim] with packed heads, got {tuple(t.shape)} with "
                         f"strides {tuple(t.stride())}")
    return int(t.stride(0)) if t.shape[0] > 1 else int(t.shape[1] * t.shape[2])


def _cache(k_cache, k_scales, v_cache, v_scales):
    """(num_blocks, kv_heads, block_size, head_dim) of a cache's four tensors, checked."""
    import torch
    if k_cache.dim() != 4:
        raise ValueError(f"k_cache: want [num_blocks x kv_heads x block_size x head_dim], got {tuple(k_cache.shape)}")
    shape = tuple(k_cache.shape)
    _want("k_cache", k_cache, shape, torch.int8)
    _want("v_cache", v_cache, shape, torch.int8)
    _want("k_scales", k_scales, shape[:2], torch.float32)
    _want("v_scales", v_scales, shape[:2], torch.float32)
    return shape


def paged_cache(num_blocks: int, kv_heads: int, block_size: int, head_dim: int, device):
    """Empty cache pool: (k_cache, k_scales, v_cache, v_scales), codes int8
    [num_blocks x kv_heads x block_size x head_dim], scales float32 [num_blocks x kv_heads]."""
    import torch
    codes = [torch.empty((num_blocks, kv_heads, block_size, head_dim), dtype=torch.int8, device=device)
             for _ in range(2)]
    scales = [torch.zeros((num_blocks, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
    return codes[0], scales[0], codes[1], scales[1]


def lq_kv_plan(cached_lens, new_lens, block_size: int, free_blocks, block_table, cu_new, kv_lens, slots, positions,
               used, dev_status=None, stream=None) -> None:
    """Block table rows, slots and positions of the requests' new tokens (see lq.h); block_table is updated."""
    import torch
    b = cached_lens.numel()
    for n, t, shape in (("cached_lens", cached_lens, (b,)), ("new_lens", new_lens, (b,)),
                        ("free_blocks", free_blocks, (free_blocks.numel(),)), ("cu_new", cu_new, (b + 1,)),
                        ("kv_lens", kv_lens, (b,)), ("positions", positions, (slots.numel(),)), ("used", used, (1,))):
        _want(n, t, shape, torch.int32)
    _want("slots", slots, (slots.numel(),), torch.int64)
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.shape[0] != b or (
            block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError(f"block_table: want int32 [{b} x blocks], got {tuple(block_table.shape)} {block_table.dtype}")
    width = block_table.shape[1]
    _check("lq_kv_plan", _get_lib().lq_kv_plan(
        _addr(cached_lens), _addr(new_lens), b, int(block_size), _addr(free_blocks), free_blocks.numel(),
        _addr(block_table), block_table.stride(0) if b > 1 else width, width, _addr(cu_new), _addr(kv_lens),
        _addr(slots), _addr(positions), slots.numel(), _addr(used), _addr(dev_status), _stream(stream)))


def lq_qk_norm_rope(q, k, q_weight, k_weight, eps: float, positions, cos_sin, q_out, k_out, interleaved: bool = False,
                    dev_status=None, stream=None) -> None:
    """RMS norm of every head of q and k (weights None: none), then the rotation; q_out, k_out may be q, k."""
    import torch
    if not q.dtype == k.dtype == q_out.dtype == k_out.dtype:
        raise TypeError("lq_qk_norm_rope: q, k and their outputs have one dtype")
    tokens, hq, d = q.shape
    if k.shape[0] != tokens or k.shape[2] != d or q_out.shape != q.shape or k_out.shape != k.shape:
        raise ValueError("lq_qk_norm_rope: q, k and their outputs do not belong together")
    for n, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _want(n, w, (d,), torch.float32)
    _want("positions", positions, (tokens,), torch.int32)
    _want("cos_sin", cos_sin, tuple(cos_sin.shape[:1]) + (cos_sin.shape[-1],), torch.float32)
    _check("lq_qk_norm_rope", _get_lib().lq_qk_norm_rope(
        _addr(q), _heads("q", q), hq, _addr(k), _heads("k", k), k.shape[1], _dtype_id(q), tokens, d, _addr(q_weight),
        _addr(k_weight), float(eps), _addr(positions), _addr(cos_sin), cos_sin.shape[0], cos_sin.shape[1],
        int(bool(interleaved)), _addr(q_out), _heads("q_out", q_out), _addr(k_out), _heads("k_out", k_out),
        _addr(dev_status), _stream(stream)))


def lq_kv_append(k, v, slots, k_cache, k_scales, v_cache, v_scales, dev_status=None, stream=None) -> None:
    """Write k, v [tokens x kv_heads x head_dim] to the cache's slots (int64 [tokens], negative: left out)."""
    import torch
    nb, hk, bs, d = _cache(k_cache, k_scales, v_cache, v_scales)
    if k.shape != v.shape or k.dtype != v.dtype or tuple(k.shape[1:]) != (hk, d):
        raise ValueError(f"lq_kv_append: k and v do not fit the cache: {tuple(k.shape)}, {tuple(v.shape)}")
    _want("slots", slots, (k.shape[0],), torch.int64)
    _check("lq_kv_append", _get_lib().lq_kv_append(
        _addr(k), _heads("k", k), _addr(v), _heads("v", v), _dtype_id(k), k.shape[0], _addr(slots), _addr(k_cache),
        _addr(k_scales), _addr(v_cache), _addr(v_scales), nb, bs, hk, d, _addr(dev_status), _stream(stream)))


def lq_kv_gather(slots, k_cache, k_scales, v_cache, v_scales, k_out, v_out, dev_status=None, stream=None) -> None:
    """The values that the cache's slots stand for, [n x kv_heads x head_dim] float32 or bf16."""
    import torch
    nb, hk, bs, d = _cache(k_cache, k_scales, v_cache, v_scales)
    n = slots.numel()
    _want("slots", slots, (n,), torch.int64)
    _want("k_out", k_out, (n, hk, d), torch.float32, torch.bfloat16)
    _want("v_out", v_out, (n, hk, d), k_out.dtype)
    _check("lq_kv_gather", _get_lib().lq_kv_gather(
        _addr(slots), n, _addr(k_cache), _addr(k_scales), _addr(v_cache), _addr(v_scales), nb, bs, hk, d, _addr(k_out),
        _addr(v_out), _dtype_id(k_out), _addr(dev_status), _stream(stream)))


def lq_attention_paged_workspace_size(batch: int, total_q: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(_get_lib().lq_attention_paged_workspace_size(int(batch), int(total_q), int(q_heads), int(kv_heads),
                                                            int(head_dim)))


def lq_attention_paged(q, cu_q, kv_lens, block_table, k_cache, k_scales, v_cache, v_scales, out, workspace,
                       sm_scale=None, dev_status=None, stream=None) -> None:
    """out = attention of q [total_q x q_heads x head_dim] over the requests' cached tokens (see lq.h);
    sm_scale defaults to head_dim ** -0.5."""
    import torch
    nb, hk, bs, d = _cache(k_cache, k_scales, v_cache, v_scales)
    b = kv_lens.numel()
    _want("kv_lens", kv_lens, (b,), torch.int32)
    _want("cu_q", cu_q, (b + 1,), torch.int32)
    if q.shape != out.shape or q.dtype != out.dtype or q.shape[2] != d:
        raise ValueError(f"lq_attention_paged: q and out do not fit: {tuple(q.shape)}, {tuple(out.shape)}")
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or block_table.shape[0] != b or (
            block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError(f"block_table: want int32 [{b} x blocks], got {tuple(block_table.shape)} {block_table.dtype}")
    width = block_table.shape[1]
    _check("lq_attention_paged", _get_lib().lq_attention_paged(
        _addr(q), _heads("q", q), _dtype_id(q), q.shape[0], _addr(cu_q), _addr(kv_lens), b, _addr(block_table),
        block_table.stride(0) if b > 1 else width, width, _addr(k_cache), _addr(k_scales), _addr(v_cache),
        _addr(v_scales), nb, bs, q.shape[1], hk, d, d ** -0.5 if sm_scale is None else float(sm_scale), _addr(out),
        _heads("out", out), _addr(workspace), workspace.numel() * workspace.element_size(), _addr(dev_status),
        _stream(stream)))


def lq_verify_draft(draft_tokens, draft_lens, target_probs, draft_probs, u_accept, u_sample, out_tokens, accepted,
                    dev_status=None, stream=None) -> None:
    """Accept or refuse draft_tokens [batch x n] and draw the token after the accepted ones (see lq.h)."""
    import torch
    b, n = draft_tokens.shape
    vocab = target_probs.shape[2]
    for name, t, rows in (("target_probs", target_probs, n + 1), ("draft_probs", draft_probs, n)):
        if t is not None and (tuple(t.shape) != (b, rows, vocab) or t.dtype != target_probs.dtype or
                              (vocab > 1 and rows > 0 and t.stride(2) != 1)):
            raise ValueError(f"{name}: want [{b} x {rows} x {vocab}] {target_probs.dtype} with packed rows, got "
                             f"{tuple(t.shape)} {t.dtype} with strides {tuple(t.stride())}")
    _want("draft_tokens", draft_tokens, (b, n), torch.int32)
    if draft_lens is not None:
        _want("draft_lens", draft_lens, (b,), torch.int32)
    _want("u_accept", u_accept, (b, n), torch.float32)
    _want("u_sample", u_sample, (b,), torch.float32)
    _want("out_tokens", out_tokens, (b, n + 1), torch.int32)
    _want("accepted", accepted, (b,), torch.int32)
    q = draft_probs
    _check("lq_verify_draft", _get_lib().lq_verify_draft(
        _addr(draft_tokens), _addr(draft_lens), b, n, vocab, _addr(target_probs), target_probs.stride(0),
        target_probs.stride(1), _addr(q), 0 if q is None else q.stride(0), 0 if q is None else q.stride(1),
        _dtype_id(target_probs), _addr(u_accept), _addr(u_sample), _addr(out_tokens), _addr(accepted),
        _addr(dev_status), _stream(stream)))


# ------------------------------------------------------------------ allocating helpers
def quantize(W, lattice: str = "e8", tile: int = 256, seed: int = 0, beta: float = 0.25,
             dev_status=None, stream=None):
    """Allocate outputs with torch on W's device and call :func:`lq_quantize`.

    Returns (codes int8 [rows x cols], scales float32 [rows x cols/tile], signs int8 [cols]).
    """
    import torch
    rows, cols = W.shape
    codes = torch.empty((rows, cols), dtype=torch.int8, device=W.device)
    scales = torch.empty((rows, cols // tile), dtype=torch.float32, device=W.device)
    signs = torch.empty((cols,), dtype=torch.int8, device=W.device)
    lq_quantize(lattice, W, tile, seed, beta, codes, scales, signs, dev_status, stream)
    return codes, scales, signs


def dequantize(codes, scales, signs, lattice: str = "e8", tile: int = 256, dtype=None, stream=None):
    import torch
    dtype = torch.float32 if dtype is None else dtype
    out = torch.empty(codes.shape, dtype=dtype, device=codes.device)
    lq_dequantize(lattice, codes, scales, signs, tile, out, stream)
    return out


def gemv(codes, scales, signs, x, lattice: str = "e8", tile: int = 256, workspace=None,
         dev_status=None, stream=None):
    import torch
    rows, cols = codes.shape
    y = torch.empty((x.shape[0], rows), dtype=torch.float32, device=codes.device)
    if workspace is None:
        workspace = torch.empty(lq_gemv_workspace_size(x.shape[0], cols, tile), dtype=torch.uint8,
                                device=codes.device)
    lq_gemv(lattice, codes, scales, signs, tile, x, y, workspace, dev_status, stream)
    return y


def gemm(codes, scales, signs, X, lattice: str = "e8", tile: int = 256, workspace=None,
         dev_status=None, stream=None, out_dtype=None):
    import torch
    N, K = codes.shape
    M = X.shape[0]
    Y = torch.empty((M, N), dtype=out_dtype or torch.float32, device=codes.device)
    if workspace is None:
        workspace = torch.empty(lq_gemm_workspace_size(M, N, K, _dtype_id(Y)), dtype=torch.uint8,
                                device=codes.device)
    lq_gemm(lattice, codes, scales, signs, tile, X, Y, workspace, dev_status, stream)
    return Y


# ------------------------------------------------------------------ checkpoint
CHECKPOINT_FORMAT = "lq-codes-v1"


def save_quantized(path, codes, scales, signs, lattice: str, tile: int, seed: int, beta: float,
                   scale_format="tile_f32", dither_seed=None) -> None:
    """Write codes, scales and signs with the header needed to use them again
    (lattice, tile, seed, beta, shape, scale format, and the dither seed of a
    dithered quantization or None) in one torch.save file."""
    import torch
    fmt = {v: k for k, v in _SCALE_FORMATS.items()}.get(_scale_format_id(scale_format))
    if fmt is None:
        raise ValueError(f"unknown scale format {scale_format!r}")
    torch.save({"format": CHECKPOINT_FORMAT, "lattice": str(lattice), "tile": int(tile), "seed": int(seed),
                "beta": float(beta), "shape": list(codes.shape), "scale_format": fmt,
                "dither_seed": None if dither_seed is None else int(dither_seed), "codes": codes.detach().cpu(),
                "scales": scales.detach().cpu(), "signs": signs.detach().cpu()}, path)


def load_quantized(path, device=None) -> dict:
    """Read a file written by :func:`save_quantized`; tensors moved to `device` when given.
    Files written before the scale formats existed read as float32 tile scales."""
    import torch
    d = torch.load(path, map_location="cpu", weights_only=True)
    if d.get("format") != CHECKPOINT_FORMAT:
        raise ValueError(f"{path}: not a {CHECKPOINT_FORMAT} file")
    d.setdefault("scale_format", "tile_f32")
    d.setdefault("dither_seed", None)
    rows, cols = d["shape"]
    want_scales = (rows,) if d["scale_format"] == "row_bf16" else (rows, cols // d["tile"])
    if tuple(d["codes"].shape) != (rows, cols) or tuple(d["scales"].shape) != want_scales \
            or tuple(d["signs"].shape) != (cols,):
        raise ValueError(f"{path}: tensor shapes do not match the header")
    if device is not None:
        for k in ("codes", "scales", "signs"):
            d[k] = d[k].to(device)
    return d

