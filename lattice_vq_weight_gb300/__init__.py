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


# These calls run once or more per layer and step, some of them shorter on the
# GPU than their marshalling, so the checks below are written to cost little:
# a failed one is explained by a second look.
def _addr(t):
    """Device address of a tensor (or None) as a plain number."""
    return None if t is None else t.data_ptr()


_raw_stream = None


def _stream_of(device: int, stream):
    """The stream of a call on tensors of a device: the one given, else the device's current one."""
    global _raw_stream
    if stream is not None:
        return int(stream)
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


def _is(t, dtype, shape) -> bool:
    return t.dtype is dtype and t.shape == shape and t.is_contiguous()


def _explain(call: str, wanted) -> None:
    """Raise for the first of (name, tensor, dtype, shape) that is not a contiguous tensor of that kind."""
    for name, t, dtype, shape in wanted:
        if t is not None and not _is(t, dtype, shape):
            raise ValueError(f"{call}: {name}: want a contiguous {tuple(shape)} tensor of {dtype}, got "
                             f"{tuple(t.shape)} {t.dtype} with strides {tuple(t.stride())}")


def _one_device(call: str, *tensors) -> int:
    """The CUDA device that all tensors (None aside) are on; tensors in host memory or on several are refused."""
    d = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != d or d < 0):
            raise ValueError(f"{call}: want tensors on one CUDA device, got "
                             f"{sorted({str(x.device) for x in tensors if x is not None})}")
    return d


def _heads(name: str, t) -> int:
    """Token stride of a [tokens x heads x head_dim] tensor whose heads are packed."""
    if t.dim() == 3:
        tokens, heads, d = t.shape
        s0, s1, s2 = t.stride()
        if s2 == 1 and (s1 == d or heads == 1):
            return s0 if tokens > 1 else heads * d
    raise ValueError(f"{name}: want [tokens x heads x head_dim] with packed heads, got {tuple(t.shape)} with "
                     f"strides {tuple(t.stride())}")


def _cache(call, k_cache, k_scales, v_cache, v_scales):
    """(num_blocks, kv_heads, block_size, head_dim) of a cache's four tensors, checked."""
    import torch
    i8, f32, shape = torch.int8, torch.float32, k_cache.shape
    if len(shape) != 4:
        raise ValueError(f"{call}: k_cache: want [num_blocks x kv_heads x block_size x head_dim], got {tuple(shape)}")
    if not (_is(k_cache, i8, shape) and _is(v_cache, i8, shape) and _is(k_scales, f32, shape[:2])
            and _is(v_scales, f32, shape[:2])):
        _explain(call, (("k_cache", k_cache, i8, shape), ("v_cache", v_cache, i8, shape),
                        ("k_scales", k_scales, f32, shape[:2]), ("v_scales", v_scales, f32, shape[:2])))
    return shape


def _table(call, t, batch):
    """(row stride, width) of a block table int32 [batch x blocks] with packed rows."""
    import torch
    rows, width = t.shape if t.dim() == 2 else (-1, 0)
    if rows != batch or t.dtype is not torch.int32 or (width > 1 and t.stride(1) != 1):
        raise ValueError(f"{call}: block_table: want int32 [{batch} x blocks] with packed rows, got {tuple(t.shape)} "
                         f"{t.dtype} with strides {tuple(t.stride())}")
    return (t.stride(0) if rows > 1 else width), width


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
    i32 = torch.int32
    b, n, free = cached_lens.numel(), slots.numel(), free_blocks.numel()
    if not (_is(cached_lens, i32, (b,)) and _is(new_lens, i32, (b,)) and _is(free_blocks, i32, (free,))
            and _is(cu_new, i32, (b + 1,)) and _is(kv_lens, i32, (b,)) and _is(positions, i32, (n,))
            and _is(used, i32, (1,)) and _is(slots, torch.int64, (n,))):
        _explain("lq_kv_plan", (
            ("cached_lens", cached_lens, i32, (b,)), ("new_lens", new_lens, i32, (b,)),
            ("free_blocks", free_blocks, i32, (free,)), ("cu_new", cu_new, i32, (b + 1,)), ("kv_lens", kv_lens, i32, (b,)),
            ("positions", positions, i32, (n,)), ("used", used, i32, (1,)), ("slots", slots, torch.int64, (n,))))
    stride, width = _table("lq_kv_plan", block_table, b)
    dev = _one_device("lq_kv_plan", cached_lens, new_lens, free_blocks, block_table, cu_new, kv_lens, slots, positions,
                      used, dev_status)
    st = _get_lib().lq_kv_plan(
        cached_lens.data_ptr(), new_lens.data_ptr(), b, block_size, free_blocks.data_ptr(), free, block_table.data_ptr(),
        stride, width, cu_new.data_ptr(), kv_lens.data_ptr(), slots.data_ptr(), positions.data_ptr(), n, used.data_ptr(),
        _addr(dev_status), _stream_of(dev, stream))
    if st:
        _check("lq_kv_plan", st)


def lq_qk_norm_rope(q, k, q_weight, k_weight, eps: float, positions, cos_sin, q_out, k_out, interleaved: bool = False,
                    dev_status=None, stream=None) -> None:
    """RMS norm of every head of q and k (weights None: none), then the rotation; q_out, k_out may be q, k."""
    import torch
    f32, dt, shape, kshape = torch.float32, q.dtype, q.shape, k.shape
    if k.dtype is not dt or q_out.dtype is not dt or k_out.dtype is not dt:
        raise TypeError("lq_qk_norm_rope: q, k and their outputs have one dtype")
    ldq, ldk, ldqo, ldko = _heads("q", q), _heads("k", k), _heads("q_out", q_out), _heads("k_out", k_out)
    tokens, hq, d = shape
    if kshape[0] != tokens or kshape[2] != d or q_out.shape != shape or k_out.shape != kshape:
        raise ValueError("lq_qk_norm_rope: q, k and their outputs do not belong together")
    rows, rot = cos_sin.shape
    if not (_is(positions, torch.int32, (tokens,)) and _is(cos_sin, f32, (rows, rot))
            and (q_weight is None or _is(q_weight, f32, (d,))) and (k_weight is None or _is(k_weight, f32, (d,)))):
        _explain("lq_qk_norm_rope", (("positions", positions, torch.int32, (tokens,)),
                                     ("cos_sin", cos_sin, f32, (rows, rot)), ("q_weight", q_weight, f32, (d,)),
                                     ("k_weight", k_weight, f32, (d,))))
    dev = _one_device("lq_qk_norm_rope", q, k, q_weight, k_weight, positions, cos_sin, q_out, k_out, dev_status)
    st = _get_lib().lq_qk_norm_rope(
        q.data_ptr(), ldq, hq, k.data_ptr(), ldk, kshape[1], _dtype_id(q), tokens, d, _addr(q_weight), _addr(k_weight),
        eps, positions.data_ptr(), cos_sin.data_ptr(), rows, rot, 1 if interleaved else 0, q_out.data_ptr(), ldqo,
        k_out.data_ptr(), ldko, _addr(dev_status), _stream_of(dev, stream))
    if st:
        _check("lq_qk_norm_rope", st)


def lq_kv_append(k, v, slots, k_cache, k_scales, v_cache, v_scales, dev_status=None, stream=None) -> None:
    """Write k, v [tokens x kv_heads x head_dim] to the cache's slots (int64 [tokens], negative: left out)."""
    import torch
    nb, hk, bs, d = _cache("lq_kv_append", k_cache, k_scales, v_cache, v_scales)
    n = k.shape[0]
    if k.shape != v.shape or k.dtype is not v.dtype or k.shape != (n, hk, d):
        raise ValueError(f"lq_kv_append: k and v do not fit the cache: {tuple(k.shape)}, {tuple(v.shape)}")
    if not _is(slots, torch.int64, (n,)):
        _explain("lq_kv_append", (("slots", slots, torch.int64, (n,)),))
    dev = _one_device("lq_kv_append", k, v, slots, k_cache, k_scales, v_cache, v_scales, dev_status)
    st = _get_lib().lq_kv_append(
        k.data_ptr(), _heads("k", k), v.data_ptr(), _heads("v", v), _dtype_id(k), n, slots.data_ptr(),
        k_cache.data_ptr(), k_scales.data_ptr(), v_cache.data_ptr(), v_scales.data_ptr(), nb, bs, hk, d,
        _addr(dev_status), _stream_of(dev, stream))
    if st:
        _check("lq_kv_append", st)


def lq_kv_gather(slots, k_cache, k_scales, v_cache, v_scales, k_out, v_out, dev_status=None, stream=None) -> None:
    """The values that the cache's slots stand for, [n x kv_heads x head_dim] float32 or bf16."""
    import torch
    nb, hk, bs, d = _cache("lq_kv_gather", k_cache, k_scales, v_cache, v_scales)
    n, dt, shape = slots.numel(), k_out.dtype, (slots.numel(), hk, d)
    if not (_is(slots, torch.int64, (n,)) and _is(k_out, dt, shape) and _is(v_out, dt, shape)):
        _explain("lq_kv_gather", (("slots", slots, torch.int64, (n,)), ("k_out", k_out, dt, shape),
                                  ("v_out", v_out, dt, shape)))
    dev = _one_device("lq_kv_gather", slots, k_cache, k_scales, v_cache, v_scales, k_out, v_out, dev_status)
    st = _get_lib().lq_kv_gather(
        slots.data_ptr(), n, k_cache.data_ptr(), k_scales.data_ptr(), v_cache.data_ptr(), v_scales.data_ptr(), nb, bs, hk,
        d, k_out.data_ptr(), v_out.data_ptr(), _dtype_id(k_out), _addr(dev_status), _stream_of(dev, stream))
    if st:
        _check("lq_kv_gather", st)


def lq_attention_paged_workspace_size(batch: int, total_q: int, q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(_get_lib().lq_attention_paged_workspace_size(int(batch), int(total_q), int(q_heads), int(kv_heads),
                                                            int(head_dim)))


def lq_attention_paged(q, cu_q, kv_lens, block_table, k_cache, k_scales, v_cache, v_scales, out, workspace,
                       sm_scale=None, dev_status=None, stream=None) -> None:
    """out = attention of q [total_q x q_heads x head_dim] over the requests' cached tokens (see lq.h);
    sm_scale defaults to head_dim ** -0.5."""
    import torch
    nb, hk, bs, d = _cache("lq_attention_paged", k_cache, k_scales, v_cache, v_scales)
    b, i32 = kv_lens.numel(), torch.int32
    ldq, ldo = _heads("q", q), _heads("out", out)
    total, hq, dq = q.shape
    if out.shape != q.shape or q.dtype is not out.dtype or dq != d:
        raise ValueError(f"lq_attention_paged: q and out do not fit: {tuple(q.shape)}, {tuple(out.shape)}")
    if not (_is(kv_lens, i32, (b,)) and _is(cu_q, i32, (b + 1,))):
        _explain("lq_attention_paged", (("kv_lens", kv_lens, i32, (b,)), ("cu_q", cu_q, i32, (b + 1,))))
    stride, width = _table("lq_attention_paged", block_table, b)
    dev = _one_device("lq_attention_paged", q, cu_q, kv_lens, block_table, k_cache, k_scales, v_cache, v_scales, out,
                      workspace, dev_status)
    st = _get_lib().lq_attention_paged(
        q.data_ptr(), ldq, _dtype_id(q), total, cu_q.data_ptr(), kv_lens.data_ptr(), b, block_table.data_ptr(), stride,
        width, k_cache.data_ptr(), k_scales.data_ptr(), v_cache.data_ptr(), v_scales.data_ptr(), nb, bs, hq, hk, d,
        d ** -0.5 if sm_scale is None else sm_scale, out.data_ptr(), ldo, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _addr(dev_status), _stream_of(dev, stream))
    if st:
        _check("lq_attention_paged", st)


def lq_verify_draft(draft_tokens, draft_lens, target_probs, draft_probs, u_accept, u_sample, out_tokens, accepted,
                    dev_status=None, stream=None) -> None:
    """Accept or refuse draft_tokens [batch x n] and draw the token after the accepted ones (see lq.h)."""
    import torch
    i32, f32, dt = torch.int32, torch.float32, target_probs.dtype
    b, n = draft_tokens.shape
    vocab = target_probs.shape[2]

    def rows_of(name, t, rows):
        s0, s1, s2 = t.stride()
        if t.shape != (b, rows, vocab) or t.dtype is not dt or (s2 != 1 and vocab > 1 and rows > 0):
            raise ValueError(f"lq_verify_draft: {name}: want [{b} x {rows} x {vocab}] {dt} with packed rows, got "
                             f"{tuple(t.shape)} {t.dtype} with strides {(s0, s1, s2)}")
        return s0, s1

    t0, t1 = rows_of("target_probs", target_probs, n + 1)
    q0, q1 = (0, 0) if draft_probs is None else rows_of("draft_probs", draft_probs, n)
    if not (_is(draft_tokens, i32, (b, n)) and _is(u_accept, f32, (b, n)) and _is(u_sample, f32, (b,))
            and _is(out_tokens, i32, (b, n + 1)) and _is(accepted, i32, (b,))
            and (draft_lens is None or _is(draft_lens, i32, (b,)))):
        _explain("lq_verify_draft", (
            ("draft_tokens", draft_tokens, i32, (b, n)), ("u_accept", u_accept, f32, (b, n)),
            ("u_sample", u_sample, f32, (b,)), ("out_tokens", out_tokens, i32, (b, n + 1)),
            ("accepted", accepted, i32, (b,)), ("draft_lens", draft_lens, i32, (b,))))
    dev = _one_device("lq_verify_draft", draft_tokens, draft_lens, target_probs, draft_probs, u_accept, u_sample,
                      out_tokens, accepted, dev_status)
    st = _get_lib().lq_verify_draft(
        draft_tokens.data_ptr(), _addr(draft_lens), b, n, vocab, target_probs.data_ptr(), t0, t1, _addr(draft_probs), q0,
        q1, _dtype_id(target_probs), u_accept.data_ptr(), u_sample.data_ptr(), out_tokens.data_ptr(), accepted.data_ptr(),
        _addr(dev_status), _stream_of(dev, stream))
    if st:
        _check("lq_verify_draft", st)


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

