"""ctypes binding of libmxgg.so (include/mxgg.h).

Argument marshalling only: every step of the path runs in the library's HIP
kernels. torch supplies device memory and the current stream; output tensors
are allocated here when the caller passes none. Importing this module fails
loudly when the built library is missing -- there is no fallback.
"""
from __future__ import annotations

import array
import ctypes
import operator
import os
import re

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_PATH = os.path.join(PKG, "libmxgg.so")
HEADER = os.path.join(ROOT, "include", "mxgg.h")

# mxgg_format
MXFP4, MXFP8, FP8_1x128, FP8_128x128, FP8_1x128_P2, FP8_128x128_P2, INT8 = 0, 1, 2, 3, 4, 5, 6
FORMATS = {"mxfp4": MXFP4, "mxfp8": MXFP8, "fp8_1x128": FP8_1x128, "fp8_128x128": FP8_128x128,
           "fp8_1x128_p2": FP8_1x128_P2, "fp8_128x128_p2": FP8_128x128_P2, "int8": INT8}
POW2_SCALES = 1
MAX_EXPERTS = 512
# mxgg_dtype, mxgg_norm and the limits and flags of mxgg_moe_layer
BF16, F32 = 0, 1
I32, I64 = 0, 1   # mxgg_itype
NORM_L2, NORM_MAX = 0, 1
MOE_MAX_TOKENS, MOE_MAX_TOP_K, MOE_RENORMALIZE, MOE_W13_KBLOCK, MOE_W2_KBLOCK = 64, 16, 1, 4, 8
# mxgg_scale_layout: OR-ed into an MX format to state the layout of its scales
LAYOUT_BLOCK_MAJOR, LAYOUT_ROW_MAJOR, LAYOUT_MFMA, LAYOUT_MASK = 0x000, 0x100, 0x200, 0xF00
# MX code layouts: row-wise / column-wise codes in 64-byte K blocks
KBLOCK_ROWS, KBLOCK_COLS, KBLOCK_MASK = 0x1000, 0x2000, 0x3000

STATUS = {
    0: "MXGG_OK", 1: "MXGG_ERR_NULL", 2: "MXGG_ERR_SHAPE", 3: "MXGG_ERR_SPLITS",
    4: "MXGG_ERR_FORMAT", 5: "MXGG_ERR_ALIGN", 6: "MXGG_ERR_WORKSPACE",
    7: "MXGG_ERR_DEVICE", 8: "MXGG_ERR_ARCH", 9: "MXGG_ERR_HIP",
}


class MxggError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{self.name}: {message}")


_vp, _i64, _i32, _u32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
_i64p = ctypes.POINTER(ctypes.c_int64)
_f32, _i32p, _vpp = ctypes.c_float, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_void_p)

_SIGS = {
    "mxgg_quantize_rowwise": [_vp, _i64, _i64, _i64, _i32, _u32, _vp, _vp, _vp],
    "mxgg_quantize_colwise_segpad": [_vp, _i64, _i64, _i64, _i64p, _i32, _i32, _u32, _vp, _vp, _i64, _vp],
    "mxgg_quantize_dual": [_vp, _i64, _i64, _i64, _i64p, _i32, _i32, _u32, _vp, _vp, _vp, _vp, _i64, _vp],
    "mxgg_grouped_fwd": [_vp, _vp, _i32, _vp, _vp, _i32, _i64p, _i32, _i64, _i64, _i64, _vp, _vp, _sz, _vp],
    "mxgg_grouped_dgrad": [_vp, _vp, _vp, _vp, _i32, _i64p, _i32, _i64, _i64, _i64, _vp, _vp, _sz, _vp],
    "mxgg_transpose_128x128": [_vp, _vp, _i32, _i64, _i64, _vp, _vp, _vp],
    "mxgg_grouped_wgrad": [_vp, _vp, _vp, _vp, _i32, _i64p, _i32, _i64, _i64, _i64, _vp, _i32, _i32, _vp, _sz,
                           _vp],
    "mxgg_mx_scales_relayout": [_vp, _i32, _i64, _i64, _vp, _i32, _vp],
    "mxgg_layer_norm_fwd": [_vp, _i64, _i64, _i64, _i32, _vp, _vp, _i32, _f32, _vp, _i64, _vp, _vp, _vp],
    "mxgg_layer_norm_bwd": [_vp, _i64, _vp, _i64, _i64, _i64, _i32, _vp, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _i32,
                            _vp, _sz, _vp],
    "mxgg_grad_norm": [_vpp, _i64p, _i32p, _i64, _i32, _vp, _vp, _sz, _vp],
    "mxgg_clip_grad_norm": [_vpp, _i64p, _i32p, _i64, _i32, _f32, _vp, _vp, _sz, _vp],
    "mxgg_clip_grads_with_norm": [_vpp, _i64p, _i32p, _i64, _f32, _vp, _vp],
    "mxgg_moe_layer": [_vp, _i64, _vp, _i64, _i32, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i32, _u32, _vp,
                       _vp, _vp, _vp, _sz, _vp],
    "mxgg_moe_sort": [_vp, _i32, _i64, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp],
    "mxgg_moe_dispatch": [_vp, _i64, _i32, _i64, _i64, _vp, _i64, _vp, _i64, _i64, _vp],
    "mxgg_moe_combine": [_vp, _i64, _i32, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp],
    "mxgg_moe_combine_bwd": [_vp, _i64, _vp, _i64, _i32, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _vp, _vp],
    "mxgg_dropout": [_vp, _i64, _i32, _i64, _i64, _f32, _vp, _u32, _vp, _i64, _vp, _i64, _vp],
}
# functions that return a size
_SIZES = {
    "mxgg_layer_norm_bwd_workspace": [_i64, _i64],
    "mxgg_grad_norm_workspace": [_i64],
    "mxgg_moe_layer_workspace": [_i64, _i64, _i64, _i64],
    "mxgg_moe_sort_workspace": [_i64, _i64, _i64],
}


def _load():
    # torch's HIP runtime must be the one in the process before the library
    # binds to libamdhip64.so (it links that same runtime)
    import torch  # noqa: F401
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python moe_grouped_block_mx_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    for name, args in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name, args in _SIZES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = _sz
    lib.mxgg_workspace_size.argtypes = [_i32]
    lib.mxgg_workspace_size.restype = _sz
    lib.mxgg_segpad_rows.argtypes = [_i64p, _i32, _i32]
    lib.mxgg_segpad_rows.restype = _i64
    lib.mxgg_mx_scale_stride.argtypes = [_i64]
    lib.mxgg_mx_scale_stride.restype = _i64
    lib.mxgg_status_string.argtypes = [_i32]
    lib.mxgg_status_string.restype = ctypes.c_char_p
    lib.mxgg_last_error.argtypes = []
    lib.mxgg_last_error.restype = ctypes.c_char_p
    return lib


lib = _load()


def header_functions() -> list[str]:
    """Names of the functions include/mxgg.h declares."""
    txt = open(HEADER).read()
    return sorted(set(re.findall(r"\b(mxgg_[a-z_0-9]+)\s*\(", txt)))


def _check(status: int):
    if status != 0:
        raise MxggError(status, lib.mxgg_last_error().decode())


def _splits(m_splits):
    vals = [int(v) for v in m_splits]
    arr = (ctypes.c_int64 * max(1, len(vals)))(*vals)
    return arr, len(vals)


def _fmt(f) -> int:
    return FORMATS[f] if isinstance(f, str) else int(f)


def _torch():
    import torch
    return torch


def _stream(t):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_bf16_2d(x):
    torch = _torch()
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16 tensor")
    if x.numel() and x.stride(1) != 1:
        raise ValueError("x must have unit inner stride")


def _ld(x):
    """Leading dimension in elements (the column count for an empty tensor)."""
    return x.stride(0) if x.numel() else x.shape[1]


def _expect(t, name, shape, dtypes):
    """The C ABI sees only pointers, so this is the one place where a buffer
    of the wrong shape, dtype or layout is caught before the GPU reads or
    writes past its end."""
    if t is not None and t.dtype is dtypes and t.shape == shape and t.is_contiguous():
        return t
    shape = tuple(int(v) for v in shape)
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != shape or t.dtype not in dtypes or not t.is_contiguous():
        want = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        got = f"{str(t.dtype).replace('torch.', '')} {tuple(t.shape)}" + ("" if t.is_contiguous() else " non-contiguous")
        raise ValueError(f"{name} must be a contiguous {want} tensor of shape {shape}, got {got}")
    return t


def _is_mx(f):
    return (f & 0xFF) in (MXFP4, MXFP8)


def _row_major(f):
    return (f & LAYOUT_MASK) == LAYOUT_ROW_MAJOR


def _mfma(f):
    return (f & LAYOUT_MASK) == LAYOUT_MFMA


def _rows32(rows):
    return (rows + 31) // 32 * 32 if rows > 0 else 0


def _layout_shape(layout, rows, blocks):
    """u8 scales of an operand with `rows` rows and `blocks` blocks of 32 along
    its contraction, in one of the three MX scale layouts."""
    if layout == LAYOUT_ROW_MAJOR:
        return (rows, blocks)
    if layout == LAYOUT_MFMA:                                     # [blocks/4, R32/32, 64, 2]
        return (blocks // 4, _rows32(rows) * 4)
    return (blocks, mxgg_mx_scale_stride(rows))                   # block-major


def _code_bytes(f, n):
    """Code bytes of n elements (E2M1 packs two per byte)."""
    return n // 2 if (f & 0xFF) == MXFP4 else n


def _q_shape(f, rows, cols):
    """Codes of a [rows, cols] operand quantized along cols: rows of codes,
    or 64-byte blocks along cols, u8 [bytes per row / 64, rows, 64]
    (blockwise formats always, MX with KBLOCK_ROWS; int8 never)."""
    if (f & 0xFF) == INT8:
        return (rows, cols)
    if not _is_mx(f) or (f & KBLOCK_ROWS):
        return (_code_bytes(f, cols) // 64, rows, 64)
    return (rows, _code_bytes(f, cols))


def _q_rows(q, f):
    """Row count of a code tensor laid out as _q_shape gives it (a tensor of
    another rank then fails the shape check that follows)."""
    if (_is_mx(f) and not (f & KBLOCK_ROWS)) or (f & 0xFF) == INT8:
        return q.shape[0] if q.dim() >= 1 else 0
    return q.shape[1] if q.dim() >= 2 else 0


def _col_q_shape(f, cols, mpad):
    """Codes of the column-wise segment-padded [cols, mpad] operand: rows, or
    64-byte blocks along the padded length (blockwise, MX with KBLOCK_COLS)."""
    if not _is_mx(f) or (f & KBLOCK_COLS):
        return (_code_bytes(f, mpad) // 64, cols, 64)
    return (cols, _code_bytes(f, mpad))


def _row_scale_shape(f, rows, cols):
    """Scales of a [rows, cols] operand quantized along cols (row-major scales
    when the format says so: the library refuses them, never misreads them).
    1x128 fp32 scales are block-major [cols/128, rows], int8 ones [rows]."""
    if (f & 0xFF) == INT8:
        return (rows,)
    if _is_mx(f):
        return _layout_shape(f & LAYOUT_MASK, rows, cols // 32)
    if (f & 0xFF) in (FP8_1x128, FP8_1x128_P2):
        return (cols // 128, rows)
    return (rows // 128, cols // 128)


def _col_scale_shape(f, cols, mpad):
    """Scales of the column-wise segment-padded [cols, mpad] operand (1x128:
    block-major f32 [mpad/128, cols])."""
    if _is_mx(f):
        return _layout_shape(f & LAYOUT_MASK, cols, mpad // 32)
    return (mpad // 128, cols)


def _sdtype(f):
    torch = _torch()
    return torch.uint8 if _is_mx(f) else torch.float32


def _qdtype(f):
    torch = _torch()
    return torch.int8 if (f & 0xFF) == INT8 else torch.uint8


def mxgg_workspace_size(G: int) -> int:
    return int(lib.mxgg_workspace_size(G))


def mxgg_segpad_rows(m_splits, fmt) -> int:
    arr, G = _splits(m_splits)
    r = int(lib.mxgg_segpad_rows(arr, G, _fmt(fmt) & 0xFF))
    if r < 0:
        raise MxggError(2, "invalid splits or format for mxgg_segpad_rows")
    return r


def _flags(flags, f):
    """Power-of-two scales are the blockwise default; MX formats take no flags."""
    if flags is None:
        return POW2_SCALES if (f & 0xFF) in (FP8_1x128, FP8_128x128, FP8_1x128_P2, FP8_128x128_P2) else 0
    return int(flags)


def mxgg_mx_scales_relayout(src, rows, blocks, src_layout, dst_layout, dst=None):
    """MX scales from one layout into another: row-major u8 [rows, blocks],
    block-major u8 [blocks, mx_scale_stride(rows)], MFMA u8 [blocks/4,
    R32*4] (R32 = rows rounded up to 32; padding rows 0). Returns dst."""
    torch = _torch()
    src_shape = _layout_shape(src_layout, rows, blocks)
    dst_shape = _layout_shape(dst_layout, rows, blocks)
    _expect(src, "src", src_shape, torch.uint8)
    if dst is None:
        dst = torch.empty(dst_shape, dtype=torch.uint8, device=src.device)
    _expect(dst, "dst", dst_shape, torch.uint8)
    _check(lib.mxgg_mx_scales_relayout(_ptr(src), int(src_layout), int(rows), int(blocks), _ptr(dst),
                                       int(dst_layout), _stream(src)))
    return dst


def mxgg_mx_scale_stride(rows):
    """Block stride (bytes) of block-major MX scales of an operand with `rows` rows."""
    return int(lib.mxgg_mx_scale_stride(int(rows)))


def mxgg_quantize_rowwise(x, fmt="mxfp4", flags=None, q=None, scales=None):
    """x: bf16 [rows, cols] (row stride may exceed cols). Returns (q, scales).
    flags: None = default (MXGG_POW2_SCALES for the blockwise formats).
    "int8": codes int8 [rows, cols], one scale a row (a token, or a weight's
    channel)."""
    torch = _torch()
    f = _fmt(fmt)
    if f == INT8:
        return _quantize_int8(x, flags, q, scales)
    flags = _flags(flags, f)
    rows, cols = x.shape
    _check_bf16_2d(x)
    if q is None:
        q = torch.empty(_q_shape(f, rows, cols), dtype=_qdtype(f), device=x.device)
    if scales is None:
        # MX: block-major, block stride = rows rounded up to a multiple of 4
        scales = torch.empty(_row_scale_shape(f, rows, cols), dtype=_sdtype(f), device=x.device)
    _expect(q, "q", _q_shape(f, rows, cols), _qdtype(f))
    _expect(scales, "scales", _row_scale_shape(f, rows, cols), _sdtype(f))
    _check(lib.mxgg_quantize_rowwise(_ptr(x), rows, cols, _ld(x), f, flags, _ptr(q), _ptr(scales),
                                     _stream(x)))
    return q, scales


def mxgg_quantize_colwise_segpad(x, m_splits, fmt="mxfp4", flags=None, q=None, scales=None):
    """x: bf16 [rows, cols]. Returns (q, scales, mpad): q [cols, mpad(/2)],
    or for the 1x128 formats u8 [mpad/64, cols, 64] (64-byte K blocks)."""
    torch = _torch()
    f = _fmt(fmt)
    flags = _flags(flags, f)
    rows, cols = x.shape
    _check_bf16_2d(x)
    arr, G = _splits(m_splits)
    mpad = int(lib.mxgg_segpad_rows(arr, G, f & 0xFF))
    if mpad < 0:
        mpad = 0
    if q is None:
        q = torch.empty(_col_q_shape(f, cols, mpad), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(_col_scale_shape(f, cols, mpad), dtype=_sdtype(f), device=x.device)
    _expect(q, "q", _col_q_shape(f, cols, mpad), torch.uint8)
    _expect(scales, "scales", _col_scale_shape(f, cols, mpad), _sdtype(f))
    _check(lib.mxgg_quantize_colwise_segpad(_ptr(x), rows, cols, _ld(x), arr, G, f, flags, _ptr(q),
                                            _ptr(scales), mpad, _stream(x)))
    return q, scales, mpad


def mxgg_quantize_dual(x, m_splits, fmt="mxfp4", flags=None, q_row=None, s_row=None, q_col=None, s_col=None):
    """x: bf16 [rows, cols]. Row-wise and column-wise segment-padded
    quantization (MX, or blockwise 1x128) from one read.
    Returns (q_row, s_row, q_col, s_col, mpad)."""
    torch = _torch()
    f = _fmt(fmt)
    flags = _flags(flags, f)
    rows, cols = x.shape
    _check_bf16_2d(x)
    arr, G = _splits(m_splits)
    mpad = int(lib.mxgg_segpad_rows(arr, G, f & 0xFF))
    if mpad < 0:
        mpad = 0
    u8 = dict(dtype=torch.uint8, device=x.device)
    if q_row is None:
        q_row = torch.empty(_q_shape(f, rows, cols), **u8)
    if s_row is None:
        s_row = torch.empty(_row_scale_shape(f, rows, cols), dtype=_sdtype(f), device=x.device)
    if q_col is None:
        q_col = torch.empty(_col_q_shape(f, cols, mpad), **u8)
    if s_col is None:
        s_col = torch.empty(_col_scale_shape(f, cols, mpad), dtype=_sdtype(f), device=x.device)
    _expect(q_row, "q_row", _q_shape(f, rows, cols), torch.uint8)
    _expect(s_row, "s_row", _row_scale_shape(f, rows, cols), _sdtype(f))
    _expect(q_col, "q_col", _col_q_shape(f, cols, mpad), torch.uint8)
    _expect(s_col, "s_col", _col_scale_shape(f, cols, mpad), _sdtype(f))
    _check(lib.mxgg_quantize_dual(_ptr(x), rows, cols, _ld(x), arr, G, f, flags, _ptr(q_row), _ptr(s_row),
                                  _ptr(q_col), _ptr(s_col), mpad, _stream(x)))
    return q_row, s_row, q_col, s_col, mpad


def mxgg_grouped_fwd(a_q, a_s, w_q, w_s, m_splits, N, K, a_fmt="mxfp4", w_fmt="mxfp4", out=None, ws=None):
    """out[M, N] (bf16) = per-expert A . W_g^T; W packed [G*N, ...]."""
    torch = _torch()
    af, wf = _fmt(a_fmt), _fmt(w_fmt)
    if af == wf == INT8:
        return _grouped_fwd_int8(a_q, a_s, w_q, w_s, m_splits, N, K, out, ws)
    arr, G = _splits(m_splits)
    M = _q_rows(a_q, af)
    _expect(a_q, "a_q", _q_shape(af, M, K), _qdtype(af))
    _expect(a_s, "a_s", _row_scale_shape(af, M, K), _sdtype(af))
    _expect(w_q, "w_q", _q_shape(wf, G * N, K), _qdtype(wf))
    _expect(w_s, "w_s", _row_scale_shape(wf, G * N, K), _sdtype(wf))
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a_q.device)
    _expect(out, "out", (M, N), torch.bfloat16)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.mxgg_grouped_fwd(_ptr(a_q), _ptr(a_s), _fmt(a_fmt), _ptr(w_q), _ptr(w_s), _fmt(w_fmt), arr, G, M, N,
                                K, _ptr(out), _ptr(ws), ws_bytes, _stream(a_q)))
    return out


def mxgg_transpose_128x128(w_q, w_s, G, N, K, wt_q=None, wt_s=None):
    """128x128-block FP8 weights [G*N, K] (+ f32 [G*N/128, K/128]) transposed
    to [G*K, N] (+ f32 [G*K/128, N/128]): the input gradient's weights (codes
    in 64-byte K blocks on both sides)."""
    torch = _torch()
    if wt_q is None:
        wt_q = torch.empty(_q_shape(FP8_128x128, G * K, N), dtype=torch.uint8, device=w_q.device)
    if wt_s is None:
        wt_s = torch.empty((G * K // 128, N // 128), dtype=torch.float32, device=w_q.device)
    _expect(w_q, "w_q", _q_shape(FP8_128x128, G * N, K), torch.uint8)
    _expect(w_s, "w_s", (G * N // 128, K // 128), torch.float32)
    _expect(wt_q, "wt_q", _q_shape(FP8_128x128, G * K, N), torch.uint8)
    _expect(wt_s, "wt_s", (G * K // 128, N // 128), torch.float32)
    _check(lib.mxgg_transpose_128x128(_ptr(w_q), _ptr(w_s), G, N, K, _ptr(wt_q), _ptr(wt_s), _stream(w_q)))
    return wt_q, wt_s


def mxgg_grouped_dgrad(dy_q, dy_s, wcol_q, wcol_s, m_splits, N, K, fmt="mxfp4", dx=None, ws=None):
    """dx[M, K] (bf16) = per-expert dY . W_g. fmt is dY's format: "mxfp4" /
    "mxfp8" with W quantized along N in MXFP4, or "fp8_1x128" / "fp8_1x128_p2"
    with W^T from mxgg_transpose_128x128."""
    torch = _torch()
    arr, G = _splits(m_splits)
    f = _fmt(fmt)
    M = _q_rows(dy_q, f)
    # layout bits of fmt describe wcol_s; dY's scales are block-major
    _expect(dy_q, "dy_q", _q_shape(f, M, N), torch.uint8)
    _expect(dy_s, "dy_s", _row_scale_shape(f & 0xFF, M, N), _sdtype(f))
    if _is_mx(f):                       # W along N, MXFP4: [K, G*N/2] + [G*N/32, K]
        _expect(wcol_q, "wcol_q", _col_q_shape(MXFP4 | (f & KBLOCK_COLS), K, G * N), torch.uint8)
        _expect(wcol_s, "wcol_s", _col_scale_shape(MXFP4 | (f & LAYOUT_MASK), K, G * N), torch.uint8)
    else:                               # transposed 128x128 blocks
        _expect(wcol_q, "wcol_q", _q_shape(FP8_128x128, G * K, N), torch.uint8)
        _expect(wcol_s, "wcol_s", (G * K // 128, N // 128), torch.float32)
    if dx is None:
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dy_q.device)
    _expect(dx, "dx", (M, K), torch.bfloat16)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.mxgg_grouped_dgrad(_ptr(dy_q), _ptr(dy_s), _ptr(wcol_q), _ptr(wcol_s), _fmt(fmt), arr, G, M, N, K,
                                  _ptr(dx), _ptr(ws), ws_bytes, _stream(dy_q)))
    return dx


def mxgg_grouped_wgrad(dycol_q, dycol_s, xcol_q, xcol_s, m_splits, N, K, mpad, main_grad, accumulate=True,
                       fmt="mxfp4", ws=None):
    """main_grad [G, N, K] (fp32 or bf16) += / = per-expert dY_g^T . X_g."""
    torch = _torch()
    arr, G = _splits(m_splits)
    f = _fmt(fmt)
    _expect(dycol_q, "dycol_q", _col_q_shape(f, N, mpad), torch.uint8)
    _expect(dycol_s, "dycol_s", _col_scale_shape(f, N, mpad), _sdtype(f))
    _expect(xcol_q, "xcol_q", _col_q_shape(f, K, mpad), torch.uint8)
    _expect(xcol_s, "xcol_s", _col_scale_shape(f, K, mpad), _sdtype(f))
    _expect(main_grad, "main_grad", (G, N, K), (torch.float32, torch.bfloat16))
    out_bf16 = 1 if main_grad.dtype == torch.bfloat16 else 0
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.mxgg_grouped_wgrad(_ptr(dycol_q), _ptr(dycol_s), _ptr(xcol_q), _ptr(xcol_s), _fmt(fmt), arr, G, N, K,
                                  mpad, _ptr(main_grad), out_bf16, 1 if accumulate else 0, _ptr(ws), ws_bytes,
                                  _stream(main_grad)))
    return main_grad


# The operators below are called for single tokens too, where a launch takes a
# few microseconds: their bindings pass addresses as plain ints and look a
# caller's buffer over only where one was given.
_f32_t, _u8_t, _i32_t = _torch().float32, _torch().uint8, _torch().int32
_bf16_t, _i8_t, _i64_t = _torch().bfloat16, _torch().int8, _torch().int64
_KINDS = {_bf16_t: BF16, _f32_t: F32}
_INTS = {_i32_t: I32, _i64_t: I64}
_raw_stream = _torch()._C._cuda_getCurrentRawStream


def _dtype(t, name):
    kind = _KINDS.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name} must be bf16 or fp32, got {str(t.dtype).replace('torch.', '')}")
    return kind


def _at(t):
    return None if t is None else t.data_ptr()


def _stream_of(t):
    index = t.get_device()
    if index < 0:
        raise ValueError(f"expected a GPU tensor, got one on {t.device}")
    return _raw_stream(index)


def _rows2d(t, name):
    """Leading dimension of a 2-D tensor with unit inner stride."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(t.shape)}")
    rows, cols = t.shape
    if rows == 0 or cols == 0:
        return cols
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit inner stride")
    return t.stride(0) if rows > 1 else cols


def _rows_like(t, x, name):
    """The same, of a tensor with x's shape, dtype and device."""
    if t.shape != x.shape or t.dtype is not x.dtype or t.get_device() != x.get_device():
        raise ValueError(f"{name} must be a {str(x.dtype).replace('torch.', '')} tensor of shape {tuple(x.shape)} on "
                         f"{x.device}, got {str(t.dtype).replace('torch.', '')} {tuple(t.shape)} on {t.device}")
    return _rows2d(t, name)


def _on(t, x, name):
    if t.get_device() != x.get_device():
        raise ValueError(f"{name} is on {t.device}, not on {x.device}")
    return t


def _cols_vector(t, name, x):
    """dtype of a contiguous [cols] vector beside x, None for None."""
    if t is None:
        return None
    if t.shape != x.shape[1:] or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape ({x.shape[1]},), got {tuple(t.shape)}")
    return _dtype(_on(t, x, name), name)


def _f32_out(t, name, n, x):
    """fp32 [n] beside x: the caller's, or a new one."""
    if t is None:
        return x.new_empty(n, dtype=_f32_t)
    return _on(_expect(t, name, (n,), _f32_t), x, name)


def _ws(ws, need, like):
    """The caller's workspace, or one from torch's allocator on the current
    stream (which keeps it from other streams until this one's work is done)."""
    if ws is None:
        return like.new_empty(need, dtype=_u8_t), need
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return _on(ws, like, "ws"), ws.numel() * ws.element_size()


def mxgg_layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, y=None, mean=None, rstd=None):
    """x: bf16 or fp32 [rows, cols] (any row stride); weight, bias: [cols], bf16
    or fp32 alike, None for 1 and 0. Returns (y, mean, rstd): y like x, mean and
    rstd fp32 [rows]."""
    dt, ldx = _dtype(x, "x"), _rows2d(x, "x")
    rows, cols = x.shape
    wd, bd = _cols_vector(weight, "weight", x), _cols_vector(bias, "bias", x)
    if wd is not None and bd is not None and wd != bd:
        raise ValueError("weight and bias must have the same dtype")
    if y is None:
        y, ldy = x.new_empty((rows, cols)), cols
    else:
        ldy = _rows_like(y, x, "y")
    mean, rstd = _f32_out(mean, "mean", rows, x), _f32_out(rstd, "rstd", rows, x)
    _check(lib.mxgg_layer_norm_fwd(x.data_ptr(), rows, cols, ldx, dt, _at(weight), _at(bias), wd or bd or 0, eps,
                                   y.data_ptr(), ldy, mean.data_ptr(), rstd.data_ptr(), _stream_of(x)))
    return y, mean, rstd


def mxgg_layer_norm_bwd(dy, x, weight, mean, rstd, dx=None, dweight=None, dbias=None, accumulate=False, ws=None):
    """dy, x: [rows, cols] alike (any row strides); mean, rstd from the forward.
    Returns (dx, dweight, dbias): dx like x; dweight and dbias fp32 [cols],
    added to the given ones with accumulate=True. False for dweight or dbias:
    not computed (None comes back)."""
    dt, ldx = _dtype(x, "x"), _rows2d(x, "x")
    rows, cols = x.shape
    lddy = _rows_like(dy, x, "dy")
    wd = _cols_vector(weight, "weight", x)
    if dx is None:
        dx, lddx = x.new_empty((rows, cols)), cols
    else:
        lddx = _rows_like(dx, x, "dx")
    if accumulate and (dweight is None or dbias is None):
        raise ValueError("accumulate=True needs dweight and dbias (or False for one that is not wanted)")
    dweight = None if dweight is False else _f32_out(dweight, "dweight", cols, x)
    dbias = None if dbias is False else _f32_out(dbias, "dbias", cols, x)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd are required")
    mean, rstd = _f32_out(mean, "mean", rows, x), _f32_out(rstd, "rstd", rows, x)
    ws, ws_bytes = _ws(ws, int(lib.mxgg_layer_norm_bwd_workspace(rows, cols)), x)
    _check(lib.mxgg_layer_norm_bwd(dy.data_ptr(), lddy, x.data_ptr(), ldx, rows, cols, dt, _at(weight), wd or 0,
                                   mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), lddx, _at(dweight), _at(dbias),
                                   1 if accumulate else 0, ws.data_ptr(), ws_bytes, _stream_of(x)))
    return dx, dweight, dbias


def _host_array(kind, code, values, n):
    """A ctypes array of n values (array.array takes them faster)."""
    return (kind * n).from_buffer(array.array(code, values)) if n else (kind * 1)()


def _grad_list(grads, total):
    """The host arrays of a gradient list, and a tensor of its device (the
    library checks that every pointer is memory of that GPU)."""
    grads = list(grads)
    n, T = len(grads), _torch().Tensor
    like = grads[0] if grads else total
    if n and like.get_device() < 0:
        raise ValueError(f"the gradients must be on a GPU, got one on {like.device}")
    # one pass in C for each property: a list of hundreds is the common case
    dtypes = list(map(_KINDS.get, map(operator.attrgetter("dtype"), grads)))
    if None in dtypes or not all(map(T.is_contiguous, grads)):
        for i, g in enumerate(grads):
            if g.dtype not in _KINDS or not g.is_contiguous():
                raise ValueError(f"gradient {i} must be a contiguous bf16 or fp32 tensor, got "
                                 f"{str(g.dtype).replace('torch.', '')} {tuple(g.shape)} with strides {g.stride()}")
    return (n, _host_array(ctypes.c_void_p, "Q", map(T.data_ptr, grads), n),
            _host_array(ctypes.c_int64, "q", map(T.numel, grads), n), _host_array(ctypes.c_int32, "i", dtypes, n), like)


def _quantize_int8(x, flags, q, scales):
    _check_bf16_2d(x)
    rows, cols = x.shape
    q = x.new_empty((rows, cols), dtype=_i8_t) if q is None else _expect(q, "q", (rows, cols), _i8_t)
    scales = x.new_empty(rows, dtype=_f32_t) if scales is None else _expect(scales, "scales", (rows,), _f32_t)
    _check(lib.mxgg_quantize_rowwise(x.data_ptr(), rows, cols, x.stride(0) if rows > 1 else cols, INT8, flags or 0,
                                     q.data_ptr(), scales.data_ptr(), _stream_of(x)))
    return q, scales


def _int8_splits(m_splits):
    """The array of _splits, faster for a list of ints, and its length."""
    vals = m_splits if isinstance(m_splits, (list, tuple)) else list(m_splits)
    try:
        return _host_array(ctypes.c_int64, "q", vals, len(vals)), len(vals)
    except TypeError:           # 2.0, as the other formats take it
        return _splits(vals)


def _grouped_fwd_int8(a_q, a_s, w_q, w_s, m_splits, N, K, out, ws):
    splits, G = _int8_splits(m_splits)
    M = a_q.shape[0] if a_q.dim() else 0
    _expect(a_q, "a_q", (M, K), _i8_t)
    _expect(a_s, "a_s", (M,), _f32_t)
    _expect(w_q, "w_q", (G * N, K), _i8_t)
    _expect(w_s, "w_s", (G * N,), _f32_t)
    out = a_q.new_empty((M, N), dtype=_bf16_t) if out is None else _expect(out, "out", (M, N), _bf16_t)
    ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.mxgg_grouped_fwd(a_q.data_ptr(), a_s.data_ptr(), INT8, w_q.data_ptr(), w_s.data_ptr(), INT8,
                                splits, G, M, N, K, out.data_ptr(), _at(ws), ws_bytes, _stream_of(a_q)))
    return out


def _norm_kind(norm_type):
    if float(norm_type) == 2.0:
        return NORM_L2
    if float(norm_type) == float("inf"):
        return NORM_MAX
    raise ValueError(f"norm_type must be 2 or inf, got {norm_type}")


def _total(total, like):
    torch = _torch()
    if total is None:
        return torch.empty((), dtype=torch.float32, device="cuda") if like is None \
            else like.new_empty((), dtype=_f32_t)
    if total.dtype != torch.float32 or total.numel() != 1:
        raise ValueError("total must be one fp32 value")
    return total if like is None else _on(total, like, "total")


def mxgg_grad_norm(grads, norm_type=2.0, total=None, ws=None):
    """The norm (2 or inf) of all gradients together, an fp32 scalar on their
    device. grads: contiguous bf16 / fp32 tensors, mixed; they must not
    overlap."""
    kind = _norm_kind(norm_type)
    n, ptrs, numels, dtypes, like = _grad_list(grads, total)
    total = _total(total, like)
    ws, ws_bytes = _ws(ws, int(lib.mxgg_grad_norm_workspace(n)), total)
    _check(lib.mxgg_grad_norm(ptrs, numels, dtypes, n, kind, total.data_ptr(), ws.data_ptr(), ws_bytes, _stream_of(total)))
    return total


def mxgg_clip_grad_norm(grads, max_norm, norm_type=2.0, total=None, ws=None):
    """grad_norm, then every gradient *= min(1, max_norm / (norm + 1e-6)) in
    place. Returns the norm (an fp32 scalar on the device; no host wait)."""
    kind = _norm_kind(norm_type)
    n, ptrs, numels, dtypes, like = _grad_list(grads, total)
    total = _total(total, like)
    ws, ws_bytes = _ws(ws, int(lib.mxgg_grad_norm_workspace(n)), total)
    _check(lib.mxgg_clip_grad_norm(ptrs, numels, dtypes, n, kind, max_norm, total.data_ptr(), ws.data_ptr(), ws_bytes,
                                   _stream_of(total)))
    return total


def mxgg_clip_grads_with_norm(grads, max_norm, total):
    """Scale the gradients in place by min(1, max_norm / (total + 1e-6)); total:
    fp32 scalar on the device, e.g. combined over ranks from grad_norm."""
    if total is None:
        raise ValueError("total is required")
    total = _total(total, None)
    n, ptrs, numels, dtypes, like = _grad_list(grads, total)
    _on(total, like, "total")
    _check(lib.mxgg_clip_grads_with_norm(ptrs, numels, dtypes, n, max_norm, total.data_ptr(), _stream_of(total)))
    return total


def mxgg_moe_layer(x, logits, w13_q, w13_s, w2_q, w2_s, top_k, fmt="mxfp4", renormalize=True, out=None, ids=None,
                   weights=None, ws=None, w2_fmt=None):
    """The whole expert layer for at most 64 tokens. x: bf16 [tokens, hidden];
    logits: the gate's output, bf16 or fp32 [tokens, experts]; w13: [experts *
    2 * inner, hidden] (gate rows, then up rows of each expert) and w2: [experts
    * hidden, inner] as quantize_rowwise(..., fmt) writes them, fmt "mxfp4",
    "mxfp8" (also | KBLOCK_ROWS) or "fp8_128x128" (_p2); w2_fmt: w2's where its
    code layout is another (with or without KBLOCK_ROWS). Returns (out, ids,
    weights): bf16 [tokens, hidden], int32 and fp32 [tokens, top_k]."""
    torch = _torch()
    f = _fmt(fmt)
    f2 = f if w2_fmt is None else _fmt(w2_fmt)
    if (f ^ f2) & ~KBLOCK_ROWS:
        raise ValueError("w2_fmt may differ from fmt in the code layout only (KBLOCK_ROWS)")
    if (f & 0xFF) not in (MXFP4, MXFP8, FP8_128x128, FP8_128x128_P2):
        raise ValueError("fmt must be a weight format: mxfp4, mxfp8 or fp8_128x128(_p2)")
    _check_bf16_2d(x)
    T, H = x.shape
    ldl, ldt = _rows2d(logits, "logits"), _dtype(logits, "logits")
    if logits.shape[0] != T:
        raise ValueError(f"logits must have {T} rows, got {logits.shape[0]}")
    E = logits.shape[1]
    inner = _q_rows(w13_q, f) // (2 * E) if E else 0
    _expect(w13_q, "w13_q", _q_shape(f, E * 2 * inner, H), torch.uint8)
    _expect(w13_s, "w13_s", _row_scale_shape(f, E * 2 * inner, H), _sdtype(f))
    _expect(w2_q, "w2_q", _q_shape(f2, E * H, inner), torch.uint8)
    _expect(w2_s, "w2_s", _row_scale_shape(f2, E * H, inner), _sdtype(f2))
    flags = MOE_RENORMALIZE if renormalize else 0
    if f != f2:
        flags |= MOE_W13_KBLOCK if f & KBLOCK_ROWS else MOE_W2_KBLOCK
    out = x.new_empty((T, H)) if out is None else _expect(out, "out", (T, H), torch.bfloat16)
    ids = x.new_empty((T, top_k), dtype=_i32_t) if ids is None else _expect(ids, "ids", (T, top_k), _i32_t)
    weights = x.new_empty((T, top_k), dtype=_f32_t) if weights is None \
        else _expect(weights, "weights", (T, top_k), _f32_t)
    ws, ws_bytes = _ws(ws, int(lib.mxgg_moe_layer_workspace(T, E, top_k, inner)), x)
    _check(lib.mxgg_moe_layer(x.data_ptr(), x.stride(0) if T > 1 else H, logits.data_ptr(), ldl, ldt, T, H, inner, E,
                              top_k, w13_q.data_ptr(), w13_s.data_ptr(), w2_q.data_ptr(), w2_s.data_ptr(),
                              f & f2, flags, out.data_ptr(), ids.data_ptr(), weights.data_ptr(), ws.data_ptr(), ws_bytes,
                              _stream_of(x)))
    return out, ids, weights


def _lead(t, name):
    """Leading dimension of a 2-D tensor with unit inner stride (one look for the
    common case)."""
    return t.shape[1] if t.is_contiguous() and t.dim() == 2 else _rows2d(t, name)


def _rows_index(rows):
    """(tokens, top_k) of the places that moe_sort writes."""
    shape = rows.shape
    if len(shape) != 2 or rows.dtype is not _i32_t or not rows.is_contiguous():
        raise ValueError(f"rows must be a contiguous int32 tensor [tokens, top_k], got "
                         f"{str(rows.dtype).replace('torch.', '')} {tuple(shape)}")
    return shape


def _like_rows(t, name, n, cols, x, named=None):
    """[n, cols] of x's type, the caller's or a new one, and its leading dimension.
    Of a new one only `named` rows may be written, the others are zeros. (That it
    is on x's device the library checks, as of every pointer.)"""
    if t is None:
        return x.new_empty((n, cols)) if named is None or n <= named else x.new_zeros((n, cols)), cols
    if t.shape != (n, cols) or t.dtype is not x.dtype:
        raise ValueError(f"{name} must be a {str(x.dtype).replace('torch.', '')} tensor [{n}, {cols}], got "
                         f"{str(t.dtype).replace('torch.', '')} {tuple(t.shape)}")
    return t, _lead(t, name)


def _i32_out(t, name, shape, like):
    return like.new_empty(shape, dtype=_i32_t) if t is None else _expect(t, name, shape, _i32_t)


def mxgg_moe_sort(ids, experts, rows=None, choices=None, counts=None, ws=None):
    """A router's choices in the order of their experts (stable). ids: int32 or
    int64 [tokens, top_k]; a choice outside [0, experts) is dropped. Returns
    (rows, choices, counts), int32: the place of each choice [tokens, top_k]
    (~place, behind all others, of a dropped one), the choice at each place
    [tokens * top_k], the rows of each expert [experts]: counts.tolist() are the
    grouped GEMMs' m_splits."""
    kind = _INTS.get(ids.dtype)
    if kind is None:
        raise ValueError(f"ids must be int32 or int64, got {str(ids.dtype).replace('torch.', '')}")
    ldi = _lead(ids, "ids")
    T, k = ids.shape
    rows = _i32_out(rows, "rows", (T, k), ids)
    choices = _i32_out(choices, "choices", (T * k,), ids)
    counts = _i32_out(counts, "counts", (experts,), ids)
    need = lib.mxgg_moe_sort_workspace(T, k, experts)
    at, ws_bytes = None, 0
    if need or ws is not None:
        ws, ws_bytes = _ws(ws, need, ids)
        at = ws.data_ptr()
    _check(lib.mxgg_moe_sort(ids.data_ptr(), kind, ldi, T, k, experts, rows.data_ptr(), choices.data_ptr(),
                             counts.data_ptr(), at, ws_bytes, _stream_of(ids)))
    return rows, choices, counts


def mxgg_moe_dispatch(x, rows, expert_rows=None, out=None):
    """Tokens' rows to the places of their choices: out[rows[t, j]] = x[t], zeros
    at the places of dropped ones. x: bf16 or fp32 [tokens, cols] (any row
    stride); rows from moe_sort; expert_rows: the rows of out (tokens * top_k, or
    sum(m_splits) to leave the dropped ones out; rows behind them are zeros, of a
    given out left as they were)."""
    dt, ldx = _dtype(x, "x"), _lead(x, "x")
    T, k = _rows_index(rows)
    n, cols = x.shape
    if n != T:
        raise ValueError(f"x has {n} rows, rows is of {T} tokens")
    if expert_rows is None:
        expert_rows = T * k if out is None else out.shape[0]
    out, ldo = _like_rows(out, "out", expert_rows, cols, x, T * k)
    _check(lib.mxgg_moe_dispatch(x.data_ptr(), ldx, dt, T, cols, rows.data_ptr(), k, out.data_ptr(), ldo, expert_rows,
                                 _stream_of(x)))
    return out


def mxgg_moe_combine(y, rows, weights=None, out=None):
    """Experts' rows back to their tokens: out[t] = sum_j weights[t, j] y[rows[t,
    j]] over the choices that are not dropped, summed in fp32. y: bf16 or fp32
    [expert rows, cols] (any row stride); weights: fp32 [tokens, top_k], None for
    1 (then it is the gradient of moe_dispatch)."""
    dt, ldy = _dtype(y, "y"), _lead(y, "y")
    T, k = _rows_index(rows)
    if weights is not None:
        _expect(weights, "weights", (T, k), _f32_t)
    n, cols = y.shape
    out, ldo = _like_rows(out, "out", T, cols, y)
    _check(lib.mxgg_moe_combine(y.data_ptr(), ldy, dt, n, cols, rows.data_ptr(), _at(weights), T, k, out.data_ptr(), ldo,
                                _stream_of(y)))
    return out


def mxgg_moe_combine_bwd(dout, y, rows, weights, dy=None, dweights=None):
    """The gradients of moe_combine: (dy, dweights), dy like y (zeros at the
    places of dropped choices and in rows behind all; a given dy keeps those),
    dweights fp32 [tokens, top_k]."""
    dt, ldy = _dtype(y, "y"), _lead(y, "y")
    T, k = _rows_index(rows)
    if dout is None:
        raise ValueError("dout is required")
    n, cols = y.shape
    dout, lddo = _like_rows(dout, "dout", T, cols, y)
    _expect(weights, "weights", (T, k), _f32_t)
    dy, lddy = _like_rows(dy, "dy", n, cols, y, T * k)
    dweights = y.new_empty((T, k), dtype=_f32_t) if dweights is None else _expect(dweights, "dweights", (T, k), _f32_t)
    _check(lib.mxgg_moe_combine_bwd(dout.data_ptr(), lddo, y.data_ptr(), ldy, dt, n, cols, rows.data_ptr(),
                                    weights.data_ptr(), T, k, dy.data_ptr(), lddy, dweights.data_ptr(), _stream_of(y)))
    return dy, dweights


def mxgg_dropout(x, p, state, stream=0, residual=None, out=None):
    """residual + x / (1 - p) where kept, residual where dropped; the mask is a
    function of state (int64 [2] on the device: seed and step), of `stream` (an
    int that tells the calls of a step apart) and of the element's row and column,
    so the same call on the gradient of out, without residual, is the gradient of
    x. x: bf16 or fp32 [rows, cols] (any row stride), residual and out like it; out
    may be x or residual."""
    dt, ldx = _dtype(x, "x"), _lead(x, "x")
    rows, cols = x.shape
    _expect(state, "state", (2,), _i64_t)
    if not 0 <= stream < 1 << 32:
        raise ValueError(f"stream={stream} outside [0, 2^32)")
    ldr = cols if residual is None else _like_rows(residual, "residual", rows, cols, x)[1]
    out, ldo = _like_rows(out, "out", rows, cols, x)
    _check(lib.mxgg_dropout(x.data_ptr(), ldx, dt, rows, cols, p, state.data_ptr(), stream, _at(residual), ldr,
                            out.data_ptr(), ldo, _stream_of(x)))
    return out


# short names
quantize_rowwise = mxgg_quantize_rowwise
quantize_colwise_segpad = mxgg_quantize_colwise_segpad
quantize_dual = mxgg_quantize_dual
grouped_fwd = mxgg_grouped_fwd
grouped_dgrad = mxgg_grouped_dgrad
transpose_128x128 = mxgg_transpose_128x128
grouped_wgrad = mxgg_grouped_wgrad
workspace_size = mxgg_workspace_size
segpad_rows = mxgg_segpad_rows
mx_scale_stride = mxgg_mx_scale_stride
mx_scales_relayout = mxgg_mx_scales_relayout
layer_norm_fwd = mxgg_layer_norm_fwd
layer_norm_bwd = mxgg_layer_norm_bwd
grad_norm = mxgg_grad_norm
clip_grad_norm = mxgg_clip_grad_norm
clip_grads_with_norm = mxgg_clip_grads_with_norm
moe_layer = mxgg_moe_layer
moe_sort = mxgg_moe_sort
moe_dispatch = mxgg_moe_dispatch
moe_combine = mxgg_moe_combine
moe_combine_bwd = mxgg_moe_combine_bwd
dropout = mxgg_dropout
