"""ctypes binding of libfp4_mi355x.so (include/fp4.h).

Argument marshalling only: torch tensors provide device memory, the current
torch stream is passed as the hipStream_t, and every computation runs in the
library's HIP kernels.  The library is loaded on first use; if it is missing
(not built) every call raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp4_mi355x.so")

NVFP4, UE5M3, MXFP4, MXFP8, FP8_E4M3, FP8_E5M2 = 0, 1, 2, 3, 5, 6
FORMATS = {"nvfp4": NVFP4, "ue5m3": UE5M3, "mxfp4": MXFP4, "mxfp8": MXFP8, "fp8": FP8_E4M3,
           "fp8_e5m2": FP8_E5M2}
FP8 = (FP8_E4M3, FP8_E5M2)      # one power-of-two scale per block of 128
BLOCK_LEN = {NVFP4: 16, UE5M3: 16, MXFP4: 32, MXFP8: 32, FP8_E4M3: 128, FP8_E5M2: 128}
RNE, SR = 0, 1
BLOCK_1D, BLOCK_2D16, BLOCK_2D128 = 0, 1, 2
ROWWISE, COLWISE = 0, 1
SCALES_ROWMAJOR, SCALES_TILED, SCALES_KMAJOR = 0, 1, 2
SCALE_LAYOUTS = {"rowmajor": SCALES_ROWMAJOR, "tiled": SCALES_TILED, "kmajor": SCALES_KMAJOR}
ACTS = {"swiglu": 0, "relu2": 1}
GLOBAL_TENSOR, GLOBAL_ROW = 0, 1
COUNT_LEVELS = {"all": 0, "scales": 1}
GLOBAL_SCOPES = {"tensor": GLOBAL_TENSOR, "row": GLOBAL_ROW}
COUNTER_NAMES = ("scale_saturated", "scale_underflow", "scale_subnormal",
                 "elem_saturated", "elem_underflow")


class Fp4Error(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(msg)
        self.status = status


class QuantDesc(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int), ("block", ctypes.c_int), ("orient", ctypes.c_int),
                ("round", ctypes.c_int), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("rht", ctypes.c_int), ("rht_signs", ctypes.c_uint32), ("target", ctypes.c_float),
                ("amax_given", ctypes.c_int), ("emit_transpose", ctypes.c_int),
                ("scale_layout", ctypes.c_int), ("rht_n", ctypes.c_int),
                ("rht_signs_hi", ctypes.c_uint32 * 3), ("scale_round", ctypes.c_int),
                ("global_scope", ctypes.c_int), ("count_level", ctypes.c_int)]


SCALE_ROUND = {"rne": 0, "up": 1}


def _sign_words(signs):
    """An up-to-128-bit sign mask as (bits 0-31, [bits 32-63, 64-95, 96-127])."""
    signs = int(signs)
    m = 0xFFFFFFFF
    return signs & m, (ctypes.c_uint32 * 3)((signs >> 32) & m, (signs >> 64) & m, (signs >> 96) & m)


class Operand(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int), ("codes", ctypes.c_void_p), ("ld_codes", ctypes.c_int64),
                ("scales", ctypes.c_void_p), ("scale_stride_row", ctypes.c_int64),
                ("scale_stride_kblk", ctypes.c_int64), ("scale_row_group", ctypes.c_int32),
                ("s_dec", ctypes.c_void_p), ("scale_layout", ctypes.c_int),
                ("s_dec_scope", ctypes.c_int)]


class Heads(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64), ("heads", ctypes.c_int64)]


class QKNormDesc(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("weight_f32", ctypes.c_int), ("eps", ctypes.c_float), ("table", ctypes.c_void_p),
                ("table_rows", ctypes.c_int64), ("rotary_dim", ctypes.c_int),
                ("interleaved", ctypes.c_int)]


class KVCacheDesc(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("page_size", ctypes.c_int), ("pages", ctypes.c_int64),
                ("k_codes", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("scale_page_stride", ctypes.c_int64),
                ("scale_head_stride", ctypes.c_int64), ("scale_block_stride", ctypes.c_int64),
                ("amax", ctypes.c_void_p), ("target", ctypes.c_float)]


_lib = None
EXPORTS = ("fp4_amax", "fp4_quantize", "fp4_dequantize", "fp4_rht16", "fp4_gemm",
           "fp4_gemm_ws", "fp4_gemm_workspace", "fp4_requantize_t", "fp4_act_quantize",
           "fp4_act_backward", "fp4_qk_norm_rope", "fp4_qk_norm_rope_backward",
           "fp4_qk_norm_workspace", "fp4_kv_cache_write", "fp4_kv_cache_read",
           "fp4_attention_decode", "fp4_attention_workspace",
           "fp4_status_string", "fp4_last_error")


def load_library(path=None):
    """Load (once) and return the ctypes library; raises if it is not built.
    The path defaults to $FP4_LIB if set (e.g. the sanitized host build of
    the argument checks), else the in-tree library."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("FP4_LIB") or LIB_PATH
    if not os.path.exists(path):
        raise Fp4Error(-1, "%s is missing: build it with __graft_entry__.build() "
                           "(python fp4_block_scaled_x16_amd/build.py)" % path)
    lib = ctypes.CDLL(path)
    i64, vp, u32, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int
    lib.fp4_amax.argtypes = [ctypes.POINTER(QuantDesc), vp, i64, i64, i64, vp, vp]
    lib.fp4_quantize.argtypes = [ctypes.POINTER(QuantDesc), vp, i64, i64, i64, vp, vp, vp, vp,
                                 vp, vp, vp]
    lib.fp4_quantize_dual.argtypes = [ctypes.POINTER(QuantDesc), ctypes.POINTER(QuantDesc), vp, i64,
                                      i64, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    lib.fp4_dequantize.argtypes = [i32, i32, i32, vp, vp, vp, i32, i64, i64, vp, i32, vp]
    lib.fp4_rht16.argtypes = [ctypes.POINTER(QuantDesc), vp, i64, i64, i64, vp, vp]
    lib.fp4_requantize_t.argtypes = [i32, vp, vp, i64, i64, vp, vp, vp]
    lib.fp4_act_quantize.argtypes = [i32, vp, i64, i64, i64, vp, vp, vp, i64, vp, vp, vp]
    lib.fp4_act_backward.argtypes = [i32, vp, vp, vp, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp,
                                     vp, i64, vp, i64, vp]
    lib.fp4_gemm.argtypes = [ctypes.POINTER(Operand), ctypes.POINTER(Operand), i64, i64, i64, vp,
                             i32, i64, i32, vp]
    lib.fp4_gemm_ws.argtypes = lib.fp4_gemm.argtypes[:-1] + [vp, i64, vp]
    lib.fp4_gemm_workspace.argtypes = [ctypes.POINTER(Operand), ctypes.POINTER(Operand), i64, i64,
                                       i64, i32]
    lib.fp4_gemm_workspace.restype = i64
    heads = norm = cache = vp       # structs by address: a byref, or what addressof gives
    lib.fp4_qk_norm_rope.argtypes = [norm, heads, heads, vp, i64, i64, heads, heads, vp]
    lib.fp4_qk_norm_rope_backward.argtypes = [norm, heads, heads, vp, i64, i64, heads, heads, heads,
                                              heads, vp, vp, i32, vp, i64, vp]
    lib.fp4_qk_norm_workspace.argtypes = [i64]
    lib.fp4_kv_cache_write.argtypes = [cache, heads, heads, vp, i64, norm, vp, heads, heads, vp]
    lib.fp4_kv_cache_read.argtypes = [cache, vp, i64, vp, vp, i32, vp]
    lib.fp4_attention_decode.argtypes = [cache, heads, vp, i64, i64, vp, i64, ctypes.c_float, vp, i32,
                                         vp, vp, i64, vp]
    lib.fp4_attention_workspace.argtypes = [cache, i64, i64, i64]
    lib.fp4_qk_norm_workspace.restype = lib.fp4_attention_workspace.restype = i64
    lib.fp4_selftest_set_attention_splits.argtypes = [i32]
    lib.fp4_selftest_sweep.argtypes = [i32, vp, i32, vp, vp]
    lib.fp4_selftest_gemm_decode.argtypes = [i32, vp, vp]
    lib.fp4_selftest_set_geometry.argtypes = [i32, i32]
    lib.fp4_selftest_set_fp8_plan.argtypes = [i32, i32]
    for f in ("fp4_amax", "fp4_quantize", "fp4_quantize_dual", "fp4_dequantize", "fp4_rht16",
              "fp4_requantize_t", "fp4_act_quantize", "fp4_act_backward", "fp4_gemm", "fp4_gemm_ws",
              "fp4_selftest_sweep", "fp4_selftest_gemm_decode", "fp4_selftest_set_geometry",
              "fp4_selftest_set_fp8_plan", "fp4_qk_norm_rope", "fp4_qk_norm_rope_backward",
              "fp4_kv_cache_write", "fp4_kv_cache_read", "fp4_attention_decode",
              "fp4_selftest_set_attention_splits"):
        getattr(lib, f).restype = ctypes.c_int
    lib.fp4_status_string.argtypes = [ctypes.c_int]
    lib.fp4_status_string.restype = ctypes.c_char_p
    lib.fp4_last_error.argtypes = []
    lib.fp4_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status, what):
    if status != 0:
        lib = load_library()
        raise Fp4Error(status, "%s: %s (%s)" % (what, lib.fp4_status_string(status).decode(),
                                               lib.fp4_last_error().decode()))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device=None):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


# the current stream's handle, without an object around it where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch(what, fn, device, *args):
    """fn(*args, stream) on the device's current stream, with the device made
    current where another one is."""
    if device.type != "cuda":
        raise ValueError("%s: tensors must be on the GPU (got %s)" % (what, device))
    if device.index == torch.cuda.current_device():
        stream = (_raw_stream(device.index) if _raw_stream
                  else torch.cuda.current_stream(device).cuda_stream)
        status = fn(*args, stream)
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if status:
        _check(status, what)


def _addr(t):
    return None if t is None else t.data_ptr()


def _as_bf16_bits(x):
    if x.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError("x must be bfloat16 (or its int16 bit view)")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D row-major tensor")
    return x


def _fmt(fmt):
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


# ------------------------------------------------------------------ amax --
def _rht_desc(orient, rht, signs, rht_n):
    s_lo, s_hi = _sign_words(signs)
    return QuantDesc(NVFP4, BLOCK_1D, COLWISE if orient == "col" else ROWWISE, RNE, 0, 0,
                     int(bool(rht)), s_lo, 448.0, 0, 0, SCALES_ROWMAJOR, int(rht_n), s_hi, 0)


def amax(x, rht=False, signs=0, out=None, rht_n=16, orient="col"):
    """Tensor amax -> device fp32 [1]; with rht, of the tensor rotated along
    the blocked axis of `orient` ("col": N-row groups of each column, the
    Wgrad operands; "row": N-column groups of each row, Fprop / Dgrad)."""
    x = _as_bf16_bits(x)
    out = torch.empty(1, dtype=torch.float32, device=x.device) if out is None else out
    desc = _rht_desc(orient, rht, signs, rht_n)
    lib = load_library()
    _check(lib.fp4_amax(ctypes.byref(desc), _ptr(x), x.shape[0], x.shape[1], x.stride(0),
                        _ptr(out), _stream(x.device)), "fp4_amax")
    return out


# -------------------------------------------------------------- quantize --
@dataclass
class Quantized:
    """Codes and scales of one quantized matrix, plus what a GEMM needs."""
    fmt: int
    block: int
    rows: int               # rows of the code matrix
    cols: int               # cols of the code matrix (the blocked axis for 1D)
    codes: torch.Tensor     # uint8 [rows, cols/2] (MXFP8: [rows, cols], a byte per element;
                            # FP8: [rows, cols up to 128], zeros from cols on)
    scales: torch.Tensor    # uint8 1D: [rows, cols/BS] (TILED: flat, tiled_scale_bytes);
                            # 2D: [rows/16, cols/16]; FP8: [blocks of cols, rows up to 16]
    s_dec: torch.Tensor     # fp32 [1], or [rows] with per-row global scales (FP8: None)
    amax: torch.Tensor      # fp32 [1] or [rows] (two-level formats)
    codes_t: torch.Tensor = None   # 2D with emit_transpose: [cols, rows/2]
    scale_layout: int = SCALES_ROWMAJOR
    scope: int = GLOBAL_TENSOR     # GLOBAL_ROW: one global scale per row

    def operand(self, transposed=False):
        """GEMM operand over the K-major code matrix (K = cols), or for 2D
        weights with transposed=True over the codes of the transpose.

        The operand holds raw device pointers; it keeps this object (and so
        its tensors) alive for as long as the operand itself is referenced.
        """
        bs = BLOCK_LEN[self.fmt]
        if self.fmt == MXFP8:
            raise ValueError("no GEMM takes MXFP8 operands")
        if self.fmt in FP8:
            if transposed:
                raise ValueError("an FP8 transpose is a Quantized of its own (quantize_dual)")
            op = Operand(self.fmt, self.codes.data_ptr(), self.codes.shape[1],
                         self.scales.data_ptr(), 0, self.scales.shape[1], 1, None, SCALES_KMAJOR,
                         GLOBAL_TENSOR)
        elif self.block == BLOCK_1D:
            assert not transposed
            op = Operand(self.fmt, self.codes.data_ptr(), self.cols // 2, self.scales.data_ptr(),
                         self.cols // bs, 1, 1, self.s_dec.data_ptr(), self.scale_layout,
                         self.scope)
        elif not transposed:
            op = Operand(self.fmt, self.codes.data_ptr(), self.cols // 2, self.scales.data_ptr(),
                         self.cols // 16, 1, 16, self.s_dec.data_ptr(), SCALES_ROWMAJOR)
        else:
            assert self.codes_t is not None
            op = Operand(self.fmt, self.codes_t.data_ptr(), self.rows // 2, self.scales.data_ptr(),
                         1, self.cols // 16, 16, self.s_dec.data_ptr(), SCALES_ROWMAJOR)
        op._owner = self
        return op


def tiled_scale_bytes(rows, blocks_per_row):
    """Size of the TILED scale buffer of a [rows, blocks_per_row] scale matrix:
    2 KiB atoms of 256 rows x 8 blocks."""
    return -(-rows // 256) * -(-blocks_per_row // 8) * 2048


def quantize(x, fmt="nvfp4", block="1d", orient="row", rnd="rne", seed=0, offset=0, rht=False,
             signs=0, target=448.0, amax_in=None, emit_transpose=False, counters=None,
             scale_layout=None, rht_n=16, scale_round="rne", global_scope="tensor",
             count="all"):
    """Quantize a bf16 [R, C] matrix.  orient="col" quantizes X^T ([C, R]).
    scale_layout: "rowmajor" (the default) or "tiled" (1D blocks only).
    fmt "fp8" (E4M3) and "fp8_e5m2": any R and C, block "1d" (1x128) or "2d"
    (128x128), orient "row" or "col", rnd "rne"; scales "kmajor"; x's row pitch a
    multiple of 8, as ever; their scales are always rounded up and depend on x
    alone, so scale_round and target mean nothing there.  rht_n: size of the RHT (4, 16, 32, 64, 128); signs:
    its sign mask, up to 128 bits.
    scale_round: "rne" or "up" (truncation-free block scales).
    global_scope: "tensor" or "row" (rowwise 1D NVFP4 / UE5M3: one global
    scale per row, amax and s_dec of R entries, no separate amax pass).

    amax_in: None -> computed on the device; else a device fp32 [1] tensor read
    as the (possibly stale) tensor amax ([R] per-row amaxes with "row").
    counters: optional device uint64 [5] tensor, accumulated; count: "all"
    or "scales" (block-scale events only).
    """
    x = _as_bf16_bits(x)
    f = _fmt(fmt)
    if f in FP8:
        return _quantize_fp8(x, f, block, orient, orient != "col", orient == "col", rnd, rht,
                             amax_in, emit_transpose, counters, scale_layout, global_scope,
                             count)[0]
    scale_layout = "rowmajor" if scale_layout is None else scale_layout
    R, C = x.shape
    blk = BLOCK_2D16 if block == "2d" else BLOCK_1D
    col = orient == "col"
    rows, cols = (C, R) if col else (R, C)
    bs = 16 if blk == BLOCK_2D16 else BLOCK_LEN[f]
    dev = x.device
    code_cols = cols if f == MXFP8 else cols // 2
    codes = torch.empty((rows, code_cols), dtype=torch.uint8, device=dev)
    layout = SCALE_LAYOUTS[scale_layout] if isinstance(scale_layout, str) else int(scale_layout)
    if blk == BLOCK_2D16:
        scales = torch.empty((rows // 16, cols // 16), dtype=torch.uint8, device=dev)
    elif layout == SCALES_TILED:
        scales = torch.empty(tiled_scale_bytes(rows, cols // bs), dtype=torch.uint8, device=dev)
    else:
        scales = torch.empty((rows, cols // bs), dtype=torch.uint8, device=dev)
    codes_t = (torch.empty((cols, rows // 2), dtype=torch.uint8, device=dev)
               if emit_transpose else None)
    scope = GLOBAL_SCOPES[global_scope]
    n_g = rows if scope == GLOBAL_ROW else 1
    s_dec = torch.empty(n_g, dtype=torch.float32, device=dev)
    am = amax_in if amax_in is not None else torch.empty(n_g, dtype=torch.float32, device=dev)
    s_lo, s_hi = _sign_words(signs)
    desc = QuantDesc(f, blk, COLWISE if col else ROWWISE, SR if rnd == "sr" else RNE,
                     int(seed), int(offset), int(bool(rht)), s_lo, float(target),
                     int(amax_in is not None), int(bool(emit_transpose)), layout, int(rht_n), s_hi,
                     SCALE_ROUND[scale_round], scope, COUNT_LEVELS[count])
    lib = load_library()
    _check(lib.fp4_quantize(ctypes.byref(desc), _ptr(x), R, C, x.stride(0), _ptr(codes),
                            _ptr(scales), _ptr(codes_t), _ptr(am), _ptr(s_dec), _ptr(counters),
                            _stream(dev)), "fp4_quantize")
    return Quantized(f, blk, rows, cols, codes, scales, s_dec, am, codes_t, layout, scope)


def _scales_1d(rows, blocks, layout, dev):
    if layout == SCALES_TILED:
        return torch.empty(tiled_scale_bytes(rows, blocks), dtype=torch.uint8, device=dev)
    return torch.empty((rows, blocks), dtype=torch.uint8, device=dev)


def quantize_dual(x, fmt="nvfp4", rnd="rne", seed=0, offset=0, offset_t=None, rht=False, signs=0,
                  target=448.0, amax_in=None, amax_t_in=None, counters=None,
                  scale_layout=None, scale_layout_t=None, rht_n=16, scale_round="rne",
                  rht_row=False, signs_row=0, rht_n_row=16, count="all", block="1d"):
    """Rowwise and colwise 1D quantization of a bf16 [R, C] matrix from one
    read: returns (rowwise Quantized [R, C], colwise Quantized of X^T [C, R]).

    Both sides use `rnd` and `seed`; the colwise side uses offset_t (default
    offset + 1), the RHT (rht/signs/rht_n, along the columns) and
    scale_layout_t (default scale_layout); the rowwise side may rotate along
    the rows (rht_row/signs_row, rht_n_row 4 or 16).  amax_in / amax_t_in:
    None -> computed on the device, else device fp32 [1] tensors read as
    the given amax of each side.  count: "all" or "scales" (block-scale
    events only).  block: "1d", or with the FP8 formats "2d" (one scale per
    128x128 tile, so the colwise codes are the rowwise ones transposed).
    """
    x = _as_bf16_bits(x)
    f = _fmt(fmt)
    if f in FP8:
        return _quantize_fp8(x, f, block, "row", True, True, rnd, rht or rht_row,
                             amax_in if amax_in is not None else amax_t_in, False, counters,
                             scale_layout, "tensor", count, scale_layout_t)
    if block != "1d":
        raise ValueError("2D dual quantization needs an FP8 format (NVFP4, UE5M3: quantize with "
                         "emit_transpose)")
    scale_layout = "rowmajor" if scale_layout is None else scale_layout
    R, C = x.shape
    bs = BLOCK_LEN[f]
    dev = x.device
    lay = SCALE_LAYOUTS[scale_layout] if isinstance(scale_layout, str) else int(scale_layout)
    lay_t = lay if scale_layout_t is None else (
        SCALE_LAYOUTS[scale_layout_t] if isinstance(scale_layout_t, str) else int(scale_layout_t))
    if offset_t is None:
        offset_t = offset + 1
    codes = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
    codes_t = torch.empty((C, R // 2), dtype=torch.uint8, device=dev)
    scales = _scales_1d(R, C // bs, lay, dev)
    scales_t = _scales_1d(C, R // bs, lay_t, dev)
    s_dec = torch.empty(1, dtype=torch.float32, device=dev)
    s_dec_t = torch.empty(1, dtype=torch.float32, device=dev)
    am = amax_in if amax_in is not None else torch.empty(1, dtype=torch.float32, device=dev)
    am_t = amax_t_in if amax_t_in is not None else torch.empty(1, dtype=torch.float32, device=dev)
    r = SR if rnd == "sr" else RNE
    s_lo, s_hi = _sign_words(signs)
    sr_mode = SCALE_ROUND[scale_round]
    r_lo, r_hi = _sign_words(signs_row)
    cl = COUNT_LEVELS[count]
    d_row = QuantDesc(f, BLOCK_1D, ROWWISE, r, int(seed), int(offset), int(bool(rht_row)), r_lo,
                      float(target), int(amax_in is not None), 0, lay, int(rht_n_row), r_hi,
                      sr_mode, GLOBAL_TENSOR, cl)
    d_col = QuantDesc(f, BLOCK_1D, COLWISE, r, int(seed), int(offset_t), int(bool(rht)), s_lo,
                      float(target), int(amax_t_in is not None), 0, lay_t, int(rht_n), s_hi,
                      sr_mode, GLOBAL_TENSOR, cl)
    lib = load_library()
    _check(lib.fp4_quantize_dual(ctypes.byref(d_row), ctypes.byref(d_col), _ptr(x), R, C,
                                 x.stride(0), _ptr(codes), _ptr(scales), _ptr(codes_t),
                                 _ptr(scales_t), _ptr(am), _ptr(am_t), _ptr(s_dec), _ptr(s_dec_t),
                                 _ptr(counters), _stream(dev)), "fp4_quantize_dual")
    return (Quantized(f, BLOCK_1D, R, C, codes, scales, s_dec, am, None, lay),
            Quantized(f, BLOCK_1D, C, R, codes_t, scales_t, s_dec_t, am_t, None, lay_t))


def _up(v, to):
    return -(-v // to) * to


def _fp8_buffers(fmt, rows, cols, near, block=BLOCK_1D):
    """An FP8 code matrix [rows, cols] whose contents a kernel writes, on the
    device of `near` (new_empty of a uint8 tensor is the cheapest allocation)."""
    kb = (cols + 127) >> 7
    if near.dtype is torch.uint8:
        codes = near.new_empty(rows, kb << 7)
    else:
        codes = near.new_empty((rows, kb << 7), dtype=torch.uint8)
    scales = codes.new_empty(kb, (rows + 15) & -16)
    return Quantized(fmt, block, rows, cols, codes, scales, None, None, None, SCALES_KMAJOR)


def _quantize_fp8(x, f, block, orient, row, col, rnd, rht, amax_in, emit_transpose, counters,
                  scale_layout, global_scope, count, scale_layout_t=None):
    R, C = x.shape
    blk, d, d_t = _fp8_descs(f, block, orient, rnd, bool(rht), amax_in is not None,
                             bool(emit_transpose), scale_layout, scale_layout_t, global_scope,
                             count)
    if counters is not None and (counters.device != x.device or counters.dtype != torch.int64
                                 or counters.shape != (5,) or not counters.is_contiguous()):
        raise ValueError("counters must be an int64 [5] tensor on x's device (new_counters)")
    lib = load_library()
    if row and col:
        q = _fp8_buffers(f, R, C, x, blk)
        q_t = _fp8_buffers(f, C, R, q.codes, blk)
        _launch("fp4_quantize_dual", lib.fp4_quantize_dual, x.device, d, d_t, x.data_ptr(), R, C,
                _ld(x), q.codes.data_ptr(), q.scales.data_ptr(), q_t.codes.data_ptr(),
                q_t.scales.data_ptr(), None, None, None, None, _addr(counters))
        return q, q_t
    q = _fp8_buffers(f, R, C, x, blk) if row else _fp8_buffers(f, C, R, x, blk)
    _launch("fp4_quantize", lib.fp4_quantize, x.device, d if row else d_t, x.data_ptr(), R, C,
            _ld(x), q.codes.data_ptr(), q.scales.data_ptr(), None, None, None, _addr(counters))
    return q,


@functools.lru_cache(maxsize=64)
def _fp8_descs(f, block, orient, rnd, rht, amax_given, emit_transpose, scale_layout, scale_layout_t,
               scope, count):
    """The block's code and the (never written) descriptors of either orientation."""
    if block not in ("1d", "2d") or orient not in ("row", "col"):
        raise ValueError("block must be '1d' or '2d' and orient 'row' or 'col'")

    def layout_of(layout):
        return SCALE_LAYOUTS[layout] if isinstance(layout, str) else int(layout)

    layout = SCALES_KMAJOR
    if scale_layout is not None or scale_layout_t is not None:
        layout = layout_of(scale_layout_t if scale_layout is None else scale_layout)
    layout_t = layout if scale_layout_t is None else layout_of(scale_layout_t)
    blk = BLOCK_2D128 if block == "2d" else BLOCK_1D
    return blk, *(ctypes.byref(QuantDesc(f, blk, o, SR if rnd == "sr" else RNE, 0, 0, int(rht), 0,
                                         448.0, int(amax_given), int(emit_transpose), lay, 0,
                                         (ctypes.c_uint32 * 3)(), 0, GLOBAL_SCOPES[scope],
                                         COUNT_LEVELS[count]))
                  for o, lay in ((ROWWISE, layout), (COLWISE, layout_t)))


def _bytes(t, dtype, name):
    """uint8 t, or the bytes of one of the dtype."""
    if t.dtype == torch.uint8:
        return t
    if t.dtype != dtype:
        raise ValueError("%s must be uint8 or %s, not %s" % (name, dtype, t.dtype))
    return t.view(torch.uint8)


def fp8_matrix(codes, scales, rows, cols, fmt="fp8"):
    """A Quantized of FP8 codes and scales that exist already (a checkpoint's
    weights): codes uint8 (or fmt's torch dtype, float8_e4m3fn or float8_e5m2)
    [rows, cols up to 128], zeros from cols on; scales uint8 (or float8_e8m0fnu)
    [blocks of cols, rows up to 16], the byte of (block j, row r) being e + 127 of
    the scale 2^e."""
    f = _fmt(fmt)
    if f not in FP8:
        raise ValueError("fmt must be 'fp8' or 'fp8_e5m2'")
    codes = _bytes(codes, torch.float8_e4m3fn if f == FP8_E4M3 else torch.float8_e5m2, "codes")
    scales = _bytes(scales, torch.float8_e8m0fnu, "scales")
    kb = -(-cols // 128)
    if codes.shape != (rows, 128 * kb) or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous [%d, %d] tensor" % (rows, 128 * kb))
    if scales.shape != (kb, _up(rows, 16)) or not scales.is_contiguous():
        raise ValueError("scales must be a contiguous [%d, %d] tensor" % (kb, _up(rows, 16)))
    if codes.device != scales.device:
        raise ValueError("codes and scales are on different devices")
    return Quantized(f, BLOCK_1D, rows, cols, codes, scales, None, None,
                     scale_layout=SCALES_KMAJOR)


def _fp8_only(q, what):
    if q.fmt not in FP8:
        raise ValueError("%s takes FP8 codes" % what)


def requantize_t(q: Quantized):
    """The Quantized [cols, rows] of the transpose, in blocks along q's rows,
    from FP8 codes along its columns: the Wgrad operand of an activation that
    was kept as its 8-bit Fprop operand alone.  Exact but for elements below the
    normal range of their new block."""
    _fp8_only(q, "requantize_t")
    t = _fp8_buffers(q.fmt, q.cols, q.rows, q.codes)
    _launch("fp4_requantize_t", load_library().fp4_requantize_t, q.codes.device, q.fmt,
            q.codes.data_ptr(), q.scales.data_ptr(), q.rows, q.cols, t.codes.data_ptr(),
            t.scales.data_ptr())
    return t


# ------------------------------------------------------------ activation --
def _checkpoint_cols(act, cols):
    """Columns of the checkpoint of an activation of `cols` outputs: SwiGLU's u
    starts at a whole block."""
    return _up(cols, 128) + cols if act == "swiglu" else cols


def _ld(x):
    """Row pitch of a bf16 matrix for the library (a multiple of 8): a single
    row's is free to choose."""
    return x.stride(0) if x.shape[0] > 1 else _up(x.shape[1], 8)


def _bf16_rows(rows, cols, device):
    """A bf16 [rows, cols] matrix whose rows start 16-byte aligned."""
    return torch.empty((rows, _up(cols, 8)), dtype=torch.bfloat16, device=device)[:, :cols]


def _act_bits(x, name):
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("%s must be a row-major 2-D bfloat16 tensor" % name)
    return x


def act_quantize(h, act="swiglu", a="fp8", checkpoint=True):
    """(a, checkpoint) of a feed-forward layer's activation, from one read of
    bf16 h: [tokens, 2F] = [g | u] for "swiglu" (a = silu(g) u, F a multiple of
    8), [tokens, F] for "relu2" (a = max(h, 0)^2).

    a: "fp8" -> the E4M3 Quantized [tokens, F] that the second linear's product
    takes; "bf16" -> the values, for a linear of another format; None -> None.
    checkpoint: h as E4M3 codes (a Quantized; its u starts at a multiple of 128
    columns), from which `act_backward` works; False -> None.
    """
    h = _act_bits(h, "h")
    if act not in ACTS:
        raise ValueError("act must be one of %s" % (tuple(ACTS),))
    if a not in ("fp8", "bf16", None):
        raise ValueError("a must be 'fp8', 'bf16' or None")
    rows, cols = h.shape
    if act == "swiglu":
        if cols % 2:
            raise ValueError("h must be [tokens, 2F] for 'swiglu'")
        cols //= 2
    dev = h.device
    qa = _fp8_buffers(FP8_E4M3, rows, cols, h) if a == "fp8" else None
    av = _bf16_rows(rows, cols, dev) if a == "bf16" else None
    qh = (_fp8_buffers(FP8_E4M3, rows, _checkpoint_cols(act, cols), qa.codes if qa else h)
          if checkpoint else None)
    _launch("fp4_act_quantize", load_library().fp4_act_quantize, dev, ACTS[act], h.data_ptr(), rows,
            cols, _ld(h), qa and qa.codes.data_ptr(), qa and qa.scales.data_ptr(), _addr(av),
            0 if av is None else _ld(av), qh and qh.codes.data_ptr(), qh and qh.scales.data_ptr())
    return (av if a == "bf16" else qa), qh


def act_backward(qh: Quantized, da, act="swiglu", fmt="fp8", out="fp8"):
    """The backward pass of `act_quantize` at the values of its checkpoint qh,
    for da, the bf16 [tokens, F] gradient of a.

    out "fp8": (dh, dh_t, a_t) -- dh along its rows (columns as the checkpoint's)
    and dh^T [2F or F, tokens] in `fmt` ("fp8" or "fp8_e5m2"), the operands of the
    first linear's Dgrad and Wgrad, and E4M3 a^T [F, tokens], recomputed, of
    the second linear's Wgrad.
    out "bf16": (dh [tokens, 2F or F], a [tokens, F]) as values.
    """
    da = _act_bits(da, "da")
    f = _fmt(fmt)
    if act not in ACTS:
        raise ValueError("act must be one of %s" % (tuple(ACTS),))
    if f not in FP8 or out not in ("fp8", "bf16"):
        raise ValueError("fmt must be 'fp8' or 'fp8_e5m2' and out 'fp8' or 'bf16'")
    rows, cols = da.shape
    if qh.fmt != FP8_E4M3 or (qh.rows, qh.cols) != (rows, _checkpoint_cols(act, cols)):
        raise ValueError("the checkpoint must be the E4M3 [%d, %d] one of act_quantize"
                         % (rows, _checkpoint_cols(act, cols)))
    dev = da.device
    if qh.codes.device != dev:
        raise ValueError("the checkpoint and da are on different devices")
    halves = 2 if act == "swiglu" else 1
    o = [None] * 6
    dh = av = None
    if out == "fp8":
        near = qh.codes
        q = (_fp8_buffers(f, rows, qh.cols, near), _fp8_buffers(f, halves * cols, rows, near),
             _fp8_buffers(FP8_E4M3, cols, rows, near))
        o = [t.data_ptr() for p in q for t in (p.codes, p.scales)]
    else:
        dh, av = _bf16_rows(rows, halves * cols, dev), _bf16_rows(rows, cols, dev)
    _launch("fp4_act_backward", load_library().fp4_act_backward, dev, ACTS[act],
            qh.codes.data_ptr(), qh.scales.data_ptr(), da.data_ptr(), rows, cols, _ld(da), f,
            *o, _addr(dh), 0 if dh is None else _ld(dh), _addr(av),
            0 if av is None else _ld(av))
    return q if out == "fp8" else (dh, av)


def new_counters(device="cuda"):
    return torch.zeros(5, dtype=torch.int64, device=device)


def counters_dict(c):
    return dict(zip(COUNTER_NAMES, [int(v) for v in c.cpu().tolist()]))


# ------------------------------------------------------------ dequantize --
def dequantize(q: Quantized, out_dtype=torch.float32, out=None):
    """Values of a quantized matrix as fp32 or bf16 [rows, cols] (into `out`,
    a contiguous tensor of that shape and dtype, when given)."""
    if out is None:
        out = torch.empty((q.rows, q.cols), dtype=out_dtype, device=q.codes.device)
    elif (out.dtype != out_dtype or tuple(out.shape) != (q.rows, q.cols)
          or not out.is_contiguous()):
        raise ValueError("out must be a contiguous %s tensor of shape (%d, %d)"
                         % (out_dtype, q.rows, q.cols))
    elif out.device != q.codes.device:
        raise ValueError("out and the codes are on different devices")
    _launch("fp4_dequantize", load_library().fp4_dequantize, out.device, q.fmt, q.block,
            q.scale_layout, q.codes.data_ptr(), q.scales.data_ptr(), _addr(q.s_dec), q.scope,
            q.rows, q.cols, out.data_ptr(), int(out_dtype == torch.float32))
    return out


# ------------------------------------------------------------------- RHT --
def rht16(x, signs, rht_n=16, orient="col", out=None):
    """The RHT alone (fp32 [R, C]) along the blocked axis of `orient` (into
    `out`, a contiguous fp32 tensor of x's shape, when given)."""
    x = _as_bf16_bits(x)
    if out is None:
        y = torch.empty(x.shape, dtype=torch.float32, device=x.device)
    elif out.dtype != torch.float32 or out.shape != x.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous fp32 tensor of the input's shape")
    else:
        y = out
    desc = _rht_desc(orient, True, signs, rht_n)
    lib = load_library()
    _check(lib.fp4_rht16(ctypes.byref(desc), _ptr(x), x.shape[0], x.shape[1], x.stride(0),
                         _ptr(y), _stream(x.device)), "fp4_rht16")
    return y


# ------------------------------------------------------------------ GEMM --
OUT_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def gemm(a: Operand, b: Operand, M, N, K, out=None, accumulate=False, device=None,
         out_dtype=torch.float32):
    """D[M, N] (+)= s_A s_B sum_k a[m, k] b[n, k], written as fp32 or bf16
    (the dtype of `out` when given, else out_dtype).  FP8: a is "fp8" or
    "fp8_e5m2" and b "fp8"; K is their code matrices' cols, whole.  A row's bf16
    result may differ in its last bit with the number of rows beside it: up to 16
    rows are summed in fp32 throughout, more by the 8-bit matrix instructions."""
    if a.format in FP8 and b.format in FP8:
        qa, qb = getattr(a, "_owner", None), getattr(b, "_owner", None)
        if qa and qb and (qa.cols != K or qb.cols != K or M > qa.rows or N > qb.rows):
            raise ValueError("operands [%d, %d] and [%d, %d] do not make a product of M=%d, N=%d, "
                             "K=%d" % (qa.rows, qa.cols, qb.rows, qb.cols, M, N, K))
        if device is None and qa:
            device = qa.codes.device
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=device or "cuda")
    if out.dtype not in OUT_TYPES or out.dim() != 2 or (out.stride(1) != 1 and out.shape[1] > 1):
        raise ValueError("out must be a row-major 2-D fp32 or bf16 tensor")
    if out.shape[0] < M or out.shape[1] < N:
        raise ValueError("out is smaller than [%d, %d]" % (M, N))
    lib = load_library()
    t, dev = OUT_TYPES[out.dtype], out.device
    ws, n = None, 0
    if a.format in FP8 and b.format in FP8:
        if qa and qb and (qa.codes.device != dev or qb.codes.device != dev):
            raise ValueError("the operands and out are on different devices")
        n = _gemm_workspace(dev, M, N, K, t, a.format, b.format, a.ld_codes, b.ld_codes)
        if n:
            ws = torch.empty(n, dtype=torch.uint8, device=dev)
    _launch("fp4_gemm", lib.fp4_gemm_ws, dev, ctypes.byref(a), ctypes.byref(b), M, N, K,
            out.data_ptr(), t, out.stride(0), int(bool(accumulate)), _addr(ws), n)
    return out


@functools.lru_cache(maxsize=4096)
def _gemm_workspace(device, M, N, K, out_type, fmt_a, fmt_b, ld_a, ld_b):
    """Bytes of workspace that an FP8 product of these sizes can use."""
    a = Operand(fmt_a, None, ld_a, None, 0, 0, 1, None, SCALES_KMAJOR, GLOBAL_TENSOR)
    b = Operand(fmt_b, None, ld_b, None, 0, 0, 1, None, SCALES_KMAJOR, GLOBAL_TENSOR)
    with torch.cuda.device(device):
        return load_library().fp4_gemm_workspace(ctypes.byref(a), ctypes.byref(b), M, N, K,
                                                 out_type)


# ------------------------------------------------- attention on a cache --
HEAD_DIMS = (64, 128, 256)
_plan_changes = 0          # by selftest_set_attention_splits
CACHE_FORMATS = (FP8_E4M3, MXFP8, MXFP4, NVFP4, UE5M3)
PAIRINGS = {"half": 0, "interleaved": 1}


_BF16 = torch.bfloat16


def _heads(x, name):
    """(tokens, heads, head_dim, a Heads' fields) of a bf16 [tokens, heads, head_dim]
    tensor of any strides but the last."""
    if x.dtype is not _BF16 or x.dim() != 3:
        raise ValueError("%s must be a 3-D bfloat16 tensor [tokens, heads, head_dim]" % name)
    t, h, d = x.shape
    st, sh, sd = x.stride()
    if sd != 1:
        raise ValueError("%s: the elements of a head must be contiguous" % name)
    return t, h, d, (x.data_ptr(), st if t > 1 else 0, sh if h > 1 else 0, h)


def _heads_like(x, name, like, device):
    """A Heads' fields of a tensor that must have the shape of `like`, on its device."""
    t, h, d, fields = _heads(x, name)
    if (t, h, d) != like:
        raise ValueError("%s must be %s, not %s" % (name, list(like), [t, h, d]))
    if x.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, x.device, device))
    return fields


# several Heads in one buffer, which is cheaper than an object each: the fields of
# each, 32 bytes
_HEADS = [None] + [ctypes.c_int64 * (4 * n) for n in range(1, 7)]


def _index(x, name, n, device, dtype=torch.int64):
    if x.dtype is not dtype or x.shape != (n,) or x.device != device or (n > 1 and x.stride(0) != 1):
        raise ValueError("%s must be a contiguous %s [%d] tensor on %s" % (name, dtype, n, device))
    return x.data_ptr()


class QKNorm:
    """RMS norm of each head of queries and keys, a weight, and the rotation of
    their positions; either may be left out.

    q_weight, k_weight: [head_dim], both bfloat16 or both float32 (None: no norm).
    table: float32 [positions, rotary_dim], each row the cosines and then the sines
    of rotary_dim / 2 angles (`attention.rotary_table`; None: no rotation); the first
    rotary_dim elements of a head are turned.  style: which elements make a pair,
    "half" (i and i + rotary_dim / 2) or "interleaved" (2 i and 2 i + 1).
    """

    def __init__(self, q_weight=None, k_weight=None, table=None, eps=1e-6, style="half"):
        if style not in PAIRINGS:
            raise ValueError("style must be one of %s" % (tuple(PAIRINGS),))
        if (q_weight is None) != (k_weight is None):
            raise ValueError("q_weight and k_weight are given together or not at all")
        if q_weight is None and table is None:
            raise ValueError("neither weights nor a table")
        self.head_dim = None
        for w in (q_weight, k_weight) if q_weight is not None else ():
            if (w.dim() != 1 or w.dtype not in (torch.bfloat16, torch.float32) or w.dtype != q_weight.dtype
                    or w.shape != q_weight.shape or w.device != q_weight.device or not w.is_contiguous()):
                raise ValueError("the weights must be contiguous bfloat16 or float32 [head_dim] "
                                 "tensors, alike")
            self.head_dim = w.shape[0]
        if table is not None and (table.dtype != torch.float32 or table.dim() != 2 or not table.is_contiguous()
                                  or table.shape[1] % 2):
            raise ValueError("table must be a contiguous float32 [positions, rotary_dim] tensor")
        if table is not None and q_weight is not None and table.device != q_weight.device:
            raise ValueError("the weights and the table are on different devices")
        self.q_weight, self.k_weight, self.table = q_weight, k_weight, table
        self.eps, self.style = float(eps), style
        self.device = (table if q_weight is None else q_weight).device
        rows, dim = (0, 0) if table is None else table.shape
        self._desc = QKNormDesc(_addr(q_weight), _addr(k_weight),
                                int(q_weight is not None and q_weight.dtype == torch.float32), self.eps,
                                _addr(table), rows, dim, PAIRINGS[style])
        self._at = ctypes.addressof(self._desc)
        self._of = self._addresses()

    def _addresses(self):
        return _addr(self.q_weight), _addr(self.k_weight), _addr(self.table)

    def _positions(self, positions, tokens, head_dim, device):
        """The address of the positions of rows [tokens, heads, head_dim]; the descriptor
        (_at) is that of the tensors as they are from here on."""
        if self._addresses() != self._of:          # a tensor's .data has been replaced
            QKNorm.__init__(self, self.q_weight, self.k_weight, self.table, self.eps, self.style)
        if device != self.device or (self.head_dim is not None and head_dim != self.head_dim):
            raise ValueError("the norm is for heads of %s on %s" % (self.head_dim, self.device))
        if self.table is None:
            return None
        if positions is None:
            raise ValueError("a rotation needs positions")
        return _index(positions, "positions", tokens, device)


def _out_heads(out, like, x, name):
    """(tensor, a Heads' fields) of an output of x's kind: `out`, or a new dense one."""
    if out is not None:
        return out, _heads_like(out, name, like, x.device)
    t, h, d = like
    out = x.new_empty(like)
    return out, (out.data_ptr(), h * d, d, h)


def qk_norm_rope(norm: QKNorm, q, k, positions=None, out=(None, None)):
    """(q, k) normed and rotated, bf16 [tokens, heads, head_dim] each; either may
    be None.  The inputs may be parts of one projection's output.  positions:
    int64 [tokens], rows of the norm's table (one outside it gives NaN).
    out: tensors to write, of any strides but the last, for q and k (the inputs
    themselves, too)."""
    tokens = d = dev = None
    results, fields, at = [None, None], [], [None] * 4
    for i, x in enumerate((q, k)):
        if x is None:
            continue
        t, h, w, row = _heads(x, "qk"[i])
        if tokens is None:
            tokens, d, dev = t, w, x.device
        elif (t, w) != (tokens, d) or x.device != dev:
            raise ValueError("k must be [%d, heads, %d] on %s" % (tokens, d, dev))
        results[i], row_out = _out_heads(out[i], (t, h, w), x, "out[%d]" % i)
        at[i], at[2 + i] = 8 * len(fields), 8 * len(fields) + 32
        fields += row + row_out
    if not fields:
        raise ValueError("q and k are None")
    pos = norm._positions(positions, tokens, d, dev)
    buf = _HEADS[len(fields) // 4](*fields)
    b = ctypes.addressof(buf)
    _launch("fp4_qk_norm_rope", load_library().fp4_qk_norm_rope, dev, norm._at,
            None if q is None else b + at[0], None if k is None else b + at[1], pos, tokens, d,
            None if q is None else b + at[2], None if k is None else b + at[3])
    return results[0], results[1]


def qk_norm_rope_backward(norm: QKNorm, q, k, positions, dq, dk, out=(None, None), weight_grads=True):
    """The gradients (of q, of k, of q_weight, of k_weight) of `qk_norm_rope` at its
    inputs q and k, for dq and dk, those of its outputs (bf16, like them).  Weight
    gradients are float32 [head_dim], summed in a fixed order (None without a norm).
    weight_grads: False for none, or a dense float32 [2, head_dim] tensor to which q's
    and k's are added (its rows are what is returned)."""
    tokens = d = dev = None
    results, fields, at = [None, None], [], [None, None]
    for i, (x, dy) in enumerate(((q, dq), (k, dk))):
        if x is None:
            continue
        t, h, w, row = _heads(x, "qk"[i])
        if tokens is None:
            tokens, d, dev = t, w, x.device
        elif (t, w) != (tokens, d) or x.device != dev:
            raise ValueError("k must be [%d, heads, %d] on %s" % (tokens, d, dev))
        like = (t, h, w)
        row_dy = _heads_like(dy, "dq" if i == 0 else "dk", like, dev)
        results[i], row_out = _out_heads(out[i], like, x, "out[%d]" % i)
        at[i] = 8 * len(fields)
        fields += row + row_dy + row_out
    if not fields:
        raise ValueError("q and k are None")
    pos = norm._positions(positions, tokens, d, dev)
    wq = wk = ws = None
    n = 0
    add = isinstance(weight_grads, torch.Tensor)
    if (add or weight_grads) and norm.q_weight is not None:
        w = weight_grads if add else torch.empty((2, d), dtype=torch.float32, device=dev)
        if add and (w.dtype != torch.float32 or w.shape != (2, d) or not w.is_contiguous() or w.device != dev):
            raise ValueError("weight_grads must be a dense float32 [2, %d] tensor on %s" % (d, dev))
        wq, wk = w.unbind(0)
        wq, wk = wq if q is not None else None, wk if k is not None else None
        n = _norm_workspace(dev, d)
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
    buf = _HEADS[len(fields) // 4](*fields)
    b = ctypes.addressof(buf)
    (q0, q1, q2), (k0, k1, k2) = ((None,) * 3 if o is None else (b + o, b + o + 32, b + o + 64) for o in at)
    _launch("fp4_qk_norm_rope_backward", load_library().fp4_qk_norm_rope_backward, dev, norm._at, q0, k0,
            pos, tokens, d, q1, k1, q2, k2, _addr(wq), _addr(wk), int(add), _addr(ws), n)
    return results[0], results[1], wq, wk


@functools.lru_cache(maxsize=64)
def _norm_workspace(device, head_dim):
    with torch.cuda.device(device):
        return load_library().fp4_qk_norm_workspace(head_dim)


class KVCache:
    """A paged cache of keys and values in one of the library's formats.

    fmt: "fp8" (E4M3, a scale per 128 elements of a row), "mxfp8", "mxfp4" (per 32),
    "nvfp4" or "ue5m3" (per 16, with tensor scales).  k_codes, v_codes: uint8
    [pages, heads, page_size, bytes of a row]; k_scales, v_scales: uint8 [pages,
    heads, blocks of a row, page_size]; V's strides those of K, and the last
    dimension contiguous.  amax: float32 [2] on the device, of K and of V, from which
    the tensor scales of "nvfp4" and "ue5m3" are made (fixed while the cache is in
    use); target: their T.  Slot s is place s % page_size of page s // page_size.
    """

    def __init__(self, fmt, k_codes, k_scales, v_codes, v_scales, amax=None, target=448.0):
        f = _fmt(fmt)
        if f not in CACHE_FORMATS:
            raise ValueError("a cache is 'fp8', 'mxfp8', 'mxfp4', 'nvfp4' or 'ue5m3'")
        if k_codes.dim() != 4 or k_scales.dim() != 4:
            raise ValueError("codes must be [pages, heads, page_size, bytes] and scales [pages, heads, "
                             "blocks, page_size]")
        pages, heads, page, width = k_codes.shape
        d = width if f in (FP8_E4M3, MXFP8) else 2 * width
        if d not in HEAD_DIMS:
            raise ValueError("head_dim must be one of %s, not %d" % (HEAD_DIMS, d))
        blocks = -(-d // BLOCK_LEN[f])
        for name, t, shape, strides in (
                ("k_codes", k_codes, k_codes.shape, k_codes), ("v_codes", v_codes, k_codes.shape, k_codes),
                ("k_scales", k_scales, (pages, heads, blocks, page), k_scales),
                ("v_scales", v_scales, (pages, heads, blocks, page), k_scales)):
            if (t.dtype != torch.uint8 or tuple(t.shape) != tuple(shape) or t.stride(3) != 1
                    or t.device != k_codes.device          # (the stride of a single entry means nothing)
                    or any(a != b for n, a, b in zip(shape, t.stride(), strides.stride()) if n > 1)):
                raise ValueError("%s must be uint8 %s on %s, its last dimension contiguous and K's and "
                                 "V's strides alike" % (name, tuple(shape), k_codes.device))
        if f in (NVFP4, UE5M3):
            if (amax is None or amax.dtype != torch.float32 or amax.shape != (2,) or not amax.is_contiguous()
                    or amax.device != k_codes.device):
                raise ValueError("amax must be a contiguous float32 [2] tensor on %s" % k_codes.device)
        else:
            amax = None
        self.fmt, self.heads, self.head_dim, self.pages, self.page_size = f, heads, d, pages, page
        self.k_codes, self.k_scales, self.v_codes, self.v_scales = k_codes, k_scales, v_codes, v_scales
        self.amax, self.target, self.device = amax, float(target), k_codes.device

        def strides(t, row):          # of a dimension of one entry: any that is valid
            return [s if n > 1 else row for s, n in zip(t.stride()[:3], t.shape)]

        self._desc = KVCacheDesc(f, heads, d, page, pages, k_codes.data_ptr(), k_scales.data_ptr(),
                                 v_codes.data_ptr(), v_scales.data_ptr(), *strides(k_codes, width),
                                 *strides(k_scales, page), _addr(amax), self.target)
        self._at = ctypes.addressof(self._desc)
        self._sizes = {}

    def _workspace(self, heads, requests, width):
        """Bytes of workspace that attention of these sizes can use."""
        key = heads, requests, width, _plan_changes
        size = self._sizes.get(key)
        if size is None:
            if len(self._sizes) > 4096:
                self._sizes.clear()
            with torch.cuda.device(self.device):
                size = load_library().fp4_attention_workspace(self._at, heads, requests, width)
            self._sizes[key] = size
        return size

    @classmethod
    def empty(cls, pages, page_size, heads, head_dim, fmt="mxfp8", device="cuda", amax=None, target=448.0):
        """A cache whose pages are yet to be written."""
        f = _fmt(fmt)
        if f not in CACHE_FORMATS:
            raise ValueError("a cache is 'fp8', 'mxfp8', 'mxfp4', 'nvfp4' or 'ue5m3'")
        if head_dim not in HEAD_DIMS:
            raise ValueError("head_dim must be one of %s, not %d" % (HEAD_DIMS, head_dim))
        width = head_dim if f in (FP8_E4M3, MXFP8) else head_dim // 2
        codes = (torch.empty((pages, heads, page_size, width), dtype=torch.uint8, device=device)
                 for _ in range(2))
        scales = (torch.empty((pages, heads, -(-head_dim // BLOCK_LEN[f]), page_size), dtype=torch.uint8,
                              device=device) for _ in range(2))
        k, v = codes
        ks, vs = scales
        return cls(f, k, ks, v, vs, amax, target)


def kv_cache_write(cache: KVCache, k, v, slots, q=None, norm: QKNorm = None, positions=None, q_out=None):
    """Encode the rows k and v (bf16 [tokens, heads, head_dim]) of new tokens into
    their slots (int64 [tokens]; a negative one, or one behind the last page, is not
    written; the others are distinct).

    norm: k goes through it first, in the same pass, without a rounding to bf16 between; with
    q, q does too and comes back (bf16; into q_out, if given).  positions as in
    `qk_norm_rope`.  Returns q's result, or None.
    """
    tokens, h, d, fields = _heads(k, "k")
    dev = cache.device
    if (h, d) != (cache.heads, cache.head_dim) or k.device != dev:
        raise ValueError("k must be [tokens, %d, %d] on %s" % (cache.heads, cache.head_dim, dev))
    fields += _heads_like(v, "v", (tokens, h, d), dev)
    at = _index(slots, "slots", tokens, dev)
    pos = where = q_at = out_at = None
    if norm is not None:
        pos = norm._positions(positions, tokens, d, dev)
        where = norm._at
    if q is not None:
        if norm is None:
            raise ValueError("q needs a norm")
        t, hq, dq, row = _heads(q, "q")
        if (t, dq) != (tokens, d) or q.device != dev:
            raise ValueError("q must be [%d, heads, %d] on %s" % (tokens, d, dev))
        q_out, row_out = _out_heads(q_out, (t, hq, d), q, "q_out")
        fields += row + row_out
    buf = _HEADS[len(fields) // 4](*fields)
    b = ctypes.addressof(buf)
    if q is not None:
        q_at, out_at = b + 64, b + 96
    _launch("fp4_kv_cache_write", load_library().fp4_kv_cache_write, dev, cache._at, b, b + 32, at, tokens,
            where, pos, q_at, out_at)
    return q_out if q is not None else None


def kv_cache_read(cache: KVCache, slots, out_dtype=torch.bfloat16):
    """(k, v): the values of slots (int64 [n], any order), [n, heads, head_dim] each,
    bf16 or fp32; zeros for what is no slot of the cache."""
    if out_dtype not in OUT_TYPES:
        raise ValueError("out_dtype must be torch.float32 or torch.bfloat16")
    if slots.dim() != 1:
        raise ValueError("slots must be an int64 [n] tensor")
    n = slots.shape[0]
    at = _index(slots, "slots", n, cache.device)
    shape = (n, cache.heads, cache.head_dim)
    k = torch.empty(shape, dtype=out_dtype, device=cache.device)
    v = k.new_empty(shape)
    _launch("fp4_kv_cache_read", load_library().fp4_kv_cache_read, cache.device, cache._at, at, n,
            k.data_ptr(), v.data_ptr(), int(out_dtype == torch.float32))
    return k, v


def attention_decode(q, cache: KVCache, page_table, lens, scale=None, out=None, out_dtype=torch.bfloat16,
                     return_lse=False):
    """Attention of one new token per request over its cached tokens (its own
    written first): q bf16 [requests, heads, head_dim], heads a multiple of the
    cache's; page_table int32 [requests, width], entry i the page of tokens
    i * page_size ..; lens int32 [requests].  scale: 1 / sqrt(head_dim) if None.

    Returns [requests, heads, head_dim] (bf16, or float32 by out_dtype or `out`, which
    is dense); zeros where a request has no tokens.  With return_lse also the float32
    [requests, heads] log of each softmax's denominator (-inf without tokens).  Tokens
    on a page that the cache does not have are left out.
    """
    n, heads, d, fields = _heads(q, "q")
    dev = cache.device
    if d != cache.head_dim or q.device != dev:
        raise ValueError("q must be [requests, heads, %d] on %s" % (cache.head_dim, dev))
    if (page_table.dtype is not torch.int32 or page_table.dim() != 2 or page_table.device != dev
            or page_table.shape[0] != n or (page_table.shape[1] > 1 and page_table.stride(1) != 1)):
        raise ValueError("page_table must be an int32 [%d, width] tensor on %s, contiguous along its rows"
                         % (n, dev))
    at = _index(lens, "lens", n, dev, torch.int32)
    if out is None:
        out = (q.new_empty((n, heads, d)) if out_dtype is _BF16
               else torch.empty((n, heads, d), dtype=out_dtype, device=dev))
    elif out.shape != q.shape or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous tensor of q's shape on its device")
    if out.dtype not in OUT_TYPES:
        raise ValueError("the output is float32 or bfloat16")
    lse = torch.empty((n, heads), dtype=torch.float32, device=dev) if return_lse else None
    width = page_table.shape[1]
    size = cache._workspace(heads, n, width)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    buf = _HEADS[1](*fields)
    _launch("fp4_attention_decode", load_library().fp4_attention_decode, dev, cache._at, ctypes.addressof(buf),
            page_table.data_ptr(), page_table.stride(0) if n > 1 else 0, width, at, n,
            d ** -0.5 if scale is None else float(scale), out.data_ptr(), OUT_TYPES[out.dtype], _addr(lse),
            _addr(ws), size)
    return (out, lse) if return_lse else out


# ------------------------------------------------------------- self-test --
SWEEPS = {"e2m1_rne": 0, "e4m3_scale": 1, "ue5m3_scale": 2, "e2m1_sr": 3, "e4m3_elem": 4}


def selftest_sweep(kind, thresholds, device="cuda"):
    """Run one of the library's conversions over its whole input domain
    against the step function `thresholds` (ascending fp32 bit patterns,
    uint32): returns (mismatches, smallest mismatching pattern or None,
    inputs checked)."""
    if len(thresholds) and int(max(thresholds)) >= 2 ** 31:
        raise ValueError("thresholds are magnitudes: patterns below 2^31")
    thr = torch.tensor([int(t) for t in thresholds], dtype=torch.int32).to(device)
    res = torch.empty(3, dtype=torch.int64, device=device)
    lib = load_library()
    _check(lib.fp4_selftest_sweep(SWEEPS[kind], _ptr(thr), thr.numel(), _ptr(res),
                                  _stream(res.device)), "fp4_selftest_sweep")
    bad, first, checked = (int(v) & (2 ** 64 - 1) for v in res.cpu().tolist())
    return bad, (None if bad == 0 else first), checked


def selftest_gemm_decode(fmt, device="cuda"):
    """The GEMM's operand decode of every (scale code, E2M1 code) pair:
    uint16 fp16 patterns [256, 4, 16] (see fp4_selftest_gemm_decode)."""
    out = torch.empty((256, 4, 16), dtype=torch.int16, device=device)
    lib = load_library()
    _check(lib.fp4_selftest_gemm_decode(_fmt(fmt), _ptr(out), _stream(out.device)),
           "fp4_selftest_gemm_decode")
    return out.cpu().numpy().view("uint16")


def selftest_set_geometry(max_workgroups=0, gemm_tile_rows=0):
    """Launch-geometry controls for race guards (0, 0: the defaults)."""
    _check(load_library().fp4_selftest_set_geometry(int(max_workgroups), int(gemm_tile_rows)),
           "fp4_selftest_set_geometry")


def selftest_set_fp8_plan(tile_rows=0, splits=1):
    """The kernel of the FP8 products (0: chosen by size)."""
    _check(load_library().fp4_selftest_set_fp8_plan(int(tile_rows), int(splits)),
           "fp4_selftest_set_fp8_plan")
    _gemm_workspace.cache_clear()


def selftest_set_attention_splits(splits=0):
    """Parts that attention shares a request's tokens among (0: chosen by size)."""
    global _plan_changes
    _check(load_library().fp4_selftest_set_attention_splits(int(splits)),
           "fp4_selftest_set_attention_splits")
    _plan_changes += 1
