"""Refusals of the FP8 block-128 calls, in the C ABI and in the Python
binding: everything here is rejected on the host, before any HIP call."""
import ctypes

import pytest
import torch

from fp4_block_scaled_x16_amd import api
from test_abi import _err, desc, dual, lib, quant  # noqa: F401 (lib: fixture)

FAKE = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)
F8, F8G = api.FP8_E4M3, api.FP8_E5M2


def fdesc(**kw):
    return desc(**dict(dict(format=F8, scale_layout=2), **kw))


@pytest.mark.parametrize("kw,rows,cols,status", [
    (dict(block=1), 32, 64, 3),               # 16x16 blocks
    (dict(block=3), 32, 64, 1),
    (dict(orient=2), 32, 64, 1),
    (dict(round=1), 32, 64, 3),               # nearest even only
    (dict(round=4), 32, 64, 1),
    (dict(scale_layout=0), 32, 64, 3),        # KMAJOR only
    (dict(scale_layout=1), 32, 64, 3),
    (dict(rht=1), 32, 64, 3),
    (dict(amax_given=1), 32, 64, 3),
    (dict(emit_transpose=1, block=2), 32, 64, 3),
    (dict(scale_round=3), 32, 64, 1),
    (dict(global_scope=1), 32, 64, 3),
    (dict(global_scope=2), 32, 64, 1),
    (dict(count_level=2), 32, 64, 1),
    (dict(), -1, 64, 2),
    (dict(), 32, -8, 2),
    (dict(), 1 << 31, 64, 2),
    (dict(format=F8G, block=1), 32, 64, 3),
])
def test_quantize_rejects(lib, kw, rows, cols, status):
    assert quant(lib, fdesc(**kw), rows, cols) == status
    assert _err(lib)


def test_quantize_rejects_pointers(lib):
    d = fdesc()
    assert quant(lib, d, x=None) == 1
    assert quant(lib, d, x=ODD) == 1
    assert quant(lib, d, ld=60) == 1
    assert quant(lib, d, ld=68) == 1
    assert quant(lib, d, codes=None) == 1
    assert quant(lib, d, scales=None) == 1
    assert quant(lib, d, codes=ODD) == 1
    assert quant(lib, d, scales=ODD) == 1
    assert quant(lib, d, codes_t=FAKE) == 3            # the dual quantizer's
    assert quant(lib, fdesc(), rows=0) == 0            # empty: nothing to do
    assert quant(lib, fdesc(), cols=0) == 0


@pytest.mark.parametrize("rkw,ckw,status", [
    (dict(), dict(orient=1, format=F8G), 3),
    (dict(), dict(orient=1, format=0, scale_layout=0), 3),
    (dict(block=2), dict(orient=1), 3),
    (dict(), dict(), 3),
    (dict(orient=1), dict(orient=1), 3),
    (dict(), dict(orient=1, count_level=1), 3),
    (dict(round=1), dict(orient=1), 3),
])
def test_quantize_dual_rejects(lib, rkw, ckw, status):
    assert dual(lib, fdesc(**rkw), fdesc(**ckw)) == status
    assert _err(lib)


def test_quantize_dual_rejects_pointers(lib):
    r, c = fdesc(), fdesc(orient=1)
    assert dual(lib, r, c, x=None) == 1
    for name in ("codes", "scales", "codes_t", "scales_t"):
        assert dual(lib, r, c, **{name: None}) == 1
        assert dual(lib, r, c, **{name: ODD}) == 1
    assert dual(lib, r, c, rows=0) == 0


def test_other_formats_do_not_take_fp8s_layouts(lib):
    assert quant(lib, desc(scale_layout=2)) == 1
    assert quant(lib, desc(block=2)) == 1
    assert quant(lib, desc(format=4)) == 1


def test_dequantize_and_requantize_reject(lib):
    deq = lib.fp4_dequantize
    assert deq(F8, 0, 0, FAKE, FAKE, None, 0, 32, 64, FAKE, 1, None) == 3     # layout
    assert deq(F8, 1, 2, FAKE, FAKE, None, 0, 32, 64, FAKE, 1, None) == 3     # block
    assert deq(F8, 0, 2, FAKE, FAKE, None, 1, 32, 64, FAKE, 1, None) == 3     # scope
    assert deq(F8, 0, 2, FAKE, ODD, None, 0, 32, 64, FAKE, 1, None) == 1
    assert deq(F8, 0, 2, FAKE, FAKE, None, 0, 32, 64, ODD, 1, None) == 1
    assert deq(F8, 0, 2, FAKE, FAKE, None, 0, -1, 64, FAKE, 1, None) == 2
    assert deq(F8, 0, 2, None, None, None, 0, 0, 64, None, 1, None) == 0
    req = lib.fp4_requantize_t
    assert req(3, FAKE, FAKE, 32, 64, FAKE, FAKE, None) == 3                  # MXFP8
    assert req(9, FAKE, FAKE, 32, 64, FAKE, FAKE, None) == 3
    assert req(F8, None, FAKE, 32, 64, FAKE, FAKE, None) == 1
    assert req(F8, FAKE, ODD, 32, 64, FAKE, FAKE, None) == 1
    assert req(F8, FAKE, FAKE, 32, 64, None, FAKE, None) == 1
    assert req(F8, FAKE, FAKE, 32, 64, FAKE, ODD, None) == 1
    assert req(F8, FAKE, FAKE, 32, -1, FAKE, FAKE, None) == 2
    assert req(F8, None, None, 32, 0, None, None, None) == 0


def test_act_calls_reject(lib):
    f = lib.fp4_act_quantize

    def fwd(act=0, h=FAKE, rows=4, cols=64, ld=128, qa=FAKE, sa=FAKE, a=None, lda=0, qh=FAKE, sh=FAKE):
        return f(act, h, rows, cols, ld, qa, sa, a, lda, qh, sh, None)

    assert fwd(act=2) == 1
    assert fwd(cols=60, ld=128) == 2                    # SwiGLU halves start 16-byte aligned
    assert fwd(cols=-8) == 2
    assert fwd(cols=1 << 30) == 2
    assert fwd(h=None) == 1
    assert fwd(h=ODD) == 1
    assert fwd(ld=64) == 1                              # h has 2F columns
    assert fwd(ld=132) == 1
    assert fwd(sa=None) == 1                            # a pair is whole or absent
    assert fwd(qh=None) == 1
    assert fwd(qa=ODD) == 1
    assert fwd(a=ODD, lda=64) == 1
    assert fwd(a=FAKE, lda=60) == 1
    assert fwd(a=FAKE, lda=68) == 1
    assert fwd(qa=None, sa=None, qh=None, sh=None) == 1  # nothing to write
    assert fwd(rows=0, h=None) == 0

    g = lib.fp4_act_backward

    def bwd(act=0, qh=FAKE, sh=FAKE, da=FAKE, rows=4, cols=64, ld=64, fmt=F8, o=(FAKE,) * 6,
            dh=None, ldh=0, a=None, lda=0):
        return g(act, qh, sh, da, rows, cols, ld, fmt, *o, dh, ldh, a, lda, None)

    assert bwd(act=-1) == 1
    assert bwd(fmt=3) == 3
    assert bwd(cols=60) == 2
    assert bwd(qh=None) == 1
    assert bwd(sh=ODD) == 1
    assert bwd(da=None) == 1
    assert bwd(ld=60) == 1
    assert bwd(o=(FAKE, None) + (FAKE,) * 4) == 1
    assert bwd(o=(FAKE,) * 3 + (None,) + (FAKE,) * 2) == 1
    assert bwd(o=(FAKE,) * 4 + (ODD, FAKE)) == 1
    assert bwd(o=(None,) * 6) == 1
    assert bwd(o=(None,) * 6, dh=FAKE, ldh=64) == 1     # dh has 2F columns
    assert bwd(o=(None,) * 6, a=ODD, lda=64) == 1
    assert bwd(rows=0, da=None, qh=None) == 0


def op(fmt=F8, codes=0x10000, ld=128, scales=0x20000, kblk=16, layout=2, rg=1, scope=0):
    return api.Operand(fmt, codes, ld, scales, 0, kblk, rg, None, layout, scope)


@pytest.mark.parametrize("a,b,M,N,K,status", [
    (op(), op(0, layout=0), 16, 16, 128, 3),           # FP8 with another format
    (op(3), op(), 16, 16, 128, 3),
    (op(), op(F8G), 16, 16, 128, 3),                   # E5M2 is operand A's
    (op(), op(), -1, 16, 128, 2),
    (op(), op(), 1 << 31, 16, 128, 2),
    (op(layout=1), op(), 16, 16, 128, 3),
    (op(), op(rg=16), 16, 16, 128, 3),
    (op(scope=1), op(), 16, 16, 128, 3),
    (op(codes=0), op(), 16, 16, 128, 1),
    (op(), op(scales=0), 16, 16, 128, 1),
    (op(codes=0x10008), op(), 16, 16, 128, 1),
    (op(scales=0x20004), op(), 16, 16, 128, 1),
    (op(ld=128), op(ld=256), 16, 16, 129, 1),          # rows shorter than whole blocks
    (op(ld=136), op(), 16, 16, 128, 1),                # ld % 16
    (op(kblk=24), op(), 16, 16, 128, 1),
    (op(kblk=16), op(), 17, 16, 128, 1),               # scale pitch below the rows
])
def test_gemm_rejects(lib, a, b, M, N, K, status):
    assert lib.fp4_gemm(ctypes.byref(a), ctypes.byref(b), M, N, K, FAKE, 0, N, 0, None) == status
    assert _err(lib)


def test_gemm_rejects_output(lib):
    a = op()

    def call(D=FAKE, t=0, ldd=16, M=16):
        return lib.fp4_gemm(ctypes.byref(a), ctypes.byref(a), M, 16, 128, D, t, ldd, 0, None)

    assert call(D=None) == 1
    assert call(t=2) == 1
    assert call(ldd=15) == 1
    assert call(D=ctypes.c_void_p(0x10002)) == 1
    assert call(D=ctypes.c_void_p(0x10001), t=1) == 1
    assert call(M=0, D=None) == 0


def matrix(rows=4, cols=130, fmt="fp8"):
    kb = -(-cols // 128)
    return api.fp8_matrix(torch.zeros((rows, 128 * kb), dtype=torch.uint8),
                          torch.zeros((kb, -(-rows // 16) * 16), dtype=torch.uint8), rows, cols, fmt)


def test_binding_rejects():
    codes, scales = torch.zeros((4, 256), dtype=torch.uint8), torch.zeros((2, 16), dtype=torch.uint8)
    assert api.fp8_matrix(codes, scales, 4, 130).operand().scale_stride_kblk == 16
    assert api.fp8_matrix(codes.view(torch.float8_e4m3fn), scales, 4, 200).codes.dtype == torch.uint8
    for c, s, rows, cols, fmt in ((codes[:, :130], scales, 4, 130, "fp8"),
                                  (codes, scales, 5, 130, "fp8"),
                                  (codes, scales, 4, 257, "fp8"),
                                  (codes, scales[:1], 4, 130, "fp8"),
                                  (codes, scales[:, :4], 4, 130, "fp8"),
                                  (codes, scales, 4, 130, "mxfp8")):
        with pytest.raises(ValueError):
            api.fp8_matrix(c, s, rows, cols, fmt)
    x = torch.zeros((128, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.quantize(x, "fp8", block="3d")
    with pytest.raises(ValueError):
        api.quantize(x, "fp8", orient="both")
    with pytest.raises(ValueError):
        api.quantize_dual(x, "nvfp4", block="2d")
    with pytest.raises(ValueError):
        api.requantize_t(api.Quantized(api.MXFP8, 0, 32, 32, None, None, None, None))
    with pytest.raises(ValueError):
        matrix().operand(transposed=True)
    for call in (lambda: api.act_quantize(x.float()), lambda: api.act_quantize(x, "gelu"),
                 lambda: api.act_quantize(x, a="fp4"), lambda: api.act_quantize(x[:, :127]),
                 lambda: api.act_quantize(x.t()),
                 lambda: api.act_backward(matrix(), x, "relu2"),
                 lambda: api.act_backward(matrix(128, 128), x, "swiglu"),
                 lambda: api.act_backward(matrix(128, 128, "fp8_e5m2"), x, "relu2"),
                 lambda: api.act_backward(matrix(128, 128), x, "relu2", fmt="nvfp4"),
                 lambda: api.act_backward(matrix(128, 128), x, "relu2", out="fp32"),
                 lambda: api.act_backward(matrix(128, 128), x.half(), "relu2")):
        with pytest.raises(ValueError):
            call()
    a, b = matrix(4, 130).operand(), matrix(6, 130).operand()
    for M, N, K in ((5, 6, 130), (4, 7, 130), (4, 6, 128), (4, 6, 256)):
        with pytest.raises(ValueError):
            api.gemm(a, b, M, N, K, out=torch.zeros((8, 8)))
    with pytest.raises(ValueError):
        api.gemm(a, b, 4, 6, 130, out=torch.zeros((4, 5)))


def test_binding_rejects_other_devices():
    """Tensors that a kernel would reach at another device's address."""
    x = torch.zeros((128, 128), dtype=torch.bfloat16)
    for counters in (torch.zeros(5, dtype=torch.int64, device="meta"), torch.zeros(4, dtype=torch.int64),
                     torch.zeros(5, dtype=torch.int32), torch.zeros(10, dtype=torch.int64)[::2]):
        for call in (api.quantize, api.quantize_dual):
            with pytest.raises(ValueError, match="counters"):
                call(x, "fp8", counters=counters)
    with pytest.raises(ValueError, match="different devices"):
        api.dequantize(matrix(), out=torch.empty((4, 130), device="meta"))
    with pytest.raises(ValueError, match="different devices"):
        api.act_backward(matrix(128, 128), x.to("meta"), "relu2")
    a = matrix().operand()
    with pytest.raises(ValueError, match="different devices"):
        api.gemm(a, a, 4, 4, 130, out=torch.empty((4, 4), device="meta"))
    for call in (lambda: api.quantize(x, "fp8"), lambda: api.act_quantize(x, "relu2"),
                 lambda: api.requantize_t(matrix()), lambda: api.dequantize(matrix())):
        with pytest.raises(ValueError, match="on the GPU"):
            call()
