"""fp4_selftest_set_fp8_plan: what it takes, and that a product which the asked
kernel cannot run fails, without any device work, and runs on no other one."""
import ctypes
import os

import pytest

from fp4_block_scaled_x16_amd import api

FAKE = ctypes.c_void_p(0x10000)
DEVICE = 4


@pytest.fixture
def lib():
    if not os.path.exists(api.LIB_PATH):
        pytest.skip("library not built")
    lib = api.load_library()
    yield lib
    assert lib.fp4_selftest_set_fp8_plan(0, 1) == 0


def op(ld=1024):
    return api.Operand(api.FP8_E4M3, 0x10000, ld, 0x20000, 0, 4096, 1, None, 2, 0)


def gemm(lib, M, N=300, K=1000, t=0, ld=1024, ws=None, size=0):
    a = op(ld)
    return lib.fp4_gemm_ws(ctypes.byref(a), ctypes.byref(a), M, N, K, FAKE, t, N, 0, ws, size, None)


def needs(lib, M, N=300, K=1000, t=0, ld=1024):
    a = op(ld)
    return lib.fp4_gemm_workspace(ctypes.byref(a), ctypes.byref(a), M, N, K, t)


def test_values(lib):
    for rows, splits in ((16, 1), (64, 3), (128, 16), (192, 1), (256, 2), (0, 1)):
        assert lib.fp4_selftest_set_fp8_plan(rows, splits) == 0
    for rows, splits in ((1, 1), (32, 1), (-1, 1), (512, 1), (64, 0), (0, -1)):
        assert lib.fp4_selftest_set_fp8_plan(rows, splits) == 1


@pytest.mark.parametrize("rows,splits,kw", [
    (16, 1, dict(M=17)), (16, 2, dict(M=1)),                      # few rows, K not shared
    (192, 1, dict(M=300, t=1)),                                   # a bf16 D
    (192, 1, dict(M=300, K=0)), (256, 1, dict(M=300, K=0)),
    (256, 1, dict(M=300, ld=1 << 23)), (192, 1, dict(M=300, ld=1 << 23)),
    (64, 9, dict(M=40)), (256, 9, dict(M=40, t=1)),               # 8 blocks of K
    (64, 3, dict(M=40)), (128, 2, dict(M=40, ws=FAKE, size=2 * 40 * 300 * 4 - 4))])
def test_products_that_cannot_run(lib, rows, splits, kw):
    assert lib.fp4_selftest_set_fp8_plan(rows, splits) == 0
    assert gemm(lib, **kw) == DEVICE
    assert b"invalid" in lib.fp4_last_error()


def test_workspace(lib):
    for rows, splits in ((64, 3), (128, 8), (256, 2)):
        assert lib.fp4_selftest_set_fp8_plan(rows, splits) == 0
        assert needs(lib, 40, 299) == splits * 40 * 300 * 4       # rows of the parts: 4 floats at a time
    assert lib.fp4_selftest_set_fp8_plan(64, 1) == 0 and needs(lib, 40) == 0
    assert lib.fp4_selftest_set_fp8_plan(64, 9) == 0 and needs(lib, 40) == 0
