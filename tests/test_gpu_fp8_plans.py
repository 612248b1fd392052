"""Every kernel of the FP8 product, alone and with K shared, at sizes around its
tiles' edges and from one block of K to many, whichever kernel the cost model
would choose there: against 64-bit products (the bounds are those of
test_gpu_fp8_gemm.py), with E5M2 and E4M3 operands, both output types, written
and added to."""
import contextlib
import functools

import numpy as np
import pytest
import torch

from fp4_block_scaled_x16_amd import api
from fp8_check import DEV, as64, bf16, spread
from oracle import fp8
from test_gpu_fp8_gemm import TOL, close, operands, product

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# (rows of a tile, workgroups that share its K); 16: the kernel for few rows
PLANS = [(16, 1), (64, 1), (64, 3), (128, 1), (128, 3), (192, 1), (192, 3), (256, 1), (256, 3)]
# output sizes around the edges of the kernel's tiles
SIZES = {16: [(1, 33), (16, 270)], 64: [(1, 1), (65, 130), (200, 257)], 128: [(2, 129), (130, 128), (300, 517)],
         192: [(3, 257), (193, 256), (400, 520)], 256: [(1, 256), (257, 258), (515, 770)]}


@contextlib.contextmanager
def plan(rows, splits):
    api.selftest_set_fp8_plan(rows, splits)
    try:
        yield
    finally:
        api.selftest_set_fp8_plan()


def out_types(rows):
    return [F32] if rows == 192 else [F32, BF]


@functools.lru_cache(maxsize=4)
def case(M, N, K, fa):
    a, b = operands(M, N, K, fa, "1d" if fa == "fp8_e5m2" else "2d", 11)
    return a, b, product(a, b)


@pytest.mark.parametrize("fa", ["fp8", "fp8_e5m2"])
@pytest.mark.parametrize("rows,splits,K", [(r, s, K) for r, s in PLANS for K in (128, 250, 384, 870, 5120)
                                           if s <= -(-K // 128)])
def test_products(rows, splits, K, fa):
    """1, 2, 3, 7 and 40 blocks of K; aligned outputs and odd views, beside which
    nothing moves; the same bits each time."""
    for M, N in SIZES[rows]:
        a, b, (ref, bound, cut) = case(M, N, K, fa)
        for out in out_types(rows):
            with plan(rows, splits):
                d = api.gemm(a.operand(), b.operand(), M, N, K, out_dtype=out)
                close(d, ref, bound, cut)
                assert torch.equal(d, api.gemm(a.operand(), b.operand(), M, N, K, out_dtype=out))
                for off, pitch in ((0, -(-N // 8) * 8), (1, N + 3)):
                    big = torch.full((M + 2, off + pitch), 0.5, dtype=out, device=DEV)
                    view = big[1:M + 1, off:off + N]
                    api.gemm(a.operand(), b.operand(), M, N, K, out=view)
                    assert torch.equal(view, d)
                    view.fill_(0.5)
                    api.gemm(a.operand(), b.operand(), M, N, K, out=view, accumulate=True)
                    close(view, ref + 0.5, bound + 0.5 * 2.0 ** -24 / TOL, cut)
                    view.fill_(0.5)
                    assert bool((big == 0.5).all())


@pytest.mark.parametrize("M", [47, 48, 64, 80, 191, 240, 256, 272, 383, 384, 385])
def test_scales_of_three_rows(M):
    """192 rows a tile: a lane's three scales come from a word that is read from
    before the end of a block's scales and shifted; M a multiple of 16 (the
    scales end with the rows) with each remainder of 3 (shifts of 8, 24 and 16
    bits), and others.  Neighbouring rows have different scales."""
    N, K = 260, 384
    for fa in ("fp8", "fp8_e5m2"):
        a, b = operands(M, N, K, fa, "1d", 5)
        for splits in (1, 2):
            with plan(192, splits):
                close(api.gemm(a.operand(), b.operand(), M, N, K), *product(a, b))


@pytest.mark.parametrize("fa", ["fp8", "fp8_e5m2"])
@pytest.mark.parametrize("rows,splits", PLANS)
def test_exact_sums(rows, splits, fa):
    """Small whole numbers: every product and partial sum is exact."""
    rng = np.random.default_rng(5)
    K = 1000
    for M, N in SIZES[rows]:
        x, w = rng.integers(-8, 9, (M, K)), rng.integers(-8, 9, (N, K))
        if fa == "fp8_e5m2":
            x = np.where(np.abs(x) == 7, 6, np.where(np.abs(x) == 5, 4, x))    # 3 significant bits
        a, b = api.quantize(bf16(x).to(DEV), fa), api.quantize(bf16(w).to(DEV), "fp8")
        want = torch.from_numpy((x @ w.T).astype(np.float32))
        for out in out_types(rows):
            with plan(rows, splits):
                d = api.gemm(a.operand(), b.operand(), M, N, K, out_dtype=out)
                assert torch.equal(d.cpu(), want.to(out))
                api.gemm(a.operand(), b.operand(), M, N, K, out=d.zero_(), accumulate=True)
                assert torch.equal(d.cpu(), want.to(out))


@pytest.mark.parametrize("rows,splits,blocks", [(r, s, n) for r, s in PLANS for n in (1, 2, 3) if s <= n])
def test_every_code_and_scale(rows, splits, blocks):
    """A's rows pick single columns of B, so D is B's values themselves, for every
    code at every scale whose values are normal bf16 numbers (448 * 2^118 and
    2^-9 * 2^-117 among them): an odd number of blocks is where the large tiles
    multiply their last block a second time, under scales that make it zero."""
    K, N, M = 128 * blocks, 236, {16: 16, 64: 60, 128: 130, 192: 200, 256: 300}[rows]
    codes = np.tile((np.arange(K) * 37 % 256).astype(np.uint8), (N, 1))       # 37: odd, so all 256 codes in 2 blocks
    codes[(codes & 0x7F) == 0x7F] = 0                                         # NaN
    scales = np.zeros((blocks, 240), np.uint8)
    scales[:, :N] = np.arange(10, 246)                                        # 2^-117 .. 2^118
    b = api.fp8_matrix(torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV), N, K)
    v = fp8.values(codes, scales, "fp8")
    for fa, one in (("fp8", 0x38), ("fp8_e5m2", 0x3C)):
        for first in range(0, K, M):
            n = min(M, K - first)
            ac = np.zeros((M, K), np.uint8)
            ac[np.arange(n), first + np.arange(n)] = one
            a = api.fp8_matrix(torch.from_numpy(ac).to(DEV), torch.full(
                (blocks, -(-M // 16) * 16), 127, dtype=torch.uint8, device=DEV), M, K, fa)
            want = np.zeros((M, N))
            want[:n] = v[:, first:first + n].T
            for out in out_types(rows):
                with plan(rows, splits):
                    d = api.gemm(a.operand(), b.operand(), M, N, K, out_dtype=out)
                    assert np.array_equal(as64(d), want)
                    api.gemm(a.operand(), b.operand(), M, N, K, out=d.zero_(), accumulate=True)
                    assert np.array_equal(as64(d), want)


@pytest.mark.parametrize("fa,code", [("fp8", 0x7F), ("fp8_e5m2", 0x7E), ("fp8_e5m2", 0x7C), ("fp8_e5m2", 0xFC)])
@pytest.mark.parametrize("rows,splits", PLANS)
def test_non_finite_codes(rows, splits, fa, code):
    """NaN and infinite elements in the first and the last block: their rows and
    columns, and no others, are not finite."""
    M, N = {16: 5, 64: 70, 128: 140, 192: 200, 256: 300}[rows], 270
    for K in (384, 512):
        a, b = operands(M, N, K, fa, "1d", 9)
        a.codes[1, 17] = code
        a.codes[M - 1, K - 3] = code
        b.codes[3, K - 2] = 0xFF
        b.codes[N - 1, 5] = 0x7F
        keep = np.ones((M, N), bool)
        keep[[1, M - 1]] = False
        keep[:, [3, N - 1]] = False
        for out in out_types(rows):
            with plan(rows, splits):
                for d in (api.gemm(a.operand(), b.operand(), M, N, K, out_dtype=out),
                          api.gemm(a.operand(), b.operand(), M, N, K, accumulate=True,
                                   out=torch.zeros((M, N), dtype=out, device=DEV))):
                    assert np.array_equal(np.isfinite(as64(d)), keep)


@pytest.mark.parametrize("rows,splits", PLANS)
def test_rows_do_not_depend_on_their_neighbours(rows, splits):
    """An outlier row, zero blocks, and scales 2^-70 and 2^40 that multiply out."""
    M, N, K = {16: 16, 64: 100, 128: 200, 192: 300, 256: 300}[rows], 300, 384
    x, w = spread((M, K), 1).float(), spread((N, K), 2).float()
    x[M // 2] *= 2.0 ** 60
    x[:, 128:256] *= 2.0 ** -70
    w[:, 128:256] *= 2.0 ** 40
    w[5] = 0.0
    w[7] *= 2.0 ** -50
    a, b = api.quantize(bf16(x).to(DEV), "fp8"), api.quantize(bf16(w).to(DEV), "fp8")
    for out in out_types(rows):
        with plan(rows, splits):
            d = api.gemm(a.operand(), b.operand(), M, N, K, out_dtype=out)
            close(d, *product(a, b))
            assert not d[:, 5].any()


@pytest.mark.parametrize("rows,splits", PLANS)
def test_captured(rows, splits):
    M, N, K = {16: 9, 64: 100, 128: 200, 192: 300, 256: 600}[rows], 520, 900
    sets = [operands(M, N, K, seed=s) for s in (1, 5)]
    a, b = operands(M, N, K, seed=1)
    for out in out_types(rows):
        with plan(rows, splits):
            want = [api.gemm(q.operand(), b.operand(), M, N, K, out_dtype=out) for q, _ in sets]
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                d = api.gemm(a.operand(), b.operand(), M, N, K, out_dtype=out)
            for k in (0, 1, 0, 1):
                a.codes.copy_(sets[k][0].codes)
                a.scales.copy_(sets[k][0].scales)
                g.replay()
                api.gemm(sets[0][0].operand(), b.operand(), M, N, K, out_dtype=out)
                torch.cuda.synchronize()
                assert torch.equal(d, want[k])


def test_many_tiles_per_workgroup():
    """The bf16 kernel that loops: more tiles than CUs, an odd and an even number
    of blocks."""
    M, N = 256 * 21 + 5, 256 * 13 + 9
    for K in (300, 512):
        a, b, ref = case(M, N, K, "fp8")
        with plan(256, 1):
            close(api.gemm(a.operand(), b.operand(), M, N, K, out_dtype=BF), *ref)
