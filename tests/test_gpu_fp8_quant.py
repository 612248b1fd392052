"""GPU parity of FP8 block-128 quantization (along rows, along columns, both,
128x128), dequantization and the re-encoding of row codes along the columns:
codes, padding and scales to the bit against the 64-bit oracle; sizes from one
element to several ragged tiles, strided and offset inputs, memory around the
outputs, non-finite values, counters, launch geometries, another stream and
captured graphs."""
import ctypes

import numpy as np
import pytest
import torch

from fp4_block_scaled_x16_amd import api
from fp8_check import DEV, as64, bf16, same_matrix, spread
from oracle import fp8

pytestmark = pytest.mark.gpu
FMTS = ["fp8", "fp8_e5m2"]
SIZES = [(1, 1), (1, 130), (3, 7), (17, 128), (127, 129), (128, 128), (129, 257), (300, 1000),
         (5, 4104), (1025, 60)]


def oracle(x, fmt, block="1d"):
    v = as64(x)
    return fp8.encode(v, fmt, block), fp8.encode(v.T, fmt, block)


@pytest.mark.parametrize("R,C", SIZES)
@pytest.mark.parametrize("block", ["1d", "2d"])
@pytest.mark.parametrize("fmt", FMTS)
def test_quantize(fmt, block, R, C):
    x = spread((R, -(-C // 8) * 8), R + C)[:, :C]        # rows of a wider matrix
    xd = spread((R, -(-C // 8) * 8), R + C).to(DEV)[:, :C]
    row, col = oracle(x, fmt, block)
    same_matrix(api.quantize(xd, fmt, block=block), *row)
    same_matrix(api.quantize(xd, fmt, block=block, orient="col"), *col)
    both = api.quantize_dual(xd, fmt, block=block)
    same_matrix(both[0], *row)
    same_matrix(both[1], *col)
    if block == "2d":
        assert torch.equal(both[0].codes[:, :C].t(), both[1].codes[:, :R])


@pytest.mark.parametrize("fmt", FMTS)
def test_every_bf16_value_of_a_block(fmt):
    """All finite bf16 values, each beside one that fixes its block's scale: the
    whole range of the scales, and every rounding of the elements."""
    bits = np.arange(1 << 16, dtype=np.uint16)
    v = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    v = v[torch.isfinite(v.float())]
    x = torch.cat([v, torch.zeros(-v.numel() % 128, dtype=torch.bfloat16)]).view(-1, 128)
    for amax in (None, 3.5, 448.0, 57344.0, 2.0 ** -120, 3e38):
        y = x.clone()
        if amax is not None:
            y[y.float().abs() > amax] = 0
            y[:, 5] = amax
        same_matrix(api.quantize(y.to(DEV), fmt), *fp8.encode(as64(y), fmt))


@pytest.mark.parametrize("R,C", SIZES)
@pytest.mark.parametrize("fmt", FMTS)
def test_requantize_t(fmt, R, C):
    x = spread((R, -(-C // 8) * 8), R + C + 1)[:, :C]
    q = api.quantize(x.to(DEV) if C % 8 == 0 else spread((R, -(-C // 8) * 8), R + C + 1).to(DEV)[:, :C], fmt)
    q.scales[:, R:] = 255                       # padding of unspecified value
    held = fp8.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), fmt)[:, :C]
    same_matrix(api.requantize_t(q), *fp8.encode(held.T, fmt))


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,C", [(1, 1), (17, 130), (129, 256), (40, 1001)])
@pytest.mark.parametrize("fmt", FMTS)
def test_dequantize(fmt, R, C, out):
    q = api.quantize(spread((R, -(-C // 8) * 8), 5).to(DEV)[:, :C], fmt)
    want = fp8.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), fmt)[:, :C]
    got = api.dequantize(q, out)
    assert got.dtype == out and torch.equal(got.cpu(), torch.from_numpy(want).to(torch.float32).to(out))


def raw_calls(x, R, C, fmt):
    """Every quantizing call of the ABI into buffers with a guard band behind
    each output: {name: (outputs, guards)}."""
    lib, f = api.load_library(), api.FORMATS[fmt]
    kr, kc = -(-R // 128), -(-C // 128)
    sizes = [R * kc * 128, kc * (-(-R // 16) * 16), C * kr * 128, kr * (-(-C // 16) * 16)]
    buf = [torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device=DEV) for n in sizes]
    d = [api.QuantDesc(f, 0, o, 0, 0, 0, 0, 0, 448.0, 0, 0, 2, 0, (ctypes.c_uint32 * 3)(), 0, 0, 0)
         for o in (0, 1)]
    p = [ctypes.c_void_p(b.data_ptr()) for b in buf]
    xp = ctypes.c_void_p(x.data_ptr())
    s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert lib.fp4_quantize_dual(ctypes.byref(d[0]), ctypes.byref(d[1]), xp, R, C, x.stride(0), *p,
                                 None, None, None, None, None, s) == 0
    assert lib.fp4_requantize_t(f, p[0], p[1], R, C, p[2], p[3], s) == 0
    for b, n in zip(buf, sizes):
        assert bool((b[n:] == 0xA5).all())


@pytest.mark.parametrize("R,C", [(1, 1), (17, 130), (130, 264), (256, 129)])
def test_nothing_is_written_behind_the_outputs(R, C):
    raw_calls(spread((R, -(-C // 8) * 8), 9).to(DEV)[:, :C], R, C, "fp8")


@pytest.mark.parametrize("fmt", FMTS)
def test_strided_and_offset_input(fmt):
    wide = spread((200, 1024), 3).to(DEV)
    x = wide[7:150, 64:64 + 333]                # 16-byte aligned, ld 1024
    row, col = oracle(x, fmt)
    both = api.quantize_dual(x, fmt)
    same_matrix(both[0], *row)
    same_matrix(both[1], *col)
    with pytest.raises(api.Fp4Error):
        api.quantize(wide[:, 1:257], fmt)       # not 16-byte aligned


@pytest.mark.parametrize("fmt", FMTS)
def test_non_finite_values(fmt):
    """A NaN stays one and leaves its block's scale alone; an infinity takes the
    scale of the largest finite value, under which the others are encoded."""
    v = spread((128, 256), 6).float()
    clean = v.clone()
    v[3, 5], v[4, 200], v[60, 130] = float("nan"), float("inf"), float("-inf")
    v[70, :128] = float("nan")
    clean[3, 5] = clean[4, 200] = clean[60, 130] = 0.0
    clean[70, :128] = 0.0
    q = api.quantize(bf16(v).to(DEV), fmt)
    codes, scales = fp8.encode(as64(bf16(clean)), fmt)
    got = fp8.decode_table(fmt)[q.codes.cpu().numpy()]
    assert np.isnan(got[3, 5]) and np.isnan(got[70, :128]).all()
    big = np.isnan if fmt == "fp8" else np.isinf
    assert big(got[4, 200]) and big(got[60, 130])
    s = q.scales.cpu().numpy()
    top = 127 + int(fp8.scale_exponents(np.array([np.finfo(np.float32).max], np.float64), fmt)[0])
    assert s[1, 4] == top and s[1, 60] == top
    scales[1, 4] = scales[1, 60] = top
    assert np.array_equal(s[:, :128], scales)
    keep = np.ones((128, 256), bool)
    keep[3, 5] = keep[4, 128:] = keep[60, 128:] = keep[70, :128] = False
    assert np.array_equal(q.codes.cpu().numpy()[keep], codes[keep])


@pytest.mark.parametrize("fmt,tiny", [("fp8", 0), ("fp8", 40), ("fp8_e5m2", 40)])
def test_counters(fmt, tiny):
    x = spread((130, 264), 8)
    x[:, ::5] *= 2.0 ** -tiny                   # E5M2 reaches 2^-32 below a block's largest
    row, col = oracle(x, fmt)
    nonzero = as64(x) != 0
    lost = [int((nonzero & ((c[:R, :C] & 127) == 0)).sum()) if R == 130 else
            int((nonzero.T & ((c[:R, :C] & 127) == 0)).sum())
            for c, R, C in ((row[0], 130, 264), (col[0], 264, 130))]
    assert lost[0] > 0 and lost[1] > 0
    c = api.new_counters()
    api.quantize(x.to(DEV), fmt, counters=c)
    assert api.counters_dict(c)["elem_underflow"] == lost[0]
    api.quantize_dual(x.to(DEV), fmt, counters=c)
    want = dict.fromkeys(api.COUNTER_NAMES, 0)
    want["elem_underflow"] = 2 * lost[0] + lost[1]
    assert api.counters_dict(c) == want
    api.quantize(x.to(DEV), fmt, counters=c, count="scales")
    assert api.counters_dict(c) == want


def test_empty():
    for R, C in ((0, 64), (64, 0)):
        x = torch.empty((R, C), dtype=torch.bfloat16, device=DEV)
        a, b = api.quantize_dual(x, "fp8")
        assert a.codes.shape == (R, -(-C // 128) * 128) and b.codes.shape == (C, -(-R // 128) * 128)
        assert api.requantize_t(a).codes.shape == b.codes.shape
        assert api.dequantize(a).shape == (R, C)


def test_geometry_does_not_change_results():
    x = spread((700, 900 // 8 * 8), 11).to(DEV)
    want = [t for q in api.quantize_dual(x, "fp8") for t in (q.codes, q.scales[:, :q.rows])]
    two = [t for q in api.quantize_dual(x, "fp8", block="2d") for t in (q.codes, q.scales[:, :q.rows])]
    t0 = api.requantize_t(api.quantize(x, "fp8")).codes
    try:
        for wgs in (1, 3, 37):
            api.selftest_set_geometry(wgs)
            got = [t for q in api.quantize_dual(x, "fp8") for t in (q.codes, q.scales[:, :q.rows])]
            g2 = [t for q in api.quantize_dual(x, "fp8", block="2d") for t in (q.codes, q.scales[:, :q.rows])]
            assert all(torch.equal(a, b) for a, b in zip(want + two, got + g2))
            assert torch.equal(t0, api.requantize_t(api.quantize(x, "fp8")).codes)
            r2 = api.quantize(x, "fp8", block="2d")
            assert torch.equal(two[0], r2.codes)
    finally:
        api.selftest_set_geometry()


def test_another_stream_and_a_captured_graph():
    """Calls land on the current stream; a captured sequence replays on new
    inputs, also with eager calls between the replays."""
    xs = [spread((260, 520), k).to(DEV) for k in range(4)]
    want = [oracle(x, "fp8") for x in xs]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = api.quantize_dual(xs[0], "fp8")
    torch.cuda.current_stream().wait_stream(s)
    same_matrix(got[0], *want[0][0])
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r, c = api.quantize_dual(x, "fp8")
        t = api.requantize_t(r)
    for k in (1, 2, 3, 1):
        x.copy_(xs[k])
        g.replay()
        api.quantize(xs[0], "fp8")              # the program's own work between replays
        torch.cuda.synchronize()
        same_matrix(r, *want[k][0])
        same_matrix(c, *want[k][1])
        held = fp8.values(*want[k][0], "fp8")[:, :520]
        same_matrix(t, *fp8.encode(held.T, "fp8"))
