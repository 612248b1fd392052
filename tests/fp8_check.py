"""Shared by the FP8 tests: device copies, and the comparison of codes with
values that were computed with a known relative error before they were
encoded."""
import numpy as np
import torch

from oracle import formats as F
from oracle import fp8

DEV = "cuda"


def bf16(v):
    """The bf16 bits of float32 v (nearest even)."""
    return torch.from_numpy(np.ascontiguousarray(v, np.float32)).to(torch.bfloat16)


def as64(t):
    return t.cpu().double().numpy()


def spread(shape, seed, sigma=1.0):
    """Normal values with rows of very different sizes, a zero row, a row of
    equal powers of two with one larger entry (subnormals and ties), and a few
    outliers."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal(shape).astype(np.float32) * np.float32(sigma)
    v *= np.exp2(np.arange(shape[0]) % 23 - 11.0).astype(np.float32)[:, None]
    v[rng.random(shape) < 0.002] *= np.float32(50)
    if shape[0] > 2:
        v[1] = 0.0
        v[2] = np.float32(2.0 ** -20)
        v[2, ::7] = np.float32(1.1875)
    return bf16(v)


def same_matrix(q, codes, scales):
    """Codes whole (their padding is zero) and the valid scales, to the bit."""
    got = q.codes.cpu().numpy()
    assert got.shape == codes.shape
    assert np.array_equal(got, codes), np.argwhere(got != codes)[:5].tolist()
    got = q.scales.cpu().numpy()[:, :q.rows]
    assert np.array_equal(got, scales), np.argwhere(got != scales)[:5].tolist()


def encodes(q, v, err, fmt):
    """q [R, C] holds v (float64) rounded from values within err (absolute, per
    element) of it: each scale is that of some amax within the block's error,
    each element half a step of its format at that scale, or less, from v."""
    R, C = v.shape
    codes, sc = q.codes.cpu().numpy(), q.scales.cpu().numpy()[:, :R]
    assert codes.shape == (R, -(-C // 128) * 128) and not codes[:, C:].any()
    pad = np.zeros((2, R, codes.shape[1]))
    pad[0, :, :C], pad[1, :, :C] = v, err
    a = np.abs(pad[0]).reshape(R, -1, 128)
    e = pad[1].reshape(R, -1, 128)
    lo = fp8.scale_exponents(np.maximum(a - e, 0).max(2), fmt)
    hi = fp8.scale_exponents((a + e).max(2), fmt)
    got_e = sc.T.astype(np.int64) - 127
    assert np.all((got_e >= lo) & (got_e <= hi))
    bias, m, top = fp8.FORMATS[fmt]
    got = fp8.values(codes, sc, fmt)
    s = np.repeat(np.exp2(got_e.astype(np.float64)), 128, 1)
    # half a step of the larger of the two sides' binades, at least the subnormals'
    mag = np.maximum(np.abs(pad[0]) + pad[1], s * 2.0 ** (1 - bias))
    half = np.exp2(np.floor(np.log2(mag)) - m - 1)
    bad = np.abs(got - pad[0]) > half + pad[1]
    assert not bad.any(), np.argwhere(bad)[:5].tolist()
