"""FP8 block-128 formats and the operators on them, in 64-bit arithmetic.

E4M3 (fmt "fp8": 4 exponent bits, bias 7, 3 mantissa bits, largest 448, no
infinities) and E5M2 ("fp8_e5m2": 5, bias 15, 2, largest 57344) elements with
one scale 2^e per block of 128 (1x128 or 128x128), e the smallest integer in
[-127, 127] with largest * 2^e >= amax, -127 for a zero block; element = round
to nearest even of x * 2^-e.  bf16 inputs and powers of two are exact in 64
bits, so codes and scales are defined to the bit.
"""
from __future__ import annotations

import numpy as np

# bias, mantissa bits, largest finite value
FORMATS = {"fp8": (7, 3, 448.0), "fp8_e5m2": (15, 2, 57344.0)}


def decode_table(fmt):
    """The value of each of the 256 codes (NaN and infinity included)."""
    bias, m, top = FORMATS[fmt]
    c = np.arange(256)
    e, f = (c & 127) >> m, c & ((1 << m) - 1)
    v = np.where(e > 0, np.ldexp(1.0 + f / (1 << m), e - bias), np.ldexp(f / (1 << m), 1 - bias))
    if fmt == "fp8":
        v = np.where((c & 127) == 127, np.nan, v)
    else:
        v = np.where(e == 31, np.where(f == 0, np.inf, np.nan), v)
    return np.where(c > 127, -v, v)


def encode_element(y, fmt):
    """Codes of float64 y, |y| <= largest, rounded to nearest even."""
    bias, m, top = FORMATS[fmt]
    a = np.abs(np.asarray(y, np.float64))
    assert np.all(a <= top)
    _, k = np.frexp(a)                                   # a = f 2^k, f in [0.5, 1)
    k = np.where(a > 0, np.maximum(k - 1, 1 - bias), 1 - bias)
    q = np.rint(np.ldexp(a, m - k)).astype(np.int64)     # in steps of 2^(k - m)
    code = np.where(q >= (1 << m), ((k + bias) << m) + q - (1 << m), q)   # a carry moves the exponent on
    return (code | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def scale_exponents(amax, fmt):
    """e of every block amax (float64)."""
    top = FORMATS[fmt][2]
    _, k = np.frexp(amax / top)                          # amax / top <= 2^k
    e = np.where(np.ldexp(top, k - 1) >= amax, k - 1, k)
    return np.where(amax > 0, np.clip(e, -127, 127), -127).astype(np.int64)


def _up(v, to):
    return -(-v // to) * to


def encode(x, fmt, block="1d"):
    """(codes [R, C up to 128], scale bytes [blocks, R]) of float64 x [R, C]."""
    x = np.asarray(x, np.float64)
    R, C = x.shape
    v = np.zeros((R, _up(C, 128)))
    v[:, :C] = x
    v = v.reshape(R, -1, 128)
    amax = np.abs(v).max(2) if R else np.zeros(v.shape[:2])
    if block == "2d":
        for r in range(0, R, 128):
            amax[r:r + 128] = amax[r:r + 128].max(0)
    e = scale_exponents(amax, fmt)
    codes = encode_element(np.ldexp(v, -e[:, :, None]), fmt)
    return codes.reshape(R, -1), (e + 127).astype(np.uint8).T.copy()


def values(codes, scales, fmt):
    """float64 values [R, C up to 128] of codes and scale bytes [blocks, >= R]."""
    R = codes.shape[0]
    e = scales[:, :R].astype(np.int64).T - 127
    return np.ldexp(decode_table(fmt)[codes].reshape(R, -1, 128), e[:, :, None]).reshape(codes.shape)


def gemm(a, b):
    """D = A B^T and the bound's sum |a b|, of float64 values."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def checkpoint_layout(h, cols):
    """The halves of h, each from a multiple of 128 columns on: the matrix whose
    codes the activation's checkpoint holds."""
    halves = h.shape[1] // cols
    out = np.zeros((h.shape[0], (halves - 1) * _up(cols, 128) + cols), h.dtype)
    for k in range(halves):
        out[:, k * _up(cols, 128):k * _up(cols, 128) + cols] = h[:, k * cols:(k + 1) * cols]
    return out


def _sigmoid(g):
    t = np.exp(-np.abs(g))
    return np.where(g >= 0, 1 / (1 + t), t / (1 + t))


def act(h, kind):
    """SwiGLU: silu(g) u of h = [g | u]; squared ReLU: max(h, 0)^2."""
    if kind == "relu2":
        return np.maximum(h, 0.0) ** 2
    F = h.shape[1] // 2
    return h[:, :F] * _sigmoid(h[:, :F]) * h[:, F:]


def act_grad(h, da, kind):
    """The gradient of h."""
    if kind == "relu2":
        return 2 * np.maximum(h, 0.0) * da
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    s = _sigmoid(g)
    return np.concatenate([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
