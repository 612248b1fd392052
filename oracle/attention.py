"""Attention on a quantized cache in 64-bit arithmetic: the norm and rotation of
queries and keys with their gradients, the codes of a cache's rows, and attention
of one query.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

  r = (mean x^2 + eps)^(-1/2);  z = x r w;  y = z with each pair (a, b) turned by its
  angle t: (a cos t - b sin t, b cos t + a sin t), that is (a + i b) e^(i t)
  backward: dz = dy turned by -t; dw = sum dz x r; g = dz w; dx = r (g - x r^2 mean(g x))
  out = sum_t p_t v_t,  p = softmax_t(scale q . k_t)

A cache's row is a one-row matrix in blocks along its columns, in the formats of
``oracle.quantize`` and ``oracle.fp8``; the two-level formats take a given amax.
"""
from __future__ import annotations

import numpy as np

from . import formats as F
from . import fp8
from . import quantize as Q

BLOCK = {"fp8": 128, "mxfp8": 32, "mxfp4": 32, "nvfp4": 16, "ue5m3": 16}
TWO_LEVEL = ("nvfp4", "ue5m3")


def turn(z, cos, sin, interleaved=False, back=False):
    """Rows z [..., D] with their first 2 P elements turned; cos, sin [..., P]."""
    z = np.array(z, np.float64)
    P = cos.shape[-1]
    a, b = (z[..., 0:2 * P:2], z[..., 1:2 * P:2]) if interleaved else (z[..., :P], z[..., P:2 * P])
    s = -sin if back else sin
    new = a * cos - b * s, b * cos + a * s
    for k in range(2):
        if interleaved:
            z[..., k:2 * P:2] = new[k]
        else:
            z[..., k * P:(k + 1) * P] = new[k]
    return z


def inv_rms(x, eps):
    return 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)


def norm_rope(x, w, cos, sin, eps, interleaved=False):
    """y of float64 rows x; w None: no norm; cos None: no rotation."""
    z = x if w is None else x * inv_rms(x, eps) * w
    return z if cos is None else turn(z, cos, sin, interleaved)


def norm_rope_grad(x, w, cos, sin, eps, dy, interleaved=False):
    """(dx, dw) of rows x and dy [..., D]; dw summed over every row (None without w)."""
    dz = dy if cos is None else turn(dy, cos, sin, interleaved, back=True)
    if w is None:
        return dz, None
    r = inv_rms(x, eps)
    g = dz * w
    return r * (g - x * r * r * np.mean(g * x, -1, keepdims=True)), (dz * x * r).reshape(-1, x.shape[-1]).sum(0)


def encode_rows(x_bits, fmt, amax=None, target=448.0):
    """(codes [N, bytes], scales [N, blocks]) of bf16 rows (uint16 bits, [N, D])."""
    if fmt == "fp8":
        codes, scales = fp8.encode(F.bf16_bits_to_f32(x_bits).astype(np.float64), "fp8")
        return codes[:, :x_bits.shape[1]], scales.T.copy()
    q = Q.quantize(x_bits, fmt, amax=amax if fmt in TWO_LEVEL else None, target=target)
    return q["codes"].reshape(len(x_bits), -1), q["scales"]


def s_dec(fmt, amax, target=448.0):
    return float(Q.global_scales(np.float32(amax), target)[1]) if fmt in TWO_LEVEL else 1.0


def row_values(codes, scales, fmt, D, dec=1.0):
    """float64 values [N, D] of rows of codes, times the tensor's decode scale."""
    N = codes.shape[0]
    if not N:
        return np.zeros((0, D))
    if fmt == "fp8":
        wide = np.zeros((N, -(-D // 128) * 128), np.uint8)
        wide[:, :D] = codes
        return fp8.values(wide, scales.T, "fp8")[:, :D]
    return Q.operand_values(codes, scales, fmt, "1d", N, D) * dec


def attention(q, k, v, scale):
    """(out [D], lse) of q [D] over k, v [n, D] (float64); (0, -inf) for n = 0."""
    if not len(k):
        return np.zeros(v.shape[-1]), -np.inf
    x = k @ q * scale
    top = x.max()
    p = np.exp(x - top)
    return p @ v / p.sum(), top + np.log(p.sum())
