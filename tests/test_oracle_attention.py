"""Pins of the oracle of attention on a quantized cache: rotation as multiplication of
complex numbers, gradients against differences, attention against hand examples, a
cache's rows against the one-row matrices of the other oracles."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import formats as F
from oracle import fp8
from oracle import quantize as Q

RNG = np.random.default_rng(0)


@pytest.mark.parametrize("inter", [False, True])
def test_turn_is_a_product_of_complex_numbers(inter):
    x, a = RNG.standard_normal((3, 20)), RNG.uniform(-4, 4, (3, 8))
    y = A.turn(x, np.cos(a), np.sin(a), inter)
    z = (x[:, 0:16:2] + 1j * x[:, 1:16:2]) if inter else (x[:, :8] + 1j * x[:, 8:16])
    z = z * np.exp(1j * a)
    got = (y[:, 0:16:2] + 1j * y[:, 1:16:2]) if inter else (y[:, :8] + 1j * y[:, 8:16])
    assert np.allclose(got, z, atol=1e-14) and np.array_equal(y[:, 16:], x[:, 16:])
    assert np.allclose(A.turn(y, np.cos(a), np.sin(a), inter, back=True), x, atol=1e-14)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm,rot", [(True, True), (True, False), (False, True)])
def test_gradient_against_differences(inter, norm, rot):
    x, dy, a = RNG.standard_normal((4, 16)), RNG.standard_normal((4, 16)), RNG.uniform(-4, 4, (4, 6))
    w = RNG.standard_normal(16) if norm else None
    c, s = (np.cos(a), np.sin(a)) if rot else (None, None)
    dx, dw = A.norm_rope_grad(x, w, c, s, 1e-3, dy, inter)
    f = lambda x, w: (A.norm_rope(x, w, c, s, 1e-3, inter) * dy).sum()       # noqa: E731
    h = 1e-6
    for _ in range(5):
        t = RNG.standard_normal(x.shape)
        assert np.isclose((f(x + h * t, w) - f(x - h * t, w)) / (2 * h), (dx * t).sum(), rtol=1e-7, atol=1e-8)
        if norm:
            t = RNG.standard_normal(16)
            assert np.isclose((f(x, w + h * t) - f(x, w - h * t)) / (2 * h), dw @ t, rtol=1e-7, atol=1e-8)


def test_attention_by_hand():
    k, v = np.array([[1.0, 0], [0, 1]]), np.array([[2.0, 4], [6, 0]])
    out, lse = A.attention(np.array([np.log(3.0), 0]), k, v, 1.0)             # weights 3/4, 1/4
    assert np.allclose(out, [3, 3]) and np.isclose(lse, np.log(4.0))
    out, lse = A.attention(np.zeros(2), k[:0], v[:0], 1.0)
    assert not out.any() and lse == -np.inf
    # one token: its value, whatever the score
    assert np.array_equal(A.attention(np.array([900.0, -900.0]), k[1:], v[1:], 1.0)[0], v[1])


@pytest.mark.parametrize("fmt", list(A.BLOCK))
@pytest.mark.parametrize("d", [64, 256])
def test_rows_are_one_row_matrices(fmt, d):
    bits = F.f32_to_bf16_bits(RNG.standard_normal((5, d)).astype(np.float32))
    top = 2048.0 if fmt == "ue5m3" else 448.0          # (NVFP4's scales end at 448)
    codes, scales = A.encode_rows(bits, fmt, 4.5, top)
    for i in range(5):
        if fmt == "fp8":
            c, s = fp8.encode(F.bf16_bits_to_f32(bits[i:i + 1]).astype(np.float64), "fp8")
            assert np.array_equal(c[0, :d], codes[i]) and np.array_equal(s[:, 0], scales[i])
        else:
            q = Q.quantize(bits[i:i + 1], fmt, amax=4.5 if fmt in A.TWO_LEVEL else None, target=top)
            assert np.array_equal(q["codes"][0], codes[i]) and np.array_equal(q["scales"][0], scales[i])
    v = A.row_values(codes, scales, fmt, d, A.s_dec(fmt, 4.5, top))
    x = F.bf16_bits_to_f32(bits).astype(np.float64)
    assert np.linalg.norm(v - x) < (0.04 if d == codes.shape[1] else 0.2) * np.linalg.norm(x)
