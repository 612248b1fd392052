"""Pins of the FP8 block-128 oracle: element codes against torch's float8
types and against the nearest table entry, scales against the smallest
fitting power of two in exact rationals, a hand example, and the activations'
gradients against differences."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import fp8

TORCH = {"fp8": torch.float8_e4m3fn, "fp8_e5m2": torch.float8_e5m2}
FMTS = ["fp8", "fp8_e5m2"]


@pytest.mark.parametrize("fmt", FMTS)
def test_decode_table_is_torchs(fmt):
    want = torch.arange(256, dtype=torch.uint8).view(TORCH[fmt]).double().numpy()
    np.testing.assert_array_equal(fp8.decode_table(fmt), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_elements_round_to_nearest_even(fmt):
    top = fp8.FORMATS[fmt][2]
    t = fp8.decode_table(fmt)[:128]
    t = t[np.isfinite(t)]
    mids = (t[:-1] + t[1:]) / 2
    y = np.concatenate([t, mids, np.nextafter(mids, 0), np.nextafter(mids, top),
                        np.random.default_rng(1).uniform(0, top, 4096),
                        np.exp2(np.random.default_rng(2).uniform(-20, np.log2(top), 4096))])
    for v in (y, -y):
        codes = fp8.encode_element(v, fmt)
        near = np.abs(np.abs(v)[:, None] - t[None, :])
        best = near.min(1)
        np.testing.assert_array_equal(near[np.arange(v.size), codes & 127], best)
        tie = (near == best[:, None]).sum(1) == 2
        assert np.all((codes[tie] & 1) == 0)
        f32 = v.astype(np.float32)
        same = f32 == v                            # torch converts from fp32
        want = torch.from_numpy(f32[same]).to(TORCH[fmt]).view(torch.uint8).numpy()
        np.testing.assert_array_equal(codes[same], want)


@pytest.mark.parametrize("fmt", FMTS)
def test_scale_is_the_smallest_that_fits(fmt):
    top = Fraction(fp8.FORMATS[fmt][2])
    rng = np.random.default_rng(3)
    amax = np.concatenate([np.exp2(rng.uniform(-140, 127, 500)).astype(np.float32),
                           np.float32(1.75) * np.exp2(np.arange(-30, 31)).astype(np.float32)])
    amax = np.concatenate([amax, np.nextafter(amax, np.float32(0)), np.nextafter(amax, np.float32(np.inf)),
                           [np.finfo(np.float32).max, np.float32(1e-45)]]).astype(np.float64)
    for a, e in zip(amax, fp8.scale_exponents(amax, fmt)):
        e, a = int(e), Fraction(float(a))
        assert top * Fraction(2) ** e >= a
        assert e == -127 or top * Fraction(2) ** (e - 1) < a
    assert fp8.scale_exponents(np.zeros(1), fmt)[0] == -127


def test_hand_example():
    x = np.zeros((2, 130))
    x[0, :3] = [896.0, 1.0, -3.0]        # e = 1: 448, 0.5, -1.5
    x[0, 129] = 449.0                    # e = 1: 224.5 -> 224
    x[1, 0] = 448.0                      # e = 0
    codes, scales = fp8.encode(x, "fp8")
    assert codes.shape == (2, 256) and scales.shape == (2, 2)
    assert scales.tolist() == [[128, 127], [128, 0]]
    assert codes[0, :3].tolist() == [0x7E, 0x30, 0xBC]
    assert fp8.values(codes, scales, "fp8")[0, 129] == 448.0
    two, s2 = fp8.encode(x, "fp8", "2d")
    assert s2.tolist() == [[128, 128], [128, 128]]
    t, st = fp8.encode(x.T, "fp8", "2d")
    np.testing.assert_array_equal(t[:130, :2].T, two[:, :130])
    assert codes.reshape(-1).size == 512 and not codes[:, 130:].any()


@pytest.mark.parametrize("kind", ["swiglu", "relu2"])
def test_act_grad_is_the_difference_quotient(kind):
    rng = np.random.default_rng(4)
    h = rng.standard_normal((5, 16)) * 3
    F = 8 if kind == "swiglu" else 16
    da = rng.standard_normal((5, F))
    got = fp8.act_grad(h, da, kind)
    d = 1e-5
    for j in range(16):
        e = np.zeros(16)
        e[j] = d
        want = ((fp8.act(h + e, kind) - fp8.act(h - e, kind)) * da).sum(1) / (2 * d)
        # central differences: d^2 / 6 times a third derivative below 10 * 3, and
        # 2^-52 * 100 / d of rounding
        np.testing.assert_allclose(got[:, j], want, atol=1e-8)
