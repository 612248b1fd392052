"""A recipe's formats by name or by the library's numbers, as quantize takes them."""
import pytest
import torch

from fp4_block_scaled_x16_amd import api
from fp4_block_scaled_x16_amd.ffn import QuantizedFFN
from fp4_block_scaled_x16_amd.linear import QuantizedLinear, Recipe


def w(rows, cols):
    return torch.zeros((rows, cols), dtype=torch.bfloat16)


@pytest.mark.parametrize("name", ["nvfp4", "ue5m3", "mxfp4", "fp8"])
def test_numbers(name):
    r = Recipe(fmt=api.FORMATS[name], out_dtype="bf16")
    assert r == Recipe(fmt=name, out_dtype="bf16")
    assert r.two_level == Recipe(fmt=name).two_level
    assert QuantizedLinear(w(128, 128), r).recipe is r
    assert QuantizedFFN(w(256, 64), w(64, 128), "swiglu", r).recipe.fmt == name


def test_gradient_format():
    assert Recipe(fmt="fp8", grad_fmt=api.FP8_E4M3) == Recipe(fmt="fp8", grad_fmt="fp8")


@pytest.mark.parametrize("kw", [dict(fmt=api.MXFP8), dict(fmt=99), dict(fmt="fp8", grad_fmt=api.NVFP4)])
def test_refused(kw):
    with pytest.raises(ValueError):
        QuantizedLinear(w(128, 128), Recipe(**kw))
