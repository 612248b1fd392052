"""What QuantizedLinear and QuantizedFFN refuse when they are made."""
import pytest
import torch

from fp4_block_scaled_x16_amd.ffn import QuantizedFFN
from fp4_block_scaled_x16_amd.linear import QuantizedLinear, Recipe


def w(rows, cols):
    return torch.zeros((rows, cols), dtype=torch.bfloat16)


@pytest.mark.parametrize("kw", [dict(fmt="mxfp8"), dict(fmt="fp8_e5m2"), dict(fmt="fp8", rht=True),
                                dict(fmt="fp8", rht_kd=True), dict(fmt="fp8", act_block="2d"),
                                dict(fmt="fp8", grad_fmt="nvfp4"), dict(fmt="fp8", out_dtype="fp16")])
def test_linear(kw):
    with pytest.raises(ValueError):
        QuantizedLinear(w(128, 128), Recipe(**kw))


BF = dict(out_dtype="bf16")


@pytest.mark.parametrize("up,down,act,recipe", [
    ((256, 64), (64, 128), "gelu", Recipe(fmt="fp8", **BF)),
    ((256, 64), (64, 128), "swiglu", Recipe(fmt="fp8")),              # fp32 outputs
    ((128, 64), (64, 128), "swiglu", Recipe(fmt="fp8", **BF)),        # up has 2F rows
    ((256, 64), (64, 128), "relu2", Recipe(fmt="fp8", **BF)),         # up has F rows
    ((272, 64), (64, 136), "swiglu", Recipe(fmt="fp8", **BF)),        # F % 128
    ((132, 64), (64, 132), "relu2", Recipe(fmt="fp8", **BF)),         # F % 8
])
def test_ffn(up, down, act, recipe):
    with pytest.raises(ValueError):
        QuantizedFFN(w(*up), w(*down), act, recipe)


def test_backward_needs_forward():
    layer = QuantizedFFN(w(256, 64), w(64, 128), "swiglu")
    with pytest.raises(RuntimeError):
        layer.backward(w(4, 64))
