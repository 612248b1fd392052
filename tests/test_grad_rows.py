"""The gradient that autograd hands QuantizedLinear and QuantizedFFN reaches
their backward step row-major with 16-byte aligned rows, as the quantizers take
it, whatever the number of output features and the gradient's own layout."""
import pytest
import torch

from fp4_block_scaled_x16_amd.ffn import QuantizedFFN
from fp4_block_scaled_x16_amd.linear import QuantizedLinear, Recipe

BF = torch.bfloat16
R = Recipe(fmt="fp8", out_dtype="bf16")


def layer_with(kind, outs):
    """A layer of 16 features in and `outs` out whose steps are stood in for; its
    backward step keeps the gradient that it is given."""
    if kind == "linear":
        layer = QuantizedLinear(torch.zeros((outs, 16), dtype=BF), R)
    else:
        layer = QuantizedFFN(torch.zeros((8, 16), dtype=BF), torch.zeros((outs, 8), dtype=BF), "relu2", R)
    layer.given = []
    layer._forward = lambda x: (x.new_zeros((x.shape[0], outs)), ())
    layer._backward = lambda dy, saved: (layer.given.append(dy), dy.new_zeros((dy.shape[0], 16)))[1]
    return layer


def gradient(how, rows, cols):
    v = torch.arange(rows * cols).reshape(rows, cols).to(BF)
    if how == "dense":
        return v
    if how == "padded rows":
        g = torch.zeros((rows, -(-cols // 8) * 8 + 16), dtype=BF)[:, :cols]
    elif how == "odd pitch":
        g = torch.zeros((rows, cols + 3), dtype=BF)[:, :cols]
    elif how == "odd offset":
        g = torch.zeros(rows * cols + 3, dtype=BF)[3:].view(rows, cols)
    elif how == "transposed":
        g = torch.zeros((cols, rows), dtype=BF).t()
    else:                                            # one row for all
        return v[:1].expand(rows, cols)
    g.copy_(v)
    return g


LAYOUTS = ["dense", "padded rows", "odd pitch", "odd offset", "transposed", "broadcast"]


@pytest.mark.parametrize("kind", ["linear", "ffn"])
@pytest.mark.parametrize("outs", [1, 8, 96, 100])
@pytest.mark.parametrize("rows", [0, 1, 5])
@pytest.mark.parametrize("how", LAYOUTS)
def test_rows(kind, outs, rows, how):
    if how == "broadcast" and rows == 0:
        pytest.skip("no row to broadcast")
    layer = layer_with(kind, outs)
    x = torch.zeros((rows, 16), dtype=BF, requires_grad=True)
    dy = gradient(how, rows, outs)
    layer(x).backward(dy)
    got = layer.given[0]
    assert got.shape == dy.shape and torch.equal(got, dy)
    assert got.stride(1) == 1 or rows == 0
    if rows > 1:
        assert got.stride(0) % 8 == 0 and got.stride(0) >= outs
    assert got.data_ptr() % 16 == 0


def test_rows_that_fit_are_not_copied():
    for outs, how in ((96, "dense"), (96, "padded rows"), (100, "padded rows")):
        layer = layer_with("linear", outs)
        x = torch.zeros((5, 16), dtype=BF, requires_grad=True)
        dy = gradient(how, 5, outs)
        layer(x).backward(dy)
        assert layer.given[0].data_ptr() == dy.data_ptr()
