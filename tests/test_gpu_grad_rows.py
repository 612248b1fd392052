"""Backward passes of the layers under autograd with output features that are no
multiple of 8 and gradients of any layout, against the explicit steps on the
same gradient in aligned rows."""
import pytest
import torch

from fp4_block_scaled_x16_amd.ffn import QuantizedFFN
from fp4_block_scaled_x16_amd.linear import QuantizedLinear, Recipe

pytestmark = pytest.mark.gpu
DEV = "cuda"
R = Recipe(fmt="fp8", out_dtype="bf16")


def rand(rows, cols, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, cols), generator=g) * sigma).to(torch.bfloat16).to(DEV)


def aligned(v):
    g = torch.zeros((v.shape[0], -(-v.shape[1] // 8) * 8 + 8), dtype=v.dtype, device=DEV)[:, :v.shape[1]]
    return g.copy_(v)


def layouts(v):
    yield v
    yield aligned(v)
    yield v.t().contiguous().t()
    odd = torch.zeros((v.shape[0], v.shape[1] + 3), dtype=v.dtype, device=DEV)[:, 1:v.shape[1] + 1]
    yield odd.copy_(v)


def check(make, grads_of, x, dy):
    one = make()
    y = one.forward(x)
    want = (y, one.backward(aligned(dy)), *grads_of(one))
    for g in layouts(dy):
        layer, leaf = make(), x.clone().requires_grad_()
        y = layer(leaf)
        y.backward(g)
        for got, ref in zip((y, leaf.grad, *grads_of(layer)), want):
            assert torch.equal(got, ref)


@pytest.mark.parametrize("T,O", [(1, 100), (2, 1), (70, 100), (33, 257), (40, 96)])
def test_linear(T, O):
    w = rand(O, 264, 1, 0.05)
    check(lambda: QuantizedLinear(w, R), lambda l: (l.main_grad,), rand(T, 264, 2), rand(T, O, 3, 1e-3))


@pytest.mark.parametrize("act,T,O", [("relu2", 70, 100), ("swiglu", 5, 33)])
def test_ffn(act, T, O):
    up, down = rand(256 if act == "swiglu" else 128, 64, 1, 0.1), rand(O, 128, 2, 0.1)
    check(lambda: QuantizedFFN(up, down, act), lambda l: (l.up.main_grad, l.down.main_grad),
          rand(T, 64, 3), rand(T, O, 4, 1e-2))


def test_nvfp4_linear():
    """Its own sizes are aligned already; the layouts are not."""
    w, r = rand(96, 128, 1, 0.05), Recipe(fmt="nvfp4", out_dtype="bf16")
    check(lambda: QuantizedLinear(w, r), lambda l: (l.main_grad,), rand(64, 128, 2), rand(64, 96, 3, 1e-3))


def test_a_sum():
    """The gradient of y.sum() is one number for every element."""
    w = rand(100, 64, 1, 0.05)
    layer, one = QuantizedLinear(w, R), QuantizedLinear(w, R)
    x = rand(20, 64, 2)
    layer(x.requires_grad_()).sum().backward()
    one.forward(x.detach())
    dx = one.backward(aligned(torch.ones((20, 100), dtype=torch.bfloat16, device=DEV)))
    assert torch.equal(x.grad, dx) and torch.equal(layer.main_grad, one.main_grad)
