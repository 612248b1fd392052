"""Hooks on the weights of the layers, with the real steps: eager, on a stream
of its own, and beside a captured step."""
import pytest
import torch

from fp4_block_scaled_x16_amd.ffn import QuantizedFFN
from fp4_block_scaled_x16_amd.linear import QuantizedLinear, Recipe

pytestmark = pytest.mark.gpu
DEV = "cuda"


def rand(rows, cols, seed, sigma=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, cols), generator=g) * sigma).to(torch.bfloat16).to(DEV)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("late", [False, True])
def test_hooks_see_main_grad(fmt, late):
    T, D, F = 64, 128, 128
    r = Recipe(fmt=fmt, out_dtype="bf16")
    up, down = (t.requires_grad_() for t in (rand(2 * F, D, 1, 0.1), rand(D, F, 2, 0.1)))
    x, dy = rand(T, D, 3), rand(T, D, 4, 1e-2)
    one = QuantizedFFN(up.detach(), down.detach(), "swiglu", r)
    one.forward(x)
    one.backward(dy)
    layer, seen = QuantizedFFN(up, down, "swiglu", r), {}

    def listen():
        for w, o in ((up, layer.up), (down, layer.down)):
            w.register_post_accumulate_grad_hook(lambda p, o=o: seen.update({id(p): o.main_grad.clone()}))

    with torch.cuda.stream(torch.cuda.Stream()):
        if not late:
            listen()
        y = layer(x)
        if late:
            listen()
        y.backward(dy)
    torch.cuda.synchronize()
    assert torch.equal(seen[id(up)], one.up.main_grad) and torch.equal(seen[id(down)], one.down.main_grad)
    assert up.grad is None and down.grad is None


def test_a_captured_step_beside_a_hooked_one():
    """An eager graph that holds the weight itself (its hook waits) is alive while
    a step of the layer is captured: the captured one has a leaf of its own and
    runs no hook."""
    T, D, O = 64, 128, 256
    r = Recipe(fmt="fp8", out_dtype="bf16")
    w = rand(O, D, 1, 0.1).requires_grad_()
    layer, runs = QuantizedLinear(w, r), []
    w.register_post_accumulate_grad_hook(lambda p: runs.append(1))
    xs, dy = [rand(T, D, k) for k in (3, 4)], rand(T, O, 5, 1e-2)
    want = []
    for x in xs:
        one = QuantizedLinear(w.detach(), r)
        y = one.forward(x)
        one.backward(dy)
        want.append((y, one.main_grad))
    alive = layer(xs[0])
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer(x)
        y.backward(dy)
    assert not runs
    for k in (1, 0, 1):
        x.copy_(xs[k])
        layer.main_grad.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k][0]) and torch.equal(layer.main_grad, want[k][1])
    layer.main_grad.zero_()
    alive.backward(dy)
    assert torch.equal(layer.main_grad, want[0][1]) and len(runs) == 1
