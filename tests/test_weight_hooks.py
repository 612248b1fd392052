"""Hooks on a weight of QuantizedLinear and QuantizedFFN run in the layer's
backward pass, after its gradient has been added to main_grad (from which a
training program learns that it is there), though the weight gets no .grad.
The layers' steps are stood in for by plain products, so this runs on the CPU."""
import pytest
import torch

from fp4_block_scaled_x16_amd.ffn import QuantizedFFN
from fp4_block_scaled_x16_amd.linear import QuantizedLinear, Recipe

BF = torch.bfloat16
R = Recipe(fmt="fp8", out_dtype="bf16")


class PlainLinear(QuantizedLinear):
    def _forward(self, x):
        return x @ self.weight.T, x

    def _backward(self, dy, x):
        self.main_grad += dy.T.float() @ x.float()
        return dy @ self.weight


class PlainFFN(QuantizedFFN):
    """relu2 without its square."""

    def __init__(self, up, down):
        super().__init__(up, down, "relu2", R)
        self.up, self.down = PlainLinear(up, R), PlainLinear(down, R)

    def _forward(self, x):
        h = x @ self.up.weight.T
        return h.clamp(min=0) @ self.down.weight.T, (x, h)

    def _backward(self, dy, saved):
        x, h = saved
        da = self.down._backward(dy, h.clamp(min=0))
        return self.up._backward(da * (h > 0), x)


def leaf(rows, cols):
    return torch.ones((rows, cols), dtype=BF).requires_grad_()


def make(kind):
    up, down = leaf(8, 16), leaf(16, 8)
    if kind == "linear":
        layer = PlainLinear(up, R)
        return layer, [(up, layer)]
    layer = PlainFFN(up, down)
    return layer, [(up, layer.up), (down, layer.down)]


def node_of(w):
    return w.view_as(w).grad_fn.next_functions[0][0]


def register(how, w, heard):
    """(what has to be kept alive, the handle)"""
    if how == "tensor":
        return None, w.register_hook(lambda g: heard())
    if how == "accumulated":
        return None, w.register_post_accumulate_grad_hook(lambda p: heard())
    n = node_of(w)
    return n, (n.register_hook(lambda *a: heard()) if how == "node"
               else n.register_prehook(lambda *a: heard()))


HOOKS = ["tensor", "accumulated", "node", "node before"]


@pytest.mark.parametrize("late", [False, True])
@pytest.mark.parametrize("how", HOOKS)
@pytest.mark.parametrize("kind", ["linear", "ffn"])
def test_a_hook_runs_once_per_step(kind, how, late):
    """Registered before the forward pass, or between it and the backward pass;
    x needs a gradient or none; and no longer once it is removed."""
    layer, weights = make(kind)
    x = torch.ones((4, 16), dtype=BF)
    for wants in (False, True):
        log, keep = [], []
        if late:
            y = layer(x.requires_grad_(wants))
        for w, owner in weights:
            keep.append(register(how, w, lambda w=w, o=owner: log.append((id(w), float(o.main_grad.sum())))))
        if not late:
            y = layer(x.requires_grad_(wants))
        before = {id(w): float(o.main_grad.sum()) for w, o in weights}
        y.backward(torch.ones_like(y))
        assert sorted(k for k, _ in log) == sorted(id(w) for w, _ in weights)
        for k, total in log:
            assert total > before[k]                   # main_grad is there already
        assert all(w.grad is None for w, _ in weights)
        for _, handle in keep:
            handle.remove()
        n = len(log)
        y = layer(x)
        y.backward(torch.ones_like(y))
        assert len(log) == n


def test_a_hook_of_several_weights_runs_when_all_are_done():
    layers = [make("linear") for _ in range(2)]
    done = []
    ws = [w for _, pairs in layers for w, _ in pairs]
    torch.autograd.graph.register_multi_grad_hook(ws, lambda grads: done.append(
        [float(o.main_grad.abs().sum()) for _, pairs in layers for _, o in pairs]))
    x = torch.ones((4, 16), dtype=BF)
    y = sum(layer(x) for layer, _ in layers)
    y.backward(torch.ones_like(y))
    assert len(done) == 1 and all(t > 0 for t in done[0])


def test_gradients_of_the_input_alone():
    """torch.autograd.grad of x does not reach the weights' hooks."""
    layer, weights = make("ffn")
    log = []
    for w, _ in weights:
        register("accumulated", w, lambda: log.append(1))
    x = torch.ones((4, 16), dtype=BF, requires_grad=True)
    y = layer(x)
    torch.autograd.grad(y, x, torch.ones_like(y))
    assert not log


def test_weights_without_gradients_and_steps_without_a_graph():
    layer, weights = make("ffn")
    with torch.no_grad():
        assert not layer(torch.ones((4, 16), dtype=BF)).requires_grad
    for w, _ in weights:
        w.requires_grad_(False)
    assert not layer(torch.ones((4, 16), dtype=BF)).requires_grad


@pytest.mark.parametrize("kind", ["linear", "ffn"])
def test_weights_that_are_frozen_between_the_passes(kind):
    layer, weights = make(kind)
    y = layer(torch.ones((4, 16), dtype=BF))
    for w, _ in weights:
        w.requires_grad_(False)
    y.backward(torch.ones_like(y))
    assert all(float(o.main_grad.sum()) > 0 for _, o in weights)


def test_a_weight_that_is_computed():
    """Its graph is reached without a gradient, step after step, as its hooks are."""
    base = leaf(8, 16)
    w = base * 1
    layer, log = PlainLinear(w, R), []
    w.register_hook(lambda g: log.append(g))
    for n in (1, 2):
        y = layer(torch.ones((4, 16), dtype=BF))
        y.backward(torch.ones_like(y))
        assert log == [None] * n and base.grad is None


@pytest.mark.parametrize("kind", ["linear", "ffn"])
def test_a_weight_that_nobody_listens_to_shares_no_leaf(kind):
    """Its graphs hold leaves of their own, so one that is alive does not tie a
    step that is captured on another stream to its own."""
    layer, weights = make(kind)
    ys = [layer(torch.ones((4, 16), dtype=BF)) for _ in range(2)]
    leaves = [f.variable for y in ys for f, _ in y.grad_fn.next_functions if f is not None]
    assert len({id(t) for t in leaves}) == 2 * len(weights)
    assert all(t is not w for t in leaves for w, _ in weights)
