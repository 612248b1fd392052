"""The FP8 linear and the feed-forward layer, as a training program runs them:
against the operators called one by one, against the same layer in 64 bits on
unquantized values, under autograd, and their steps captured into graphs."""
import numpy as np
import pytest
import torch

from fp4_block_scaled_x16_amd import api
from fp4_block_scaled_x16_amd.ffn import QuantizedFFN
from fp4_block_scaled_x16_amd.linear import QuantizedLinear, Recipe
from fp8_check import DEV, as64, bf16
from oracle import fp8

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rand(rows, cols, seed, sigma=1.0):
    return bf16(np.random.default_rng(seed).standard_normal((rows, cols)) * sigma).to(DEV)


def rel(got, want):
    return np.linalg.norm(as64(got) - want) / np.linalg.norm(want)


@pytest.mark.parametrize("checkpoint8", [True, False])
@pytest.mark.parametrize("grad_fmt", ["fp8", "fp8_e5m2"])
@pytest.mark.parametrize("T,I,O", [(1, 128, 256), (70, 264, 136), (300, 512, 384)])
def test_linear(T, I, O, grad_fmt, checkpoint8):
    w = rand(O, I, 1, 0.05)
    layer = QuantizedLinear(w, Recipe(fmt="fp8", out_dtype="bf16", grad_fmt=grad_fmt,
                                      checkpoint8=checkpoint8))
    grad = torch.zeros((O, I), device=DEV)
    want_dw = np.zeros((O, I))
    for step in range(2):
        x, dy = rand(T, I, 10 + step), rand(T, O, 20 + step, 1e-3)
        y = layer.forward(x)
        dx = layer.backward(dy)
        qx, (qw, qwt) = api.quantize(x, "fp8"), api.quantize_dual(w, "fp8", block="2d")
        qdy, qdyt = api.quantize_dual(dy, grad_fmt)
        qxt = api.requantize_t(qx) if checkpoint8 else api.quantize(x, "fp8", orient="col")
        assert torch.equal(y, api.gemm(qx.operand(), qw.operand(), T, O, I, out_dtype=BF))
        assert torch.equal(dx, api.gemm(qdy.operand(), qwt.operand(), T, I, O, out_dtype=BF))
        api.gemm(qdyt.operand(), qxt.operand(), O, I, T, out=grad, accumulate=True)
        want_dw += as64(dy).T @ as64(x)
        # two operands, each element within 2^-4 (E5M2: 2^-3) of itself, signs at
        # random: far less in the norm than their sum
        eps = 2.0 ** -4 + (2.0 ** -3 if grad_fmt == "fp8_e5m2" else 2.0 ** -4)
        assert rel(y, as64(x) @ as64(w).T) < 2.0 ** -3
        assert rel(dx, as64(dy) @ as64(w)) < eps
        assert rel(layer.main_grad, want_dw) < eps
    assert torch.equal(layer.main_grad, grad) and layer.step == 2


def plain_ffn(x, up, down, act, dy):
    """Y, dX and the two weight gradients in 64 bits."""
    h = x @ up.T
    a = fp8.act(h, act)
    da = dy @ down
    dh = fp8.act_grad(h, da, act)
    return a @ down.T, dh @ up, dh.T @ x, dy.T @ a


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("act,T,D,F", [("swiglu", 96, 256, 384), ("relu2", 64, 128, 264),
                                       ("relu2", 1, 128, 256), ("swiglu", 272, 128, 128)])
def test_ffn(act, T, D, F, fmt):
    if fmt == "nvfp4" and (T % 16 or F % 16):
        pytest.skip("NVFP4 blocks")
    up, down = rand((2 if act == "swiglu" else 1) * F, D, 1, D ** -0.5), rand(D, F, 2, F ** -0.5)
    layer = QuantizedFFN(up, down, act, Recipe(fmt=fmt, out_dtype="bf16"))
    x, dy = rand(T, D, 3), rand(T, D, 4, 1e-2)
    y = layer.forward(x)
    dx = layer.backward(dy)
    want = plain_ffn(*(as64(t) for t in (x, up, down)), act, as64(dy))
    # three roundings in a chain (operands, h's checkpoint, a or dh); elements
    # within 2^-4 of themselves in E4M3, 2^-3 in E5M2, 2^-2 in E2M1
    tol = 3 * (2.0 ** -3 if fmt == "fp8" else 2.0 ** -2)
    for got, ref in zip((y, dx, layer.up.main_grad, layer.down.main_grad), want):
        assert rel(got, ref) < tol
    if fmt != "fp8":
        return
    # the operators one by one
    qx, (qu, qut), (qd, qdt) = (api.quantize(x, "fp8"), api.quantize_dual(up, "fp8", block="2d"),
                                api.quantize_dual(down, "fp8", block="2d"))
    h = api.gemm(qx.operand(), qu.operand(), T, up.shape[0], D, out_dtype=BF)
    qa, qh = api.act_quantize(h, act)
    assert torch.equal(y, api.gemm(qa.operand(), qd.operand(), T, D, F, out_dtype=BF))
    qdy, qdyt = api.quantize_dual(dy, "fp8_e5m2")
    da = api.gemm(qdy.operand(), qdt.operand(), T, F, D, out_dtype=BF)
    qdh, qdht, qat = api.act_backward(qh, da, act, fmt="fp8_e5m2")
    assert torch.equal(dx, api.gemm(qdh.operand(), qut.operand(), T, D, qdh.cols, out_dtype=BF))
    dw = api.gemm(qdyt.operand(), qat.operand(), D, F, T)
    assert torch.equal(layer.down.main_grad, dw)
    du = api.gemm(qdht.operand(), api.requantize_t(qx).operand(), up.shape[0], D, T)
    assert torch.equal(layer.up.main_grad, du)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_autograd_matches_the_explicit_steps(fmt):
    T, D, F = 64, 128, 256
    up, down = rand(2 * F, D, 1, 0.1), rand(D, F, 2, 0.1)
    x, dy = rand(T, D, 3), rand(T, D, 4, 1e-2)
    a = QuantizedFFN(up, down, "swiglu", Recipe(fmt=fmt, out_dtype="bf16"))
    b = QuantizedFFN(up, down, "swiglu", Recipe(fmt=fmt, out_dtype="bf16"))
    y, dx = a.forward(x), a.backward(dy)
    xb = x.clone().requires_grad_()
    yb = b(xb)
    yb.backward(dy)
    assert torch.equal(y, yb) and torch.equal(dx, xb.grad)
    assert torch.equal(a.up.main_grad, b.up.main_grad)
    assert torch.equal(a.down.main_grad, b.down.main_grad)


def test_two_steps_in_flight():
    """Two micro-batches whose backward passes come in the other order: each
    keeps its own operands (autograd holds them)."""
    T, D, F = 48, 128, 128
    up, down = rand(2 * F, D, 1, 0.1), rand(D, F, 2, 0.1)
    make = lambda: QuantizedFFN(up, down, "swiglu")          # noqa: E731
    xs, dys = [rand(T, D, k) for k in (3, 4)], [rand(T, D, k, 1e-2) for k in (5, 6)]
    want = []
    for x, dy in zip(xs, dys):
        one = make()
        one.forward(x)
        want.append(one.backward(dy))
    layer = make()
    leaves = [x.clone().requires_grad_() for x in xs]
    ys = [layer(x) for x in leaves]
    for k in (1, 0):
        ys[k].backward(dys[k])
    for leaf, dx in zip(leaves, want):
        assert torch.equal(leaf.grad, dx)


def test_a_captured_training_step():
    """Forward and backward of the layer (explicit steps) in one graph, replayed
    on new inputs with eager steps between, against eager steps."""
    T, D, F = 130, 256, 256
    up, down = rand(2 * F, D, 1, 0.06), rand(D, F, 2, 0.06)
    xs, dys = [rand(T, D, k) for k in range(3, 6)], [rand(T, D, k, 1e-2) for k in range(6, 9)]

    def eager(k):
        one = QuantizedFFN(up, down, "swiglu")
        y = one.forward(xs[k])
        return y, one.backward(dys[k]), one.up.main_grad, one.down.main_grad

    want = [eager(k) for k in range(3)]
    layer = QuantizedFFN(up, down, "swiglu")
    x, dy = xs[0].clone(), dys[0].clone()
    layer.forward(x)
    layer.backward(dy)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer.forward(x)
        dx = layer.backward(dy)
    for k in (1, 2, 0, 1):
        x.copy_(xs[k])
        dy.copy_(dys[k])
        layer.up.main_grad.zero_()
        layer.down.main_grad.zero_()
        g.replay()
        eager(2 - k)
        torch.cuda.synchronize()
        for got, ref in zip((y, dx, layer.up.main_grad, layer.down.main_grad), want[k]):
            assert torch.equal(got, ref)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_the_graph_has_no_leaf_of_the_weights(fmt):
    """Two steps share no autograd leaf (which would carry the first step's
    stream into the second), and weights that want gradients make the output
    want one."""
    leaves = []
    up, down = (t.requires_grad_() for t in (rand(256, 128, 1, 0.1), rand(128, 128, 2, 0.1)))
    r = Recipe(fmt=fmt, out_dtype="bf16")
    ffn, linear = QuantizedFFN(up, down, "swiglu", r), QuantizedLinear(up, r)
    for layer in (ffn, linear):
        ys = [layer(rand(32, 128, k)) for k in (3, 4)]
        leaves += [f.variable for y in ys for f, _ in y.grad_fn.next_functions if f is not None]
    assert len(leaves) == 6 and len({id(t) for t in leaves}) == 6
    assert all(t is not up and t is not down for t in leaves)
    for y in ys:
        y.backward(torch.ones_like(y))
        with pytest.raises(RuntimeError):
            y.grad_fn.apply(torch.ones_like(y))
    assert up.grad is None and not QuantizedLinear(up.detach(), r)(rand(32, 128, 5)).requires_grad


def test_autograd_captured_beside_an_eager_step():
    """Weights that want gradients, an eager step whose graph is still alive, and
    a captured forward and backward of the same layer."""
    T, D, F = 64, 128, 128
    up, down = (t.requires_grad_() for t in (rand(2 * F, D, 1, 0.1), rand(D, F, 2, 0.1)))
    layer = QuantizedFFN(up, down, "swiglu")
    xs, dy = [rand(T, D, k) for k in (3, 4)], rand(T, D, 5, 1e-2)
    want = []
    for x in xs:
        one = QuantizedFFN(up, down, "swiglu")
        want.append((one.forward(x), one.backward(dy), one.up.main_grad, one.down.main_grad)[0::2])
    alive = layer(xs[0])
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = layer(x)
        y.backward(dy)
    for k in (1, 0, 1):
        x.copy_(xs[k])
        layer.up.main_grad.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[k][0]) and torch.equal(layer.up.main_grad, want[k][1])
    layer.up.main_grad.zero_()
    alive.backward(dy)
    assert torch.equal(layer.up.main_grad, want[0][1])


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
def test_no_tokens(act):
    up, down = rand(256 if act == "swiglu" else 128, 128, 1), rand(64, 128, 2)
    layer = QuantizedFFN(up, down, act)
    x = torch.empty((0, 128), dtype=BF, device=DEV)
    assert layer.forward(x).shape == (0, 64)
    assert layer.backward(torch.empty((0, 64), dtype=BF, device=DEV)).shape == (0, 128)
    assert not layer.up.main_grad.any() and not layer.down.main_grad.any()


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_backward_on_another_stream(fmt):
    """The forward pass on one stream, the backward pass on another that waits
    for it, and the first stream filling new memory meanwhile: what the step
    kept is not handed out while it is read."""
    T, D, F = 2048, 512, 512
    up, down = rand(2 * F, D, 1, 0.05), rand(D, F, 2, 0.05)
    x, dy = rand(T, D, 3), rand(T, D, 4, 1e-2)
    r = Recipe(fmt=fmt, out_dtype="bf16")
    one = QuantizedFFN(up, down, "swiglu", r)
    one.forward(x)
    want = one.backward(dy), one.up.main_grad, one.down.main_grad
    layer = QuantizedFFN(up, down, "swiglu", r)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        layer.forward(x)
    b.wait_stream(a)
    with torch.cuda.stream(b):
        torch.cuda._sleep(1_000_000)             # the first stream is ahead
        dx = layer.backward(dy)
    with torch.cuda.stream(a):
        junk = [torch.full((T, n), 0xFF, dtype=torch.uint8, device=DEV) for n in (512, 512, 1024, 2048) * 4]
    torch.cuda.synchronize()
    for got, ref in zip((dx, layer.up.main_grad, layer.down.main_grad), want):
        assert torch.equal(got, ref)
    del junk
