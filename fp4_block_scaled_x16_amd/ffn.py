"""A feed-forward layer on quantized linears with an 8-bit activation checkpoint.

  forward(X)    h = X W_up^T           bf16 [tokens, 2F] ("swiglu") or [tokens, F]
                a = act(h)             silu(g) u of h = [g | u], or max(h, 0)^2
                Y = a W_down^T
  backward(dY)  da = dY W_down         bf16 [tokens, F]
                dh from da at the values of h's checkpoint
                dX = dh W_up; the two weight gradients

Between the passes the layer keeps h as E4M3 codes (a byte per element and a
scale per 128; bf16 h and a would be 6 bytes per element of a with SwiGLU, the
codes are 2) beside what the linears keep.  With Recipe(fmt="fp8") every edge
between the products is codes: one kernel turns h into a's codes and the
checkpoint, one turns da and the checkpoint into the codes of dh along rows and
columns and of a along columns -- a's own operand for Wgrad is made anew from
the checkpoint, so the forward pass keeps none.  With an FP4 recipe the
activation passes bf16 values between its linears.

The gradient is that of the layer at the checkpoint's h, as the linears' are
those of their encoded operands.  X, dY, Y and dX are bf16; weight gradients
accumulate into the two layers' fp32 main_grad.  Calling the layer runs it under
autograd (the weights get no .grad); `forward` / `backward` are the same steps.
Both may be captured into a graph; under autograd the captured x should be no
leaf of an eager graph that is still alive (a leaf keeps its first stream).
"""
from __future__ import annotations

import torch

from . import api
from .linear import Kept, QuantizedLinear, Recipe, grad_alias, grad_rows, reach_hooks


class QuantizedFFN:
    """up: bf16 [2F, D] ("swiglu", the gate's rows first) or [F, D] ("relu2");
    down: bf16 [D_out, F] device tensors.  recipe.out_dtype must be "bf16"."""

    def __init__(self, up: torch.Tensor, down: torch.Tensor, act="swiglu",
                 recipe: Recipe = Recipe(fmt="fp8", out_dtype="bf16")):
        if act not in api.ACTS:
            raise ValueError("act must be one of %s" % (tuple(api.ACTS),))
        if recipe.out_dtype != "bf16":
            raise ValueError("the layer needs Recipe(out_dtype='bf16')")
        self.up, self.down = QuantizedLinear(up, recipe), QuantizedLinear(down, recipe)
        self.act, self.recipe = act, recipe
        self.features = self.down.in_features
        if self.up.out_features != self.features * (2 if act == "swiglu" else 1):
            raise ValueError("up must have %s rows for down's %d columns"
                             % ("2F" if act == "swiglu" else "F", self.features))
        if self.features % (128 if act == "swiglu" and recipe.fmt == "fp8" else 8):
            # rows of h and da are 16-byte aligned; SwiGLU's codes of dh start u at
            # a whole block, and those of W_up^T have no gap there
            raise ValueError("F must be a multiple of 8 (SwiGLU with fp8: of 128)")
        self._saved = None

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        return _FfnFunction.apply(x, grad_alias(self.up.weight), grad_alias(self.down.weight), self)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        y, saved = self._forward(x)
        self._saved = Kept(saved, x.device)
        return y

    def backward(self, dy: torch.Tensor) -> torch.Tensor:
        if self._saved is None:
            raise RuntimeError("backward() needs a preceding forward()")
        saved, self._saved = self._saved.take(), None
        return self._backward(dy, saved)

    def _forward(self, x):
        h, up = self.up._forward(x)
        if self.recipe.fmt == "fp8":
            qa, qh = api.act_quantize(h, self.act)
            y, down = self.down._fprop_fp8(qa, torch.bfloat16)
        else:
            a, qh = api.act_quantize(h, self.act, a="bf16")
            y, down = self.down._forward(a)
        return y, (up, qh, down)

    def _backward(self, dy, saved):
        up, qh, down = saved
        r = self.recipe
        if r.fmt != "fp8":
            dh, _ = api.act_backward(qh, self.down._backward(dy, down), self.act, out="bf16")
            return self.up._backward(dh, up)
        if dy.dim() != 2 or tuple(dy.shape) != (qh.rows, self.down.out_features):
            raise ValueError("dy must be [tokens, out_features]")
        qdy, qdy_t = api.quantize_dual(dy, r.grad_fmt, counters=self.down.counters)
        da = self.down._dgrad_fp8(qdy, down, torch.bfloat16)
        qdh, qdh_t, qa_t = api.act_backward(qh, da, self.act, fmt=r.grad_fmt)
        self.down._wgrad_fp8(qdy_t, qa_t)
        qx, qw_t, _ = up
        dx = self.up._dgrad_fp8(qdh, qw_t, torch.bfloat16)
        self.up._wgrad_fp8(qdh_t, api.requantize_t(qx) if r.checkpoint8 else qx)
        return dx


class _FfnFunction(torch.autograd.Function):
    """Autograd wrapper of one QuantizedFFN step (as the linear's: the weight
    gradients go to main_grad)."""

    @staticmethod
    def forward(ctx, x, up, down, layer):
        y, ctx.saved = layer._forward(x)
        ctx.layer, ctx.weights = layer, ((layer.up.weight, up), (layer.down.weight, down))
        return y

    @staticmethod
    def backward(ctx, dy):
        if ctx.saved is None:
            raise RuntimeError("a step's operands are freed by its first backward pass")
        saved, ctx.saved = ctx.saved, None
        dx = ctx.layer._backward(grad_rows(dy), saved)
        for weight, alias in ctx.weights:
            reach_hooks(weight, alias)
        return dx, None, None, None
