"""Attention around a quantized key-value cache.

  rotary_table   the cosines and sines that positions are rotated by
  QKNormRope     norm of each head of queries and keys and rotation by position,
                 under autograd (training)
  slots_of       the cache slots of new tokens, from a page table
  QuantizedAttention  an attention layer that generates tokens: FP8 projections around
                 norm, rotation, a cache of 8- or 4-bit codes, and attention on it

The layer's step, for one new token of each request:

  [q | k | v] = x W_qkv^T       FP8 operands, bf16 out
  q, cache    = norm and rotation of q and k; k and v encoded into their slots
  o           = softmax(q K^T / sqrt(d)) V over the request's cached tokens
  y           = o W_out^T       FP8 operands, bf16 out

The layers' computations run in the library's kernels; this module allocates outputs
and passes pointers (through `api`).  `rotary_table` and `slots_of` are torch operations,
made once and about ten small ones a step.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import api
from .linear import grad_alias, reach_hooks


def rotary_table(positions, rotary_dim, theta=10000.0, device="cuda"):
    """float32 [positions, rotary_dim]: the cosines and then the sines of the angles
    p * theta^(-2 i / rotary_dim), formed in 64 bits (in 32 the angle of a far
    position is wrong in its leading digits)."""
    i = torch.arange(rotary_dim // 2, dtype=torch.float64, device=device)
    a = (torch.arange(positions, dtype=torch.float64, device=device).unsqueeze(1)
         * torch.exp(i * (-2.0 / rotary_dim * torch.log(torch.tensor(theta, dtype=torch.float64)).item())))
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


def slots_of(page_table, positions, page_size):
    """int64 [n]: the slot of position positions[i] of request i (int64; its entry of
    the int32 [n, width] page table), -1 for a position that is negative or has no
    page."""
    if page_table.shape[1] == 0:
        return torch.full_like(positions, -1)
    page = positions // page_size
    there = (positions >= 0) & (page < page_table.shape[1])
    entry = page_table.gather(1, torch.where(there, page, 0).unsqueeze(1)).squeeze(1).long()
    return torch.where(there & (entry >= 0), entry * page_size + positions % page_size, -1)


def _grad_heads(dy):
    """A gradient as the library takes rows of heads: autograd's may be of any layout."""
    t, h, _ = dy.shape
    if (dy.stride(2) == 1 and dy.data_ptr() % 16 == 0 and (t < 2 or dy.stride(0) % 8 == 0)
            and (h < 2 or dy.stride(1) % 8 == 0)):
        return dy
    return dy.contiguous()


class QKNormRope:
    """q, k -> both normed and rotated (`api.QKNorm`), under autograd; either may be
    None, and its result then is.

    As with the linears, the gradients of the weights are added to main_grad
    (float32 [2, head_dim]: q's, then k's; zero it between optimizer steps), whether the
    weights require one or not, and the weights get no .grad; hooks on them run in the
    backward pass.  Weights or a table changed in place between the two passes are refused
    there, as is a gradient of the gradient.  A step may be captured into a graph; the
    captured q and k should be no leaves of an eager graph that is still alive (a leaf keeps
    its first stream).
    """

    def __init__(self, q_weight=None, k_weight=None, table=None, eps=1e-6, style="half"):
        data = [None if w is None else w.detach() for w in (q_weight, k_weight)]
        self.norm = api.QKNorm(*data, table, eps, style)
        self.weights = () if q_weight is None else (q_weight, k_weight)
        self.main_grad = (None if q_weight is None else
                          torch.zeros((2, q_weight.shape[0]), dtype=torch.float32, device=q_weight.device))

    def __call__(self, q, k, positions=None):
        n = self.norm
        if self.weights and [w.data_ptr() for w in self.weights] != [n.q_weight.data_ptr(), n.k_weight.data_ptr()]:
            # the weights' .data has been replaced
            self.norm = api.QKNorm(*(w.detach() for w in self.weights), n.table, n.eps, n.style)
        return _QKNormRopeFunction.apply(q, k, positions, self, *(grad_alias(w) for w in self.weights))


class _QKNormRopeFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, layer, *aliases):
        table = layer.norm.table
        if table is not None and table.is_inference():         # which has no versions, and is not saved
            table = None
        # the table and the weights for the check of their versions
        ctx.save_for_backward(q, k, positions, table, *aliases)
        ctx.layer, ctx.norm, ctx.aliases = layer, layer.norm, aliases
        return api.qk_norm_rope(layer.norm, q, k, positions)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        layer = ctx.layer
        q, k, positions, *_ = ctx.saved_tensors
        dq, dk, _, _ = api.qk_norm_rope_backward(
            ctx.norm, q, k, positions, None if q is None else _grad_heads(dq),
            None if k is None else _grad_heads(dk),
            weight_grads=False if layer.main_grad is None else layer.main_grad)
        for weight, alias in zip(layer.weights, ctx.aliases):
            reach_hooks(weight, alias)
        return dq, dk, None, None, *(None for _ in ctx.aliases)


class _NoGradient(torch.autograd.Function):
    """The y of (y,), computed from x in a way that has no backward pass (the tuple keeps
    it from being an input, and the output a view of it that cannot be changed in place)."""

    @staticmethod
    def forward(ctx, x, made):
        return made[0]

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("QuantizedAttention has no backward pass: it generates")


class QuantizedAttention:
    """The attention layer of a model that generates: one new token per request.

    qkv: bf16 [(heads + 2 kv_heads) * head_dim, D], the rows of all query heads, then
    keys, then values; out: bf16 [D_out, heads * head_dim].  Both are encoded once, in FP8
    128x128 blocks (`refresh` after they have changed).  norm: an `api.QKNorm` for
    queries and keys, or None.  scale: of the scores, 1 / sqrt(head_dim) if None.

    A prompt goes through the same call, a token per row: rows of one request share
    its page table's row (which may be expanded) and have lengths that count up.
    There is no backward pass: one that comes to the layer's output fails.
    """

    def __init__(self, qkv, out, heads, kv_heads, norm: api.QKNorm = None, scale=None):
        rows = heads + 2 * kv_heads
        if heads % kv_heads or qkv.shape[0] % rows:
            raise ValueError("qkv must have (heads + 2 kv_heads) * head_dim rows, heads a multiple of kv_heads")
        self.head_dim = qkv.shape[0] // rows
        if self.head_dim not in api.HEAD_DIMS:
            raise ValueError("head_dim must be one of %s, not %d" % (api.HEAD_DIMS, self.head_dim))
        if out.shape[1] != heads * self.head_dim:
            raise ValueError("out must have heads * head_dim = %d columns" % (heads * self.head_dim))
        self.qkv, self.out, self.heads, self.kv_heads = qkv, out, heads, kv_heads
        self.norm, self.scale = norm, scale
        self._qkv = self._out = None
        self.refresh()

    def refresh(self):
        """Encode the weights anew, where their codes are: a step that has been captured
        takes the new ones.  To be called on the stream that the steps run on."""
        self._qkv, self._out = self._encoded(self.qkv, self._qkv), self._encoded(self.out, self._out)

    @staticmethod
    def _encoded(w, old):
        new = api.quantize(w, "fp8", block="2d")
        into = None if old is None else old._owner
        if into is None or into.codes.shape != new.codes.shape or into.codes.device != new.codes.device:
            return new.operand()
        with torch.inference_mode():             # (they may have been made in it)
            into.codes.copy_(new.codes)
            into.scales.copy_(new.scales)
        return old

    @staticmethod
    def _product(x, w, n):
        return api.gemm(api.quantize(x, "fp8").operand(), w, x.shape[0], n, x.shape[1], out_dtype=torch.bfloat16)

    def __call__(self, x, cache: api.KVCache, page_table, lens, slots, positions=None):
        """bf16 [tokens, D_out] of new tokens x (bf16 [tokens, D]).

        slots: int64 [tokens], where each one's key and value go (`slots_of`); lens:
        int32 [tokens], its request's length with the token itself; positions: int64
        [tokens], for the norm's rotation."""
        if x.dim() != 2 or x.shape[1] != self.qkv.shape[1]:
            raise ValueError("x must be [tokens, %d]" % self.qkv.shape[1])
        tokens, h, kv = x.shape[0], self.heads, self.kv_heads
        rows = self._product(x, self._qkv, self.qkv.shape[0]).view(tokens, h + 2 * kv, self.head_dim)
        q, k, v = rows[:, :h], rows[:, h:h + kv], rows[:, h + kv:]
        if self.norm is None:
            api.kv_cache_write(cache, k, v, slots)
        else:
            # in place: the projection's rows are nobody else's
            q = api.kv_cache_write(cache, k, v, slots, q=q, norm=self.norm, positions=positions, q_out=q)
        o = api.attention_decode(q, cache, page_table, lens, self.scale)
        y = self._product(o.view(tokens, h * self.head_dim), self._out, self.out.shape[0])
        return _NoGradient.apply(x, (y,)) if x.requires_grad and torch.is_grad_enabled() else y
