"""The attention layer: its operators together, as a model that generates calls them --
a prompt, then tokens one by one, in batches with padding, eager and captured."""
import numpy as np
import pytest
import torch

import kv_check as C
from fp4_block_scaled_x16_amd import api, attention
from kv_check import DEV, FORMATS

pytestmark = pytest.mark.gpu
H, KV, D, MODEL, PAGE = 8, 2, 64, 256, 16


def layer_of(norm=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    qkv = (0.06 * torch.randn((H + 2 * KV) * D, MODEL, generator=g)).to(torch.bfloat16).to(DEV)
    out = (0.05 * torch.randn(MODEL, H * D, generator=g)).to(torch.bfloat16).to(DEV)
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2)]
    n = api.QKNorm(*w, attention.rotary_table(128, D, device=DEV)) if norm else None
    return attention.QuantizedAttention(qkv, out, H, KV, n)


def cache_of(fmt, pages=24):
    return C.make_cache(fmt, pages, PAGE, KV, D, amax=(8.0, 5.0))


def by_steps(layer, x, cache, page_table, slots, positions, lens):
    """The same step, from the single operators."""
    n = x.shape[0]
    rows = api.gemm(api.quantize(x, "fp8").operand(), api.quantize(layer.qkv, "fp8", block="2d").operand(), n,
                    layer.qkv.shape[0], MODEL, out_dtype=torch.bfloat16).view(n, H + 2 * KV, D)
    q, k, v = rows[:, :H], rows[:, H:H + KV], rows[:, H + KV:]
    if layer.norm is not None:
        q, _ = api.qk_norm_rope(layer.norm, q, None, positions)
    api.kv_cache_write(cache, k, v, slots, norm=layer.norm, positions=positions)
    o = api.attention_decode(q, cache, page_table, lens)
    return api.gemm(api.quantize(o.view(n, -1), "fp8").operand(), api.quantize(layer.out, "fp8", block="2d").operand(), n,
                    MODEL, H * D, out_dtype=torch.bfloat16), o


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("fmt", FORMATS)
def test_generation(fmt, norm):
    """Three requests with prompts of different lengths, then steps in which one row is
    padding; the last step's attention against attention on the values in the cache."""
    layer, cache, other = layer_of(norm), cache_of(fmt), cache_of(fmt)
    table = torch.randperm(24, generator=torch.Generator().manual_seed(2))[:18].view(3, 6).int().to(DEV)
    lens = [33, 1, 16]
    for r, n in enumerate(lens):
        x = C.rows((n, 1, MODEL), r)[:, 0].to(DEV)
        pos = torch.arange(n, device=DEV)
        t = table[r:r + 1].expand(n, 6)
        args = (t, attention.slots_of(t, pos, PAGE), pos, (pos + 1).int())
        y = layer(x, cache, args[0], args[3], args[1], args[2])
        want, _ = by_steps(layer, x, other, *args)
        assert torch.equal(y, want)
    for step in range(4):
        lens = [n + 1 for n in lens]
        x = C.rows((4, 1, MODEL), 10 + step)[:, 0].to(DEV)
        t = torch.cat([table, torch.full((1, 6), -1, dtype=torch.int32, device=DEV)])
        ln = torch.tensor(lens + [0], dtype=torch.int32, device=DEV)
        pos = torch.tensor(lens + [0], device=DEV) - 1
        slots = attention.slots_of(t, pos, PAGE)
        assert slots[3] == -1
        y = layer(x, cache, t, ln, slots, pos.clamp(min=0))
        want, o = by_steps(layer, x, other, t, slots, pos.clamp(min=0), ln)
        assert torch.equal(y, want) and not y[3].any()
    for a, b in zip(C.contents(cache), C.contents(other)):
        assert np.array_equal(a, b)
    # attention in 64 bits on what the cache holds, of the last step's queries
    rows = api.gemm(api.quantize(x, "fp8").operand(), layer._qkv, 4, layer.qkv.shape[0], MODEL,
                    out_dtype=torch.bfloat16).view(4, H + 2 * KV, D)
    q = rows[:, :H] if layer.norm is None else api.qk_norm_rope(layer.norm, rows[:, :H], None, pos.clamp(min=0))[0]
    for r, n in enumerate(lens):
        at = attention.slots_of(table[r:r + 1].expand(n, 6), torch.arange(n, device=DEV), PAGE)
        k, v = (t.double().repeat_interleave(H // KV, 1) for t in api.kv_cache_read(cache, at, torch.float32))
        p = torch.softmax((k * q[r].double()).sum(-1) / D ** 0.5, 0)
        ref = (p.unsqueeze(-1) * v).sum(0)
        # bf16's half step of the output, and 2^-12 of the values for the scores' fp32 steps
        assert torch.all((o[r].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -12 * v.abs().amax())


def test_captured_steps():
    """One step captured and replayed for several tokens: lengths, slots, positions and
    the page table change in place."""
    layer, cache, eager = layer_of(), cache_of("mxfp8"), cache_of("mxfp8")
    table = torch.arange(12, dtype=torch.int32, device=DEV).view(2, 6)
    x = torch.zeros((2, MODEL), dtype=torch.bfloat16, device=DEV)
    lens = torch.ones(2, dtype=torch.int32, device=DEV)
    slots, pos = torch.zeros(2, dtype=torch.int64, device=DEV), torch.zeros(2, dtype=torch.int64, device=DEV)
    slots.copy_(torch.tensor([0, 96]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        layer(x, cache, table, lens, slots, pos)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            y = layer(x, cache, table, lens, slots, pos)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(40):
        x.copy_(C.rows((2, 1, MODEL), step)[:, 0])
        pos.fill_(step)
        lens.fill_(step + 1)
        slots.copy_(attention.slots_of(table, pos, PAGE))
        graph.replay()
        want = layer(x, eager, table, lens, slots, pos)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_changed_weights_are_encoded_by_refresh():
    layer, cache = layer_of(), cache_of("fp8")
    t, one = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    x, at = C.rows((1, 1, MODEL), 1)[:, 0].to(DEV), torch.zeros(1, dtype=torch.int64, device=DEV)
    y = layer(x, cache, t, one, at, at)
    layer.out.mul_(2)
    assert torch.equal(layer(x, cache, t, one, at, at), y)
    layer.refresh()
    assert torch.equal(layer(x, cache, t, one, at, at), (2 * y.float()).to(torch.bfloat16))
