"""A captured step of the generating layer after its weights have changed."""
import pytest
import torch

from fp4_block_scaled_x16_amd import api, attention
from kv_check import DEV

pytestmark = pytest.mark.gpu


def test_a_captured_step_follows_refresh():
    g = torch.Generator().manual_seed(0)
    qkv, out = ((0.06 * torch.randn(s, generator=g)).to(torch.bfloat16).to(DEV) for s in ((8 * 64, 256), (256, 4 * 64)))
    layer = attention.QuantizedAttention(qkv, out, 4, 2)
    cache, eager = (api.KVCache.empty(4, 16, 2, 64, "mxfp8", DEV) for _ in range(2))
    table = torch.arange(4, dtype=torch.int32, device=DEV).view(2, 2)
    x = torch.zeros((2, 256), dtype=torch.bfloat16, device=DEV)
    lens, slots = torch.ones(2, dtype=torch.int32, device=DEV), torch.tensor([0, 32], device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        layer(x, cache, table, lens, slots)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            y = layer(x, cache, table, lens, slots)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(4):
        qkv.copy_(0.06 * torch.randn(8 * 64, 256, generator=g))
        out.copy_(0.06 * torch.randn(256, 4 * 64, generator=g))
        layer.refresh()
        # memory that codes written anew would have left
        other = [torch.full((8 * 64, 256), 0x7F, dtype=torch.uint8, device=DEV) for _ in range(4)]
        x.copy_(torch.randn(2, 256, generator=g))
        lens.fill_(step + 1)
        slots.copy_(torch.tensor([0, 32]) + step)
        graph.replay()
        want = attention.QuantizedAttention(qkv, out, 4, 2)(x, eager, table, lens, slots)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.isfinite(y).all() and y.any()
        del other
