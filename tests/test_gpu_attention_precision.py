"""Attention's probabilities meet V whole: two tokens, of which the first has score 0 and
zeros, the second score -c and ones, so that the output is p / (1 + p), p = e^-c."""
import numpy as np
import pytest
import torch

from fp4_block_scaled_x16_amd import api
from kv_check import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("d,heads,group", [(64, 1, 16), (64, 2, 3), (128, 1, 8), (128, 2, 12), (256, 1, 4), (256, 1, 9)])
@pytest.mark.parametrize("requests,width", [(600, 1), (600, 80), (20, 1), (20, 30), (20, 300)])
def test_probabilities_are_not_rounded(fmt, d, heads, group, requests, width):
    cache = api.KVCache.empty(width, 16, heads, d, fmt, DEV)
    kv = torch.zeros((2, 2, heads, d), dtype=torch.bfloat16, device=DEV)
    kv[0, 1, :, 5] = -1
    kv[1, 1] = 1
    api.kv_cache_write(cache, kv[0], kv[1], torch.arange(2, device=DEV))
    n = requests * heads * group
    c = (0.1 + 3.9 * torch.rand(n, generator=torch.Generator().manual_seed(1))).to(torch.bfloat16)
    q = torch.zeros((requests, heads * group, d), dtype=torch.bfloat16, device=DEV)
    q[..., 5] = c.view(requests, -1).to(DEV)
    table = torch.arange(width, dtype=torch.int32, device=DEV).expand(requests, width)
    lens = torch.full((requests,), 2, dtype=torch.int32, device=DEV)
    out = api.attention_decode(q, cache, table, lens, scale=1.0, out_dtype=torch.float32).cpu().double().numpy()
    p = np.exp(-c.double().numpy()).reshape(requests, -1, 1)
    want = p / (1 + p)
    # scores and products with V are exact.  The exponent, c log2(e) with c up to 4: the constant's and
    # the product's rounding, 8 x 2^-24 of p; the power of two 2 (an ulp); 1 + p, its reciprocal (an ulp) and
    # the last product 4: 14 in all
    assert np.all(np.abs(out - want) <= 14 * 2.0 ** -24 * want)
