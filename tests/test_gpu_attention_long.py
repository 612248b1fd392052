"""Attention of contexts so long that a request's parts pass 2^19 tokens: a few pages, each
named again and again by a page table that all requests share, against 64 bits on the tokens
that differ, each counted as often as it is named."""
import pytest
import torch

from fp4_block_scaled_x16_amd import api
from kv_check import DEV

pytestmark = pytest.mark.gpu
PAGE, PAGES = 1024, 8
M = 1 << 20


@pytest.mark.parametrize("kv,group,d,lens", [
    (8, 4, 128, [3 * M // 2] * 33),
    (8, 1, 128, [3 * M] * 40),
    (8, 2, 128, [3 * M // 2 - 77] * 20 + [5 * M // 2 + 1001] * 20),
    (16, 2, 128, [3 * M // 2] * 17),
    (8, 4, 128, [12 * M] * 3),
    (8, 2, 64, [6 * M, 1, 5 * M + 13, 0, 7 * M - 1] * 2),
    (8, 2, 256, [3 * M // 2 + 5] * 33),
    (1, 12, 128, [200 * M + 1, 90 * M]),
])
def test_parts_of_more_than_half_a_million_tokens(kv, group, d, lens):
    cache = api.KVCache.empty(PAGES, PAGE, kv, d, "mxfp4", DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    normal = lambda *shape: (0.5 * torch.randn(shape, generator=g, device=DEV)).to(torch.bfloat16)   # noqa: E731
    k, v = normal(PAGES * PAGE, kv, d), normal(PAGES * PAGE, kv, d)
    api.kv_cache_write(cache, k, v, torch.arange(PAGES * PAGE, device=DEV))
    # eight pages, each for an eighth of the longest context
    width = -(-max(lens) // PAGE)
    table = torch.arange(width, device=DEV) * PAGES // width
    n = len(lens)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = normal(n, kv * group, d)
    out, lse = api.attention_decode(q, cache, table.int().unsqueeze(0).expand(n, width), ln, out_dtype=torch.float32,
                                    return_lse=True)
    kk, vv = (t.double() for t in api.kv_cache_read(cache, torch.arange(PAGES * PAGE, device=DEV), torch.float32))
    place = torch.arange(PAGE, device=DEV)
    for r, length in enumerate(lens):
        if length == 0:
            assert not out[r].any() and torch.all(lse[r] == -float("inf"))
            continue
        whole = torch.bincount(table[:length // PAGE], minlength=PAGES)
        times = whole.unsqueeze(1).expand(PAGES, PAGE).clone()
        if length % PAGE:
            times[table[length // PAGE]] += place < length % PAGE
        times = times.flatten().double()
        x = (kk * q[r].double().view(kv, group, d).transpose(0, 1).unsqueeze(1)).sum(-1) / d ** 0.5    # [group, token, kv]
        x = (x + torch.log(times).unsqueeze(-1)).permute(2, 0, 1)                                       # [kv, group, token]
        want_lse = torch.logsumexp(x, -1)
        p = torch.exp(x - want_lse.unsqueeze(-1))
        want = (p @ vv.transpose(0, 1).contiguous()).view(-1, d)
        size = (p @ vv.transpose(0, 1).abs().contiguous()).view(-1, d)
        # a lane adds 8 of every 128 tokens of a part one after the other, and the parts' sums are
        # added, each sum off by 2^-24 of itself at most; parts are no longer than twice those of
        # which every CU has one.  p's own rounding 2^-17; a score's 64 steps of 2^-24 of sums
        # of products that stay below 8
        part = min(length, 2 * sum(lens) * kv // 256 + 128)
        err = (part / 16 + 512) * 2.0 ** -24 + 2.0 ** -17 + 8 * 2.0 ** -18
        assert torch.all((lse[r].double() - want_lse.flatten()).abs() <= err + 2.0 ** -20)
        assert torch.all((out[r].double() - want).abs() <= 2 * err * size)
