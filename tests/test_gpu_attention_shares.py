"""Ways of sharing requests' tokens that sizes alone do not lead to often: a workspace that is
too small or none, parts in a call of several launches, parts of more requests than are
planned by their lengths."""
import ctypes

import pytest
import torch

import kv_check as C
from fp4_block_scaled_x16_amd import api
from kv_check import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def chosen_splits():
    yield
    api.selftest_set_attention_splits(0)


def setup(fmt, requests, longest, heads, group, d, page=16, seed=1):
    """A cache whose pages requests share, and requests of 0 to `longest` tokens."""
    cache = C.make_cache(fmt, 40, page, heads, d)
    n = 40 * page
    api.kv_cache_write(cache, *(C.rows((n, heads, d), seed + i).to(DEV) for i in range(2)), torch.arange(n, device=DEV))
    g = torch.Generator().manual_seed(seed)
    table = torch.randint(0, 40, (requests, -(-longest // page)), generator=g).int().to(DEV)
    lens = torch.randint(0, longest + 1, (requests,), generator=g).int()
    lens[-1], lens[0] = 0, longest
    return cache, C.rows((requests, heads * group, d), seed + 2).to(DEV), table, lens.to(DEV)


def whole(*args):
    api.selftest_set_attention_splits(1)
    r = api.attention_decode(*args, out_dtype=torch.float32, return_lse=True)
    api.selftest_set_attention_splits(0)
    return r


def close(got, want, cache):
    """Two ways of sharing: each p off by 2^-17 (its parts), scores alike, sums of up to 1500 terms and
    the powers of two that weigh parts off by 2^-22 of themselves."""
    top = float(torch.cat([t.abs().flatten() for t in api.kv_cache_read(
        cache, torch.arange(cache.pages * cache.page_size, device=DEV), torch.float32)[1:]]).max())
    assert (got[0] - want[0]).abs().max() <= 2 * (2.0 ** -17 + 1500 * 2.0 ** -24 + 2.0 ** -22) * top
    both = torch.isfinite(want[1])
    assert torch.equal(got[1][~both], want[1][~both]) and not got[0][~both].any()
    # lse: sums alike to within that, and fp32 steps of numbers below 128
    assert (got[1][both] - want[1][both]).abs().max() <= 2 * (1500 * 2.0 ** -24 + 2.0 ** -22) + 4 * 128 * 2.0 ** -24


@pytest.mark.parametrize("fmt,heads,group,d", [("fp8", 2, 4, 64), ("mxfp8", 8, 4, 128), ("nvfp4", 4, 12, 128), ("mxfp4", 2, 20, 64),
                                               ("ue5m3", 4, 1, 256)])
@pytest.mark.parametrize("requests", [1, 7, 40, 200])
def test_a_workspace_that_is_too_small(fmt, heads, group, d, requests):
    """The requests are taken whole then, to the bit as when one part is asked for, and the
    workspace is left alone."""
    cache, q, table, lens = setup(fmt, requests, 5000, heads, group, d)
    n = q.shape[0]
    size = cache._workspace(heads * group, n, table.shape[1])
    assert size > 0
    want = whole(q, cache, table, lens)
    h = api.Heads(q.data_ptr(), q.stride(0), q.stride(1), q.shape[1])
    for bytes_given in (0, 16, size - 8):
        ws = torch.full((size + 16,), 0x5A, dtype=torch.uint8, device=DEV)
        out, lse = torch.full_like(want[0], 7), torch.full_like(want[1], 7)
        status = api.load_library().fp4_attention_decode(
            cache._at, ctypes.addressof(h), table.data_ptr(), table.stride(0), table.shape[1], lens.data_ptr(), n, d ** -0.5,
            out.data_ptr(), api.OUT_TYPES[out.dtype], lse.data_ptr(), ws.data_ptr() if bytes_given else None, bytes_given,
            torch.cuda.current_stream().cuda_stream)
        assert status == 0
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1]) and torch.all(ws == 0x5A)
    close(api.attention_decode(q, cache, table, lens, out_dtype=torch.float32, return_lse=True), want, cache)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_parts_in_a_call_of_two_launches(fmt):
    """1030 requests of 8 heads in up to 512 parts: 1024 of them in the first launch."""
    cache, q, table, lens = setup(fmt, 1030, 700, 8, 1, 64)
    want = whole(q, cache, table, lens)
    api.selftest_set_attention_splits(512)
    close(api.attention_decode(q, cache, table, lens, out_dtype=torch.float32, return_lse=True), want, cache)


@pytest.mark.parametrize("fmt,d,heads", [("mxfp8", 128, 2), ("mxfp4", 64, 1), ("ue5m3", 256, 1)])
@pytest.mark.parametrize("requests", [257, 300, 600])
def test_parts_of_more_requests_than_are_planned(fmt, d, heads, requests):
    cache, q, table, lens = setup(fmt, requests, 5000, heads, 4, d)
    assert cache._workspace(4 * heads, requests, table.shape[1]) > 0          # there are parts
    close(api.attention_decode(q, cache, table, lens, out_dtype=torch.float32, return_lse=True),
          whole(q, cache, table, lens), cache)
