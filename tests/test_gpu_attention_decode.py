"""Attention of one new token over the paged cache, against 64-bit arithmetic on the
values that the codes stand for, within the error derived for its fp32 steps."""
import numpy as np
import pytest
import torch

import kv_check as C
from fp4_block_scaled_x16_amd import api
from kv_check import DEV, DIMS, FORMATS, U
from oracle import attention as A

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def chosen_splits():
    yield
    api.selftest_set_attention_splits(0)


def filled(fmt, pages, page, heads, d, layout="heads", seed=1, sigma=1.0):
    """A cache with every slot written: rows of many sizes, K with a few large channels."""
    cache = C.make_cache(fmt, pages, page, heads, d, layout, amax=(30.0, 20.0))
    k, v = C.rows((pages * page, heads, d), seed, sigma), C.rows((pages * page, heads, d), seed + 1)
    api.kv_cache_write(cache, k.to(DEV), v.to(DEV), torch.arange(pages * page, device=DEV))
    return cache


def query(n, heads, d, seed, sigma=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy(rng.standard_normal((n, heads, d)).astype(np.float32) * np.float32(sigma)).to(torch.bfloat16)


def tables(lens, page, pages, width, seed):
    """Pages in random order (shared where there are too few), -1 behind a request's last."""
    rng = np.random.default_rng(seed)
    t = np.full((len(lens), width), -1, np.int32)
    free = list(rng.permutation(pages))
    for r, n in enumerate(lens):
        for i in range(-(-max(n, 0) // page)):
            t[r, i] = free[i % len(free)] if len(free) <= 64 else free.pop()
    return t


# Error of out, 64-bit values of the operands being exact:
#   a score: products exact, their D + 2 additions at most a step (2 U) of sum |q k| each (the
#   matrix instruction's order is its own), the factor and the subtraction of the maximum 4 U of
#   |x| + |top|: e (in units of the exponent), and p's own exp2, its sum and its second rounding 2^-16;
#   both in p v and in the sum of p, whose n additions have a step each.
#   p is relative to the largest, 1: fp32's exponents end at 2^-126, and what lies below (p, or
#   what its rounding leaves) may count as zero, which is 2^-126 of |v| for each of the two.
#   NVFP4 and UE5M3 hold p as two fp16 numbers, the largest being at least 2^7: the second ends at
#   steps of 2^-24, half of which is 2^-32 of the largest p.
def check(out, lse, q, cache, pool, table, lens, scale, dropped=()):
    d, page, group = cache.head_dim, cache.page_size, q.shape[1] // cache.heads
    q64 = C.as64(q)
    least = 2.0 ** -32 if C.name_of(cache) in A.TWO_LEVEL else 2 * 2.0 ** -126
    want, err = np.zeros(q64.shape), np.zeros(q64.shape)
    wlse, elow = np.full(q64.shape[:2], -np.inf), np.zeros(q64.shape[:2])
    for r, n in enumerate(lens):
        t = np.arange(max(n, 0))
        t = t[~np.isin(t // page, [i for rr, i in dropped if rr == r])]
        g, p = table[r][t // page], t % page
        k, v = (C.values(cache, pool, i, g, p) for i in range(2))
        for h in range(q64.shape[1]):
            kk, vv = k[:, h // group], v[:, h // group]
            want[r, h], wlse[r, h] = A.attention(q64[r, h], kk, vv, scale)
            if len(t):
                x = kk @ q64[r, h] * scale
                e = (2 * (d + 2) * U * np.abs(kk) @ np.abs(q64[r, h]) * abs(scale) + 4 * U * (np.abs(x) + np.abs(x).max())).max()
                w = np.exp(x - wlse[r, h])
                rel = 2 * e + 2.0 ** -16 + 2 * (len(t) + 64) * U
                err[r, h] = rel * (w @ np.abs(vv)) + least * np.abs(vv).sum(0)
                elow[r, h] = rel + 4 * U * abs(wlse[r, h])
    C.near(out, want, err)
    if lse is not None:
        got = C.as64(lse)
        none = np.isneginf(wlse)
        assert np.array_equal(np.isneginf(got), none)
        assert np.all(np.abs(got[~none] - wlse[~none]) <= elow[~none])


@pytest.mark.parametrize("heads,group,page,layout,lens", [
    (1, 1, 16, "heads", [1]),
    (2, 4, 16, "places", [0, 1, 15, 16, 17, 31, 33, 200]),
    (1, 8, 64, "layers", [129, 512, 63]),
    (3, 7, 32, "heads", [300, 0, 5]),
    (1, 16, 16, "heads", [257, 40]),
    (2, 12, 128, "places", [130, 1]),
    (1, 20, 16, "heads", [77, 600]),
])
@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_decode(fmt, d, heads, group, page, layout, lens):
    pages = 1040 // page
    cache = filled(fmt, pages, page, heads, d, layout)
    pool = C.contents(cache)
    width = -(-max(lens) // page) + 2
    table = tables(lens, page, pages, width, 3)
    q = query(len(lens), heads * group, d, 4)
    dev = dict(page_table=torch.from_numpy(table).to(DEV), lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    out, lse = api.attention_decode(q.to(DEV), cache, **dev, return_lse=True)
    check(out, lse, q, cache, pool, table, lens, d ** -0.5)
    out, lse = api.attention_decode(q.to(DEV), cache, **dev, return_lse=True, out_dtype=torch.float32)
    check(out, lse, q, cache, pool, table, lens, d ** -0.5)


@pytest.mark.parametrize("splits", [1, 2, 3, 5, 8, 64, 512])
@pytest.mark.parametrize("fmt,d,group", [("fp8", 128, 4), ("nvfp4", 64, 16), ("mxfp4", 256, 2)])
def test_every_number_of_parts(fmt, d, group, splits):
    """Shared among any number of workgroups, also more than there are tokens for."""
    page, lens = 16, [1000, 0, 1, 127, 128, 129, 513, 4000]
    cache = filled(fmt, 251, page, 1, d)
    pool = C.contents(cache)
    table = tables(lens, page, 251, 251, 5)
    q = query(len(lens), group, d, 6)
    api.selftest_set_attention_splits(splits)
    out, lse = api.attention_decode(q.to(DEV), cache, torch.from_numpy(table).to(DEV),
                                    torch.tensor(lens, dtype=torch.int32, device=DEV), out_dtype=torch.float32,
                                    return_lse=True)
    check(out, lse, q, cache, pool, table, lens, d ** -0.5)


@pytest.mark.parametrize("fmt", FORMATS)
def test_garbage_behind_the_last_token(fmt):
    """Codes and scales of every value behind a request's tokens, in its last page and
    elsewhere, have no part in its result."""
    d, page, heads = 128, 64, 2
    lens = [1, 40, 70, 97, 130]
    cache = filled(fmt, 16, page, heads, d)
    table = tables(lens, page, 16, 4, 7)
    table[:, :] = np.arange(20).reshape(5, 4) % 16
    table[4] = [3, 7, 11, 99]
    q = query(5, 8, d, 8).to(DEV)
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    args = dict(page_table=torch.from_numpy(table).to(DEV), lens=ln, return_lse=True)
    rows_ = []
    for fill in (0, 0xFF, 0x7F):
        got = []
        for r, n in enumerate(lens):
            keep = [t.clone() for t in C.tensors(cache)]
            mask = torch.ones(16 * page, dtype=torch.bool, device=DEV)
            t = torch.arange(n, device=DEV)
            mask[args["page_table"][r][t // page].long() * page + t % page] = False
            at = mask.nonzero().flatten()
            for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
                c[at // page, :, at % page] = fill
                s[at // page, :, :, at % page] = fill
            o = api.attention_decode(q, cache, **args)
            got += [o[0][r].clone(), o[1][r].clone()]
            for a, b in zip(C.tensors(cache), keep):
                a.copy_(b)
        rows_.append(got)
    for other in rows_[1:]:
        assert all(torch.equal(a, b) for a, b in zip(rows_[0], other))


def test_pages_that_are_not_there():
    """Tokens of a page outside the cache are left out; a request of such pages alone has
    no tokens; entries behind the length are not looked at."""
    d, page = 128, 16
    cache = filled("mxfp8", 8, page, 1, d)
    pool = C.contents(cache)
    lens = [100, 33, 48, 64]
    table = tables(lens, page, 8, 9, 9)
    table[0, 2], table[0, 5] = -1, 8
    table[1, :] = [2 ** 31 - 1, -2 ** 31, 9, 0, 0, 0, 0, 0, 0]
    table[2, 3:] = 77
    q = query(4, 4, d, 10)
    out, lse = api.attention_decode(q.to(DEV), cache, torch.from_numpy(table).to(DEV),
                                    torch.tensor(lens, dtype=torch.int32, device=DEV), return_lse=True)
    dropped = [(0, 2), (0, 5), (1, 0), (1, 1), (1, 2)]
    check(out, lse, q, cache, pool, table, lens, d ** -0.5, dropped)


def test_lengths_beyond_the_table_and_below_zero():
    cache = filled("fp8", 4, 16, 1, 64)
    table = torch.arange(4, dtype=torch.int32, device=DEV).expand(4, 4)        # one table for all
    q = query(4, 2, 64, 1).to(DEV)
    lens = torch.tensor([64, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32, device=DEV)
    q[1] = q[0]
    out, lse = api.attention_decode(q, cache, table, lens, return_lse=True)
    assert torch.equal(out[0], out[1]) and out[0].any()
    assert not out[2:].any() and torch.isneginf(lse[2:]).all()
    out = api.attention_decode(q, cache, table[:, :0], lens)
    assert not out.any()
    assert api.attention_decode(q[:0], cache, table[:0], lens[:0]).shape == (0, 2, 64)


@pytest.mark.parametrize("scale,sigma", [(1.0, 4.0), (-0.5, 1.0), (0.0, 1.0), (30.0, 3.0)])
@pytest.mark.parametrize("fmt", ["mxfp8", "ue5m3"])
def test_scales_and_sharp_scores(fmt, scale, sigma):
    """Sharp, flat and negated scores: the running maximum far from the first tile's."""
    d, page, lens = 128, 32, [700, 31]
    cache = filled(fmt, 22, page, 2, d)
    pool = C.contents(cache)
    table = tables(lens, page, 22, 22, 1)
    q = query(2, 6, d, 12, sigma)
    out, lse = api.attention_decode(q.to(DEV), cache, torch.from_numpy(table).to(DEV),
                                    torch.tensor(lens, dtype=torch.int32, device=DEV), scale=scale, return_lse=True,
                                    out_dtype=torch.float32)
    check(out, lse, q, cache, pool, table, lens, scale)


@pytest.mark.parametrize("fmt", FORMATS)
def test_queries_of_any_size(fmt):
    """Rows of q near the ends of fp32's range and a zero row, scores brought back by
    the scale."""
    d, page, lens = 64, 16, [50, 50, 50]
    cache = filled(fmt, 4, page, 1, d, sigma=0.25)
    pool = C.contents(cache)
    table = tables(lens, page, 4, 4, 1)
    lens_d, table_d = torch.tensor(lens, dtype=torch.int32, device=DEV), torch.from_numpy(table).to(DEV)
    for power in (100, -100):
        q = query(3, 2, d, 13) * 2.0 ** power
        q[1] = 0
        out, lse = api.attention_decode(q.to(DEV), cache, table_d, lens_d, scale=2.0 ** -power, return_lse=True)
        check(out, lse, q, cache, pool, table, lens, 2.0 ** -power)


def test_a_query_that_is_not_finite_spoils_its_own_rows_only():
    cache = filled("nvfp4", 4, 16, 2, 64)
    table = torch.arange(4, dtype=torch.int32, device=DEV).expand(2, 4)
    lens = torch.tensor([60, 60], dtype=torch.int32, device=DEV)
    q = query(2, 8, 64, 1).to(DEV)
    want = api.attention_decode(q, cache, table, lens)
    q[0, 1, 3], q[1, 6, 0] = float("nan"), float("inf")
    got = api.attention_decode(q, cache, table, lens)
    assert torch.isnan(got[0, 1]).all() and torch.isnan(got[1, 6]).all()
    keep = torch.ones((2, 8), dtype=torch.bool)
    keep[0, 1] = keep[1, 6] = False
    assert torch.equal(got[keep], want[keep])


def test_strided_queries_tables_and_outputs():
    cache = filled("mxfp4", 6, 16, 2, 128)
    lens = torch.tensor([90, 3, 50], dtype=torch.int32, device=DEV)
    wide = torch.zeros((3, 11), dtype=torch.int32, device=DEV)
    wide[:, 2:8] = torch.arange(6, device=DEV)
    q = query(3, 12, 128, 2).to(DEV)
    want = api.attention_decode(q[:, 4:8].contiguous(), cache, wide[:, 2:8].contiguous(), lens)
    out = torch.full((3, 4, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    assert api.attention_decode(q[:, 4:8], cache, wide[:, 2:8], lens, out=out) is out
    assert torch.equal(out, want)


def test_two_graphs_and_streams():
    """Two captured calls replayed at once on two streams, beside eager ones: each has a
    workspace of its own."""
    page, lens = 16, [2000, 333]
    cache = filled("fp8", 126, page, 2, 128)
    table = torch.from_numpy(tables(lens, page, 126, 126, 1)).to(DEV)
    lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = [query(2, 8, 128, s).to(DEV) for s in range(2)]
    streams, graphs, outs = [torch.cuda.Stream() for _ in range(2)], [], []
    for s, q in zip(streams, qs):
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            api.attention_decode(q, cache, table, lens)
            s.synchronize()
            with torch.cuda.graph(g, stream=s):
                outs.append(api.attention_decode(q, cache, table, lens))
        graphs.append(g)
    for step in range(4):
        for i, q in enumerate(qs):
            q.copy_(query(2, 8, 128, 10 * step + i).to(DEV))
            lens.copy_(torch.tensor([2000 - 7 * step, 333 + step], dtype=torch.int32))
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        want = [api.attention_decode(q, cache, table, lens) for q in qs]
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_parts_of_a_context_join_by_their_lse():
    """Two halves of a request's tokens, joined by the logs of their denominators."""
    d, page = 128, 16
    cache = filled("mxfp8", 8, page, 1, d)
    q = query(1, 4, d, 3).to(DEV)
    table = torch.arange(8, dtype=torch.int32, device=DEV).view(1, 8)
    n = lambda v: torch.tensor([v], dtype=torch.int32, device=DEV)                              # noqa: E731
    whole = api.attention_decode(q, cache, table, n(120), out_dtype=torch.float32)
    a, la = api.attention_decode(q, cache, table[:, :3], n(48), out_dtype=torch.float32, return_lse=True)
    b, lb = api.attention_decode(q, cache, table[:, 3:], n(72), out_dtype=torch.float32, return_lse=True)
    w = torch.sigmoid(la - lb).unsqueeze(-1)
    at = np.arange(120)
    kk, vv = (C.values(cache, C.contents(cache), i, at // page, at % page)[:, 0] for i in range(2))
    size = (np.abs(kk) @ np.abs(C.as64(q)[0]).T).max() * d ** -0.5
    # each of the three within its own error (see check) of max |v|, and the weight w within
    # that of both logs, times |a - b|
    rel = 2 * (2 * (d + 2) + 8) * U * size + 2.0 ** -16 + 2 * (120 + 64) * U
    assert torch.allclose(w * a + (1 - w) * b, whole, rtol=0, atol=5 * rel * np.abs(vv).max())


@pytest.mark.parametrize("group,requests,heads,page,width", [(5, 70, 4, 16, 4), (12, 130, 2, 32, 2), (1, 1600, 1, 128, 3)])
@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_many_short_requests(fmt, d, group, requests, heads, page, width):
    """One wave to a request: lengths from none to all that the table has room for."""
    pages = 768 // page
    cache = filled(fmt, pages, page, heads, d)
    pool = C.contents(cache)
    lens = [(37 * i) % (page * width + 1) for i in range(requests)]
    table = tables(lens, page, pages, width, 3)
    q = query(requests, heads * group, d, 4)
    out, lse = api.attention_decode(q.to(DEV), cache, torch.from_numpy(table).to(DEV),
                                    torch.tensor(lens, dtype=torch.int32, device=DEV), return_lse=True)
    sel = list(range(0, requests, max(1, requests // 24)))
    check(out[sel], lse[sel], q[sel], cache, pool, table[sel], [lens[i] for i in sel], d ** -0.5)


@pytest.mark.parametrize("requests", [2, 63, 65, 128, 200, 256, 257])
def test_order_of_the_requests(requests):
    """Whichever request a workgroup takes: every one is served, with equal lengths and with
    different ones, none and all that there is room for among them."""
    page, width, heads = 16, 40, 4
    cache = filled("mxfp8", 40, page, heads, 64)
    table = torch.stack([torch.randperm(40, generator=torch.Generator().manual_seed(i)) for i in range(requests)]).int().to(DEV)
    q = query(requests, 8, 64, 3).to(DEV)
    r = torch.arange(requests, device=DEV)
    for lens in (torch.full_like(r, 640), torch.full_like(r, 1), torch.zeros_like(r), r * 977 % 641, torch.where(r == 1, 640, 0),
                 r * 977 % 700 - 30, torch.where(r % 2 == 0, 2 ** 31 - 1, 0)):
        lens = lens.int()
        api.selftest_set_attention_splits(0)
        out, lse = api.attention_decode(q, cache, table, lens, return_lse=True)
        # one by one, in one part
        api.selftest_set_attention_splits(1)
        for i in range(requests):
            a, b = api.attention_decode(q[i:i + 1], cache, table[i:i + 1], lens[i:i + 1], return_lse=True, out_dtype=torch.float32)
            n = int(lens[i].clamp(0, 640))
            # bf16's half step of the output (the parts' sums and p are exact to 2^-15 of |v|, here up to 2^9)
            assert (out[i].float() - a[0]).abs().max() <= 2.0 ** -8 * a.abs().max() + 2.0 ** -6, (i, n)
            assert torch.equal(torch.isinf(lse[i]), torch.isinf(b[0])) and (n == 0) == bool(torch.isinf(b).all())
            if n:
                assert (lse[i] - b[0]).abs().max() <= 2.0 ** -10


@pytest.mark.parametrize("fmt,d,group", [("mxfp8", 128, 4), ("nvfp4", 64, 12), ("fp8", 256, 2)])
@pytest.mark.parametrize("lens", [[700], [0], [5, 700, 0, 300], [640] * 40, [1] * 70 + [1000], list(range(0, 1000, 7))])
def test_tables_wider_than_the_requests(fmt, d, group, lens):
    """Room for far more tokens than there are: parts go by the lengths.  Entries behind a
    request's last page are no pages."""
    page, heads, pages = 16, 2, 64
    cache = filled(fmt, pages, page, heads, d)
    pool = C.contents(cache)
    for width in (64, 512, 8192):
        table = tables(lens, page, pages, width, 3)
        q = query(len(lens), heads * group, d, 4)
        out, lse = api.attention_decode(q.to(DEV), cache, torch.from_numpy(table).to(DEV),
                                        torch.tensor(lens, dtype=torch.int32, device=DEV), return_lse=True)
        sel = list(range(0, len(lens), max(1, len(lens) // 12)))
        sel += [len(lens) - 1] * (sel[-1] != len(lens) - 1)
        check(out[sel], lse[sel], q[sel], cache, pool, table[sel], [lens[i] for i in sel], d ** -0.5)
