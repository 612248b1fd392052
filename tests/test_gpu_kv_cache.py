"""The paged cache on the GPU: codes and scales of written slots to the bit against
the oracle's quantizers, everything else of the pools as it was, and slots read
back to the values that fp4_dequantize defines."""
import numpy as np
import pytest
import torch

import kv_check as C
from fp4_block_scaled_x16_amd import api
from kv_check import DEV, DIMS, FORMATS
from oracle import attention as A

pytestmark = pytest.mark.gpu


def written(cache, before, k, v, slots):
    """The oracle's pools after a write."""
    want = [p.copy() for p in before]
    for i, x in enumerate((k, v)):
        codes, scales = C.encoded(cache, i, x)
        for t, s in enumerate(slots):
            if 0 <= s < cache.pages * cache.page_size:
                g, p = divmod(int(s), cache.page_size)
                want[2 * i][g, :, p] = codes[t]
                want[2 * i + 1][g, :, :, p] = scales[t]
    return want


def same_pools(cache, want):
    for got, w in zip(C.contents(cache), want):
        assert np.array_equal(got, w), np.argwhere(got != w)[:5].tolist()


@pytest.mark.parametrize("tokens,heads,page,layout", [
    (1, 1, 16, "heads"), (1, 8, 64, "places"), (7, 3, 16, "layers"), (33, 8, 32, "heads"), (130, 5, 1024, "places")])
@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_write(fmt, d, tokens, heads, page, layout):
    pages = -(-tokens // page) + 2
    cache = C.make_cache(fmt, pages, page, heads, d, layout, seed=tokens)
    before = C.contents(cache)
    k, v = C.rows((tokens, heads, d), 1), C.rows((tokens, heads, d), 2)
    slots = np.random.default_rng(3).permutation(pages * page)[:tokens]
    slots[tokens // 2] = slots[tokens // 2] if tokens < 3 else -1            # one is not written
    if tokens > 3:
        slots[1], slots[3] = pages * page, -2 ** 40                           # nor are these
    api.kv_cache_write(cache, k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV))
    same_pools(cache, written(cache, before, k, v, slots))


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_from_a_projection(fmt):
    """Parts of one projection's rows, and rows with the heads outermost."""
    d, heads, tokens = 128, 4, 21
    cache = C.make_cache(fmt, 3, 16, heads, d)
    before = C.contents(cache)
    qkv = C.rows((tokens, 3 * heads, d), 5).to(DEV)
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:].transpose(0, 1).contiguous().transpose(0, 1)
    slots = torch.arange(tokens).flip(0).to(DEV)
    api.kv_cache_write(cache, k, v, slots)
    same_pools(cache, written(cache, before, k.cpu(), v.cpu(), slots.cpu().numpy()))


@pytest.mark.parametrize("layout,out", [("heads", torch.bfloat16), ("places", torch.float32), ("layers", torch.bfloat16)])
@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_read(fmt, d, layout, out):
    heads, page, pages = 3, 16, 5
    cache = C.make_cache(fmt, pages, page, heads, d, layout)
    k, v = C.rows((pages * page, heads, d), 1), C.rows((pages * page, heads, d), 2)
    api.kv_cache_write(cache, k.to(DEV), v.to(DEV), torch.arange(pages * page, device=DEV))
    pool = C.contents(cache)
    slots = np.array([5, 79, 0, -1, 5, 80, 33, 2 ** 40, -2 ** 33])
    got = api.kv_cache_read(cache, torch.from_numpy(slots).to(DEV), out_dtype=out)
    ok = (slots >= 0) & (slots < pages * page)
    at = np.where(ok, slots, 0)
    for i in range(2):
        assert got[i].dtype == out
        # as fp4_dequantize: the product with the tensor scale rounds to fp32, then to the output
        w = C.values(cache, pool, i, at // page, at % page) * ok[:, None, None]
        w = torch.from_numpy(w.astype(np.float32)).to(out)
        assert torch.equal(got[i].cpu(), w)


@pytest.mark.parametrize("heads,d", [(1, 64), (40, 128), (9, 256)])
def test_read_of_many_and_few_heads(heads, d):
    """Slots of more and of fewer elements than a workgroup takes at once."""
    cache = C.make_cache("fp8", 9, 16, heads, d)
    n = 9 * 16
    k, v = C.rows((n, heads, d), 1), C.rows((n, heads, d), 2)
    api.kv_cache_write(cache, k.to(DEV), v.to(DEV), torch.arange(n, device=DEV))
    pool = C.contents(cache)
    slots = np.arange(n)[::-1].copy()[:n - 3]
    got = api.kv_cache_read(cache, torch.from_numpy(slots).to(DEV))
    for i in range(2):
        w = C.values(cache, pool, i, slots // 16, slots % 16)
        assert torch.equal(got[i].cpu(), torch.from_numpy(w.astype(np.float32)).to(torch.bfloat16))


def test_nothing_to_do():
    cache = C.make_cache("mxfp4", 1, 16, 2, 64)
    before = C.contents(cache)
    empty = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    api.kv_cache_write(cache, empty, empty, none)
    k, v = api.kv_cache_read(cache, none)
    assert k.shape == v.shape == (0, 2, 64)
    same_pools(cache, before)


# With the norm and rotation in the same pass, K is encoded from values formed in 64 bits; here
# each code has to be that of a value within an fp32 computation's error of the exact one, and
# each scale that of an amax within it.
@pytest.mark.parametrize("style,rot,w_dtype", [("half", None, torch.bfloat16), ("interleaved", 32, torch.float32),
                                               ("half", 32, torch.bfloat16), ("half", 0, torch.bfloat16),
                                               ("interleaved", None, None)])
@pytest.mark.parametrize("d", DIMS)
@pytest.mark.parametrize("fmt", FORMATS)
def test_write_with_norm(fmt, d, style, rot, w_dtype):
    rot = d if rot is None else rot
    hq, hk, tokens, page, eps = 6, 2, 19, 16, 1e-5
    cache = C.make_cache(fmt, 3, page, hk, d, amax=(60.0, 60.0))
    before = C.contents(cache)
    qkv = C.rows((tokens, hq + 2 * hk, d), 11).to(DEV)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
    w = None if w_dtype is None else [(1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(i)))
                                      .to(w_dtype).to(DEV) for i in range(2)]
    tab = torch.from_numpy(C.table(50, rot)).to(DEV) if rot else None
    norm = api.QKNorm(*(w or (None, None)), tab, eps=eps, style=style)
    pos = torch.arange(tokens, device=DEV) * 2 + 3 if rot else None
    slots = torch.arange(tokens, device=DEV) + 7
    slots[4] = -1
    got_q = api.kv_cache_write(cache, k, v, slots, q=q, norm=norm, positions=pos)
    # q, to the bit as without a cache
    plain = api.qk_norm_rope(norm, q, k, pos)
    assert torch.equal(got_q, plain[0])
    # V to the bit, K's other slots as they were
    s = slots.cpu().numpy()
    want = written(cache, before, k.cpu(), v.cpu(), s)
    got = C.contents(cache)
    for a, b in zip(got[2:], want[2:]):
        assert np.array_equal(a, b)
    for a, b in zip(got[:2], before[:2]):
        keep = np.ones(3 * page, bool)
        keep[s[s >= 0]] = False
        g, p = np.nonzero(keep.reshape(3, page))
        at = (g, slice(None), p) if a is got[0] else (g, slice(None), slice(None), p)
        assert np.array_equal(a[at], b[at])
    c = sn = None
    if rot:
        t = C.as64(tab)[pos.cpu().numpy()][:, None]
        c, sn = t[..., :rot // 2], t[..., rot // 2:]
    x = C.as64(k)
    wk = None if w is None else C.as64(w[1])
    y = A.norm_rope(x, wk, c, sn, eps, style == "interleaved")
    # 16 roundings of the larger of the two products (test_gpu_qk_norm.py)
    size = np.abs(x) * (1 if w is None else np.abs(wk) * A.inv_rms(x, eps))
    err = 16 * C.U * C.turned(size, c, sn, style == "interleaved")
    ok = s >= 0
    codes, scales = got[0][s[ok] // page, :, s[ok] % page], got[1][s[ok] // page, :, :, s[ok] % page]
    held(cache, codes, scales, y[ok], err[ok])


def held(cache, codes, scales, y, err):
    """Codes and scales [n, heads, ..] hold y (float64), rounded from within err."""
    fmt, d = C.name_of(cache), cache.head_dim
    n = y.shape[0] * y.shape[1]
    y, err = y.reshape(n, d), err.reshape(n, d)
    codes, scales = codes.reshape(n, -1), scales.reshape(n, -1)
    bl = min(A.BLOCK[fmt], d)
    dec = A.s_dec(fmt, float(cache.amax[0]) if cache.amax is not None else 1.0, cache.target)
    one = A.row_values(np.full_like(codes, 0x38 if codes.shape[1] == d else 0x22), scales, fmt, d)   # codes of 1.0
    scale = one.reshape(n, -1, bl)[:, :, 0]
    big = np.abs(y).reshape(n, -1, bl).max(2)
    slack = (err.reshape(n, -1, bl).max(2) + 8 * C.U * big)           # the scale's own fp32 steps
    if fmt in A.TWO_LEVEL:
        # nearest of a 3-bit mantissa, up to the format's largest (a block may exceed the given
        # amax): half a step of the larger side's binade
        low = -6 if fmt == "nvfp4" else -14
        t = np.minimum(big / 6 / dec, 448.0 if fmt == "nvfp4" else 122880.0)
        half = np.exp2(np.floor(np.log2(np.maximum(t + slack / 6 / dec, 2.0 ** low))) - 4)
        assert np.all(np.abs(scale - t) <= half + slack / 6 / dec)
    else:
        top = 448.0 if codes.shape[1] == d else 6.0
        assert np.all(scale * top >= big - slack)
        assert np.all((scale / 2 * top < big + slack) | (scale == 2.0 ** -127))
    v = A.row_values(codes, scales, fmt, d)
    s = np.repeat(scale, bl, 1)
    yy = np.where(s > 0, y / dec, 0.0)
    e = err / dec + 8 * C.U * np.abs(yy)
    m, low, top = (3, -6, 448.0) if codes.shape[1] == d else (1, 0, 6.0)
    mag = np.clip(np.abs(yy) + e, s * 2.0 ** low, s * top)
    mag = np.maximum(mag, 1e-300)
    half = s * np.exp2(np.floor(np.log2(np.maximum(mag / np.maximum(s, 1e-300), 2.0 ** low))) - m - 1)
    over = np.maximum(np.abs(yy) - s * top, 0)                        # nearest scales saturate an element
    bad = np.abs(v - yy) > half + e + over
    assert not bad.any(), np.argwhere(bad)[:5].tolist()


def test_k_alone_with_norm():
    cache = C.make_cache("mxfp8", 2, 16, 2, 128)
    other = C.make_cache("mxfp8", 2, 16, 2, 128)
    x = C.rows((9, 6, 128), 3).to(DEV)
    norm = api.QKNorm(table=torch.from_numpy(C.table(9, 128)).to(DEV))
    slots, pos = torch.arange(9, device=DEV) + 4, torch.arange(9, device=DEV)
    assert api.kv_cache_write(cache, x[:, :2], x[:, 2:4], slots, norm=norm, positions=pos) is None
    api.kv_cache_write(other, x[:, :2], x[:, 2:4], slots, q=x[:, 4:], norm=norm, positions=pos)
    for a, b in zip(C.contents(cache), C.contents(other)):
        assert np.array_equal(a, b)


def test_graph_and_stream():
    """Captured on a stream of its own and replayed with new inputs and slots."""
    cache, eager = (C.make_cache("nvfp4", 8, 16, 4, 128) for _ in range(2))
    w = [torch.ones(128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    norm = api.QKNorm(*w, torch.from_numpy(C.table(64, 128)).to(DEV))
    x = torch.zeros((3, 12, 128), dtype=torch.bfloat16, device=DEV)
    slots, pos = torch.zeros(3, dtype=torch.int64, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV)
    slots.copy_(torch.arange(3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        api.kv_cache_write(cache, x[:, 4:8], x[:, 8:], slots, q=x[:, :4], norm=norm, positions=pos)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            q = api.kv_cache_write(cache, x[:, 4:8], x[:, 8:], slots, q=x[:, :4], norm=norm, positions=pos)
            k, v = api.kv_cache_read(cache, slots)
    torch.cuda.current_stream().wait_stream(side)
    for step in range(4):
        x.copy_(C.rows((3, 12, 128), step).to(DEV))
        slots.copy_(torch.tensor([5, 40, 90]) + step)
        pos.copy_(torch.tensor([1, 7, 20]) + step)
        graph.replay()
        want = api.kv_cache_write(eager, x[:, 4:8], x[:, 8:], slots, q=x[:, :4], norm=norm, positions=pos)
        wk, wv = api.kv_cache_read(eager, slots)
        torch.cuda.synchronize()
        assert torch.equal(q, want) and torch.equal(k, wk) and torch.equal(v, wv)


@pytest.mark.parametrize("style,rot", [("half", 128), ("interleaved", 64)])
@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "mxfp4"])
def test_codes_are_those_of_the_exact_values(fmt, style, rot):
    """Of 250000 elements as many as lie next to a border between two codes: within what 64 bits
    leave (2^-50 of a value, of which a border is nearer with a chance of 1e-9 in all)."""
    d, heads, tokens, page, eps = 128, 4, 500, 16, np.float32(1e-6)
    cache = C.make_cache(fmt, 32, page, heads, d)
    k = C.rows((tokens, heads, d), 5).to(DEV)
    w = [1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(i)).to(DEV) for i in range(2)]
    tab = torch.from_numpy(C.table(tokens, rot)).to(DEV)
    pos = slots = torch.arange(tokens, device=DEV)
    api.kv_cache_write(cache, k, k, slots, norm=api.QKNorm(*w, tab, eps=float(eps), style=style), positions=pos)
    t = C.as64(tab)[:, None]
    y = A.norm_rope(C.as64(k), C.as64(w[1]), t[..., :rot // 2], t[..., rot // 2:], float(eps), style == "interleaved")
    s = np.arange(tokens)
    codes, scales, *_ = C.contents(cache)
    n = tokens * heads
    got = A.row_values(codes[s // page, :, s % page].reshape(n, -1), scales[s // page, :, :, s % page].reshape(n, -1), fmt, d)
    top, low, m = (448.0, -6, 3) if fmt != "mxfp4" else (6.0, 0, 1)
    b = y.reshape(n, -1, A.BLOCK[fmt])
    big = np.maximum(np.abs(b).max(2), 2.0 ** -110)
    by = np.exp2(np.ceil(np.log2(big / top)))
    by = np.where(big > top * by, 2 * by, np.where(big <= top * by / 2, by / 2, by))[..., None]
    z = b / by
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -200))), low) - m)
    assert np.array_equal(got, (np.rint(z / step) * step * by).reshape(n, d))
