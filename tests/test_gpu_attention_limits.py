"""The attention operators at the ends of their ranges: more tokens or requests than a
launch has threads for, pages whose bytes lie beyond 2^32, the same slot or page named
twice, no tokens, and what autograd must refuse."""
import numpy as np
import pytest
import torch

import kv_check as C
from fp4_block_scaled_x16_amd import api, attention
from kv_check import DEV, FORMATS

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
MANY = (1 << 22) + 5            # tokens or requests: two launches
ENDS = [slice(0, 9), slice((1 << 22) - 4, MANY)]


@pytest.fixture(autouse=True)
def chosen_splits():
    yield
    api.selftest_set_attention_splits(0)


def normal(*shape, scale=1.0):
    return torch.empty(shape, dtype=BF, device=DEV).normal_(0.0, scale)


def norm_of(d, rows=64):
    return api.QKNorm(*(1 + 0.2 * torch.randn(d, device=DEV) for _ in range(2)), attention.rotary_table(rows, d, device=DEV))


def test_norm_of_more_tokens_than_a_launch_has():
    norm, d = norm_of(64), 64
    q, k = normal(MANY, 1, d), normal(MANY, 2, d)
    pos = torch.arange(MANY, device=DEV) % 64
    yq, yk = api.qk_norm_rope(norm, q, k, pos)
    for s in ENDS:
        a, b = api.qk_norm_rope(norm, q[s], k[s], pos[s])
        assert torch.equal(yq[s], a) and torch.equal(yk[s], b)
    # backward: a row's gradient is its own; the weights' is that of two halves
    dq, dk = normal(MANY, 1, d), normal(MANY, 2, d)
    got = api.qk_norm_rope_backward(norm, q, k, pos, dq, dk)
    for s in ENDS:
        want = api.qk_norm_rope_backward(norm, q[s], k[s], pos[s], dq[s], dk[s])
        assert torch.equal(got[0][s], want[0]) and torch.equal(got[1][s], want[1])
    h = MANY // 2
    parts = [api.qk_norm_rope_backward(norm, q[s], k[s], pos[s], dq[s], dk[s])[2:] for s in (slice(0, h), slice(h, MANY))]
    # a wave sums up to 2^22 / 5120 = 820 of the terms one after the other (at 5 workgroups of 4 waves
    # on 256 CUs, two heads: 1640), of normal size: a random walk, whose roundings of 2^-24 of it stay
    # below 1640 x 2^-24 x sqrt(2^23) x 4 standard deviations
    for i in range(2):
        assert (got[2 + i] - parts[0][i] - parts[1][i]).abs().max() <= 1640 * 2.0 ** -24 * 2.0 ** 11.5 * 4


@pytest.mark.parametrize("fmt", ["mxfp4", "fp8"])
def test_write_of_more_tokens_than_a_launch_has(fmt):
    d, page = 64, 1024
    pages = MANY // page + 1
    norm = norm_of(d)
    cache, small = (C.make_cache(fmt, n, page, 1, d) if n < 9 else api.KVCache.empty(n, page, 1, d, fmt, DEV)
                    for n in (pages, 1))
    k, v, q = normal(MANY, 1, d), normal(MANY, 1, d), normal(MANY, 1, d)
    pos = torch.arange(MANY, device=DEV) % 64
    slots = torch.arange(MANY, device=DEV)
    y = api.kv_cache_write(cache, k, v, slots, q=q, norm=norm, positions=pos)
    kk, vv = api.kv_cache_read(cache, slots)
    for s in ENDS:
        at = torch.arange(s.stop - s.start, device=DEV)
        want = api.kv_cache_write(small, k[s], v[s], at, q=q[s], norm=norm, positions=pos[s])
        a, b = api.kv_cache_read(small, at)
        assert torch.equal(y[s], want) and torch.equal(kk[s], a) and torch.equal(vv[s], b)


@pytest.mark.parametrize("group", [1, 20])
def test_attention_of_more_requests_than_a_launch_has(group):
    """One launch's workgroups: a key head's 20 query heads take two."""
    d = 64
    n = MANY if group == 1 else (1 << 21) + 3
    cache = C.make_cache("mxfp8", 2, 16, 1, d)
    api.kv_cache_write(cache, normal(32, 1, d), normal(32, 1, d), torch.arange(32, device=DEV))
    table = torch.tensor([[1, 0]], dtype=torch.int32, device=DEV)
    lens = (torch.arange(n, device=DEV) % 34 - 1).int()
    q = normal(n, group, d)
    api.selftest_set_attention_splits(1)
    out, lse = api.attention_decode(q, cache, table.expand(n, 2), lens, return_lse=True)
    for s in (slice(0, 9), slice(n - 12, n)):
        a, b = api.attention_decode(q[s], cache, table.expand(s.stop - s.start, 2), lens[s], return_lse=True)
        assert torch.equal(out[s], a) and torch.equal(lse[s], b)


@pytest.mark.parametrize("fmt", FORMATS)
def test_pages_beyond_4_gib(fmt):
    """Three pages 2 GiB and a little apart, codes and scales: the same bytes and the same
    results as in a dense cache."""
    d, heads, page = 128, 2, 16
    dense = C.make_cache(fmt, 3, page, heads, d)
    stride = (1 << 31) + 4096
    base = torch.empty(2 * stride + 65536, dtype=torch.uint8, device=DEV)
    spread, at = [], 0
    for t in C.tensors(dense):
        spread.append(base[at:].as_strided(t.shape, (stride, *t.stride()[1:])))
        at += 16384                                      # a page has 4096 bytes or fewer
        spread[-1].copy_(t)
    far = api.KVCache(fmt, *spread, amax=dense.amax, target=dense.target)
    k, v = C.rows((40, heads, d), 1).to(DEV), C.rows((40, heads, d), 2).to(DEV)
    slots = torch.arange(48, device=DEV).flip(0)[:40].contiguous()
    for c in (dense, far):
        api.kv_cache_write(c, k, v, slots)
    for a, b in zip(C.tensors(dense), C.tensors(far)):
        assert torch.equal(a, b)
    for a, b in zip(api.kv_cache_read(dense, slots), api.kv_cache_read(far, slots)):
        assert torch.equal(a, b)
    table = torch.tensor([[2, 1, 0], [1, 2, 2]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([40, 45], dtype=torch.int32, device=DEV)
    q = C.rows((2, 8, d), 3).to(DEV)
    for splits in (0, 1, 3):
        api.selftest_set_attention_splits(splits)
        # bits: the first 8 slots hold random bytes, NaN among them, which are not equal to themselves
        a, b = (api.attention_decode(q, c, table, lens).view(torch.int16) for c in (dense, far))
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_slot_named_twice_leaves_the_others_alone(fmt):
    """It ends with bytes of either row, and no other byte changes."""
    d = 128
    caches = [C.make_cache(fmt, 2, 16, 2, d) for _ in range(3)]
    before = C.contents(caches[0])
    k, v = C.rows((2, 2, d), 1).to(DEV), C.rows((2, 2, d), 2).to(DEV)
    one = torch.tensor([21], device=DEV)
    api.kv_cache_write(caches[0], k, v, one.expand(2).contiguous())
    api.kv_cache_write(caches[1], k[:1], v[:1], one)
    api.kv_cache_write(caches[2], k[1:], v[1:], one)
    got, a, b = (C.contents(c) for c in caches)
    for i in range(4):
        there = np.zeros(got[i].shape, bool)
        (there[1, :, 5] if i % 2 == 0 else there[1, :, :, 5])[...] = True
        assert np.all((got[i] == a[i]) | (got[i] == b[i])) and np.array_equal(got[i][~there], before[i][~there])


def test_pages_and_requests_that_share():
    """A page that a request has twice, and rows of one request beside each other with
    lengths that count up: as a dense cache of the same tokens."""
    d, page = 64, 16
    cache, dense = C.make_cache("mxfp8", 3, page, 1, d), C.make_cache("mxfp8", 5, page, 1, d, seed=4)
    k, v = C.rows((48, 1, d), 1).to(DEV), C.rows((48, 1, d), 2).to(DEV)
    api.kv_cache_write(cache, k, v, torch.arange(48, device=DEV))
    order = [2, 0, 2, 1, 2]
    src = torch.tensor([16 * p + i for p in order for i in range(16)], device=DEV)
    api.kv_cache_write(dense, k[src], v[src], torch.arange(80, device=DEV))
    lens = torch.arange(0, 81, dtype=torch.int32, device=DEV)
    q = C.rows((1, 4, d), 3).to(DEV).expand(81, 4, d)
    a = api.attention_decode(q, cache, torch.tensor([order], dtype=torch.int32, device=DEV).expand(81, 5), lens)
    b = api.attention_decode(q, dense, torch.arange(5, dtype=torch.int32, device=DEV).view(1, 5).expand(81, 5), lens)
    assert torch.equal(a, b) and not a[0].any()


def test_layer_without_tokens():
    g = torch.Generator().manual_seed(0)
    qkv = (0.06 * torch.randn(8 * 64, 256, generator=g)).to(BF).to(DEV)
    out = (0.05 * torch.randn(256, 4 * 64, generator=g)).to(BF).to(DEV)
    layer = attention.QuantizedAttention(qkv, out, 4, 2)
    cache = C.make_cache("fp8", 2, 16, 2, 64)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    y = layer(torch.empty((0, 256), dtype=BF, device=DEV), cache, torch.empty((0, 2), dtype=torch.int32, device=DEV),
              none.int(), none)
    assert y.shape == (0, 256) and y.dtype == BF


def training(d=64):
    w = [(1 + 0.1 * torch.randn(d, device=DEV)).requires_grad_() for _ in range(2)]
    return w, attention.QKNormRope(*w, attention.rotary_table(32, d, device=DEV)), torch.arange(7, device=DEV)


@pytest.mark.parametrize("which", [0, 1])
def test_one_of_them_under_autograd(which):
    w, layer, pos = training()
    x, dy = normal(7, 3, 64).requires_grad_(), normal(7, 3, 64)
    args, grads = [None, None], [None, None]
    args[which], grads[which] = x, dy
    y = layer(*args, pos)
    assert y[1 - which] is None
    y[which].backward(dy)
    args[which] = x.detach()
    want = api.qk_norm_rope_backward(layer.norm, *args, pos, *grads)
    assert torch.equal(x.grad, want[which])
    assert torch.equal(layer.main_grad[which], want[2 + which]) and not layer.main_grad[1 - which].any()


def test_weights_that_change_or_move():
    w, layer, pos = training()
    q, k = normal(7, 4, 64).requires_grad_(), normal(7, 2, 64).requires_grad_()
    y = layer(q, k, pos)
    with torch.no_grad():
        w[1].mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.backward(y, [torch.ones_like(t) for t in y])
    for t in w:
        t.data = 3 * t.data
    got = layer(q, k, pos)
    want = api.qk_norm_rope(api.QKNorm(*(t.detach() for t in w), layer.norm.table), q.detach(), k.detach(), pos)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    torch.autograd.backward(got, [torch.ones_like(t) for t in got])
    assert torch.isfinite(layer.main_grad).all()


def test_no_gradient_of_the_gradient():
    w, layer, pos = training()
    q, k = normal(7, 4, 64).requires_grad_(), normal(7, 2, 64).requires_grad_()
    y, _ = layer(q, k, pos)
    dq, = torch.autograd.grad(y.float().square().sum(), q, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dq.float().sum().backward()
