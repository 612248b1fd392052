"""Shared by the tests of attention on a quantized cache: pools of several
layouts, the oracle's copies of them, and comparison with values of a known
error that were rounded once."""
import numpy as np
import torch

from fp4_block_scaled_x16_amd import api
from oracle import attention as A

DEV = "cuda"
U = 2.0 ** -24       # half a step of fp32, relative
FORMATS = ["fp8", "mxfp8", "mxfp4", "nvfp4", "ue5m3"]
DIMS = [64, 128, 256]
TARGET = {"ue5m3": 2048.0}


def row_bytes(fmt, d):
    return d if fmt in ("fp8", "mxfp8") else d // 2


def blocks(fmt, d):
    return -(-d // A.BLOCK[fmt])


def pools(fmt, pages, page, heads, d, layout="heads", seed=0, device=DEV):
    """uint8 pools of random bytes: (k_codes, k_scales, v_codes, v_scales).
    "heads": a page's heads one after the other; "places": its places, each with
    all heads; "layers": the second layer of a pool of three."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        w, b = row_bytes(fmt, d), blocks(fmt, d)
        rnd = lambda *shape: torch.randint(0, 256, shape, dtype=torch.uint8, generator=g).to(device)   # noqa: E731
        if layout == "heads":
            out += [rnd(pages, heads, page, w), rnd(pages, heads, b, page)]
        elif layout == "places":
            out += [rnd(pages, page, heads, w).permute(0, 2, 1, 3), rnd(pages, b, heads, page).transpose(1, 2)]
        else:
            out += [rnd(pages, 3, heads, page, w)[:, 1], rnd(pages, 3, heads, b, page)[:, 1]]
    return out


def make_cache(fmt, pages, page, heads, d, layout="heads", seed=0, amax=(4.0, 3.0), device=DEV):
    am = torch.tensor(amax, dtype=torch.float32, device=device) if fmt in A.TWO_LEVEL else None
    return api.KVCache(fmt, *pools(fmt, pages, page, heads, d, layout, seed, device), amax=am,
                       target=TARGET.get(fmt, 448.0))


def tensors(cache):
    return cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales


def contents(cache):
    """numpy copies of the pools."""
    return [t.cpu().numpy().copy() for t in tensors(cache)]


def name_of(cache):
    return {v: k for k, v in api.FORMATS.items()}[cache.fmt]


def bits(t):
    """uint16 bits of a bf16 tensor."""
    return t.contiguous().cpu().view(torch.int16).numpy().view(np.uint16)


def encoded(cache, i, rows):
    """The oracle's (codes, scales) of bf16 rows [N, heads, d] as K (0) or V (1)."""
    fmt, n = name_of(cache), rows.shape[0]
    amax = float(cache.amax[i]) if cache.amax is not None else None
    c, s = A.encode_rows(bits(rows).reshape(-1, cache.head_dim), fmt, amax, cache.target)
    return c.reshape(n, cache.heads, -1), s.reshape(n, cache.heads, -1)


def values(cache, pool, i, page, place):
    """float64 values [.., heads, d] of places of the oracle's pools."""
    fmt = name_of(cache)
    codes, scales = pool[2 * i][page, :, place], pool[2 * i + 1][page, :, :, place]
    dec = A.s_dec(fmt, float(cache.amax[i]) if cache.amax is not None else 1.0, cache.target)
    v = A.row_values(codes.reshape(-1, codes.shape[-1]), scales.reshape(-1, scales.shape[-1]), fmt,
                     cache.head_dim, dec)
    return v.reshape(codes.shape[:-1] + (cache.head_dim,))


def rows(shape, seed, sigma=1.0):
    """Normal bf16 values with rows of different sizes, a zero row and a few outliers."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal(shape).astype(np.float32) * np.float32(sigma)
    v *= np.exp2(np.arange(shape[0]) % 7 - 3.0).astype(np.float32)[:, None, None]
    v[rng.random(shape) < 0.003] *= np.float32(20)
    if shape[0] > 3:
        v[2] = 0.0
    return torch.from_numpy(v).to(torch.bfloat16)


def table(n, rot, dtype=np.float32):
    """cos | sin of positions 0 .. n - 1."""
    a = np.arange(n)[:, None] * np.exp(np.arange(rot // 2) * (-2.0 / rot * np.log(1e4)))
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(dtype)


def turned(size, cos, sin, interleaved=False):
    """|a cos| + |b sin| and |b cos| + |a sin| of magnitudes [.., D]."""
    if cos is None:
        return size
    c, s = np.abs(cos), np.abs(sin)
    return np.maximum(A.turn(size, c, s, interleaved), A.turn(size, c, s, interleaved, back=True))


def as64(t):
    return t.detach().cpu().double().numpy()


def near(t, v, err):
    """t holds values within err of v, rounded once to its type (half a step of the
    binade's top; a subnormal's)."""
    dtype_bits, low = {torch.bfloat16: (8, -126), torch.float32: (24, -126)}[t.dtype]
    mag = np.maximum(np.abs(v) + err, 2.0 ** low)
    half = np.exp2(np.floor(np.log2(mag)) - dtype_bits)
    got = as64(t)
    bad = ~(np.abs(got - v) <= half + err)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].tolist(), float(np.abs(got - v)[bad].max()))
