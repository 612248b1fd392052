"""K through norm and rotation into a cache whose blocks have tensor scales: its values in 64
bits, rounded once to fp32 (to odd), go through the quantizer's own fp32 steps."""
import numpy as np
import pytest
import torch

import kv_check as C
from fp4_block_scaled_x16_amd import api
from kv_check import DEV
from oracle import attention as A
from oracle import quantize as Q

pytestmark = pytest.mark.gpu


def to_odd(y):
    """fp32 of float64 y: cut off, and the last bit set where something was."""
    f = y.astype(np.float32)
    f = np.where(np.abs(f.astype(np.float64)) > np.abs(y), np.nextafter(f, np.float32(0)), f)
    bits = f.view(np.uint32) | (f.astype(np.float64) != y).astype(np.uint32)
    return bits.view(np.float32)


def test_to_odd():
    x = np.array([1.0, 1 + 2.0 ** -24, 1 + 2.0 ** -23, 1 + 3 * 2.0 ** -24, -1 - 2.0 ** -40, 0.0, 2.0 ** -3])
    want = np.array([1.0, 1 + 2.0 ** -23, 1 + 2.0 ** -23, 1 + 2.0 ** -23, -1 - 2.0 ** -23, 0.0, 2.0 ** -3])
    assert np.array_equal(to_odd(x), want.astype(np.float32))


@pytest.mark.parametrize("style,rot", [("half", 128), ("interleaved", 64), ("half", 0)])
@pytest.mark.parametrize("fmt,amax", [("nvfp4", 9.0), ("nvfp4", 1.7), ("ue5m3", 9.0)])
def test_codes_are_those_of_the_quantizers_steps(fmt, amax, style, rot):
    d, heads, tokens, page, eps = 128, 4, 500, 16, float(np.float32(1e-6))
    cache = C.make_cache(fmt, 32, page, heads, d, amax=(amax, 3.0))
    k = C.rows((tokens, heads, d), 5).to(DEV)
    w = [1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(i)).to(DEV) for i in range(2)]
    tab = torch.from_numpy(C.table(tokens, rot)).to(DEV) if rot else None
    pos = slots = torch.arange(tokens, device=DEV)
    api.kv_cache_write(cache, k, k, slots, norm=api.QKNorm(*w, tab, eps=eps, style=style), positions=pos)
    c = s = None
    if rot:
        t = C.as64(tab)[:, None]
        c, s = t[..., :rot // 2], t[..., rot // 2:]
    y = to_odd(A.norm_rope(C.as64(k), C.as64(w[1]), c, s, eps, style == "interleaved")).reshape(-1, d // 16, 16)
    enc, dec = Q.global_scales(np.float32(amax), cache.target)[:2]
    scales, by, _ = Q.block_scales_two_level(np.abs(y).max(2), enc, dec, fmt)
    codes = Q.pack_codes(Q.encode_elements(y, by[..., None])[0].reshape(-1, d))
    at = np.arange(tokens)
    got = C.contents(cache)
    assert np.array_equal(got[1][at // page, :, :, at % page].reshape(-1, d // 16), scales)
    assert np.array_equal(got[0][at // page, :, at % page].reshape(-1, d // 2), codes)
