"""Which pools a KVCache takes: the strides of dimensions with one entry mean nothing."""
import pytest
import torch

from fp4_block_scaled_x16_amd import api


def pools(pages, heads, page=16, d=128, fmt="mxfp8"):
    """Dense K and V."""
    w, b = (d, d // 32) if fmt == "mxfp8" else (d // 2, d // 32)
    return [torch.zeros(s, dtype=torch.uint8) for _ in range(2) for s in ((pages, heads, page, w), (pages, heads, b, page))]


def odd_stride(t, i, stride):
    """t with another stride of dimension i."""
    s = list(t.stride())
    s[i] = stride
    return t.as_strided(t.shape, s)


@pytest.mark.parametrize("which", range(4))
@pytest.mark.parametrize("dim,pages,heads", [(0, 1, 4), (1, 3, 1)])
def test_one_page_or_one_head_with_any_stride(which, dim, pages, heads):
    want = api.KVCache("mxfp8", *pools(pages, heads))._desc
    p = pools(pages, heads)
    p[which] = odd_stride(p[which], dim, 7)
    got = api.KVCache("mxfp8", *p)._desc
    for name in ("page_stride", "head_stride", "token_stride", "scale_page_stride", "scale_head_stride",
                 "scale_block_stride"):
        assert getattr(got, name) == getattr(want, name) and getattr(got, name) % 16 == 0


def test_one_block_with_any_stride():
    p = [torch.zeros(s, dtype=torch.uint8) for _ in range(2) for s in ((2, 3, 16, 128), (2, 3, 1, 16))]
    p[3] = odd_stride(p[3], 2, 5)
    assert api.KVCache("fp8", *p)._desc.scale_block_stride == 16


@pytest.mark.parametrize("which", range(4))
def test_strides_that_mean_something_are_compared(which):
    p = [t.unsqueeze(0).expand(3, *t.shape).contiguous()[1] for t in pools(2, 3)]
    api.KVCache("mxfp8", *p)
    shape = p[which].shape
    p[which] = torch.zeros((2, 4, *shape[2:]), dtype=torch.uint8)[:, :3]
    with pytest.raises(ValueError, match="strides alike"):
        api.KVCache("mxfp8", *p)
    p[which] = torch.zeros((*shape[:2], shape[3], shape[2]), dtype=torch.uint8).transpose(2, 3)
    with pytest.raises(ValueError, match="last dimension contiguous"):
        api.KVCache("mxfp8", *p)
