"""The scale layouts that quantize and quantize_dual take for the FP8 formats:
K-major ones, by default or by name, on either side.  The library's own checks
answer, before any device work."""
import pytest
import torch

from fp4_block_scaled_x16_amd import api

X = torch.zeros((128, 128), dtype=torch.bfloat16)


@pytest.fixture
def status(monkeypatch):
    """The status of each library call, which runs to its checks on host tensors
    (one that passes them finds no device, or its launch is left out)."""
    got = []

    def launch(what, fn, device, *args):
        args = [a for a in args]
        rows = 3 if what == "fp4_quantize_dual" else 2
        args[rows] = 0                               # no rows: accepted without device work
        got.append(fn(*args, None))

    monkeypatch.setattr(api, "_launch", launch)
    return got


@pytest.mark.parametrize("kw", [dict(), dict(scale_layout="kmajor"), dict(scale_layout_t="kmajor"),
                                dict(scale_layout="kmajor", scale_layout_t="kmajor"), dict(scale_layout=2)])
def test_dual_takes(status, kw):
    api.quantize_dual(X, "fp8", **kw)
    assert status == [0]


@pytest.mark.parametrize("kw", [dict(scale_layout="tiled"), dict(scale_layout="rowmajor"),
                                dict(scale_layout_t="tiled"), dict(scale_layout_t="rowmajor"),
                                dict(scale_layout="kmajor", scale_layout_t="tiled"),
                                dict(scale_layout="tiled", scale_layout_t="kmajor"),
                                dict(scale_layout="kmajor", scale_layout_t=0)])
@pytest.mark.parametrize("fmt", ["fp8", "fp8_e5m2"])
def test_dual_refuses(status, fmt, kw):
    api.quantize_dual(X, fmt, **kw)
    assert status == [3]


@pytest.mark.parametrize("orient", ["row", "col"])
def test_single(status, orient):
    for layout, want in ((None, 0), ("kmajor", 0), ("tiled", 3), ("rowmajor", 3)):
        api.quantize(X, "fp8", orient=orient, scale_layout=layout)
        assert status.pop() == want
