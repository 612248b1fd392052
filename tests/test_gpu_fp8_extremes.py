"""The largest bf16 values in the FP8 formats: those that round up to 2^128, and
the largest that do not."""
import pytest
import torch

from fp4_block_scaled_x16_amd import api
from fp8_check import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,first,below", [("fp8", 248, 240), ("fp8_e5m2", 240, 224)])
def test_the_largest_values(fmt, first, below):
    """first * 2^120 is half way between the format's last value below 2^128 and
    2^128 itself, whose significand is the even one."""
    n = torch.arange(192, 256, dtype=torch.float64)
    x = (n * 2.0 ** 120).to(torch.bfloat16)
    assert torch.equal(x.double(), n * 2.0 ** 120)
    x = torch.stack([x, -x]).to(DEV)
    for q in (api.quantize(x, fmt), api.quantize(x.repeat(9, 1), fmt, block="2d")):
        for dtype in (torch.float32, torch.bfloat16):
            v = api.dequantize(q, dtype).double().cpu()[:2]
            assert torch.equal(v[0], -v[1])
            assert bool((v[0][n >= first] == torch.inf).all())
            assert bool((v[0][n < first] <= below * 2.0 ** 120).all())
            assert float(v[0][n < first].max()) == below * 2.0 ** 120


def test_a_product_in_fp32():
    x = torch.tensor([[247.0, 0], [248, 0]]) * 2.0 ** 120
    a = api.quantize(torch.nn.functional.pad(x, (0, 6)).to(torch.bfloat16).to(DEV), "fp8")
    b = api.quantize(torch.full((3, 8), 2.0 ** -20, dtype=torch.bfloat16, device=DEV), "fp8")
    d = api.gemm(a.operand(), b.operand(), 2, 3, 8).cpu()
    assert bool((d[0] == 240 * 2.0 ** 100).all()) and bool((d[1] == torch.inf).logical_or(d[1].isnan()).all())
