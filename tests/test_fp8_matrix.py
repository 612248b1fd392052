"""api.fp8_matrix: codes and scales that exist already, by their dtypes."""
import pytest
import torch

from fp4_block_scaled_x16_amd import api

E4M3, E5M2, E8M0 = torch.float8_e4m3fn, torch.float8_e5m2, torch.float8_e8m0fnu
FNUZ = [torch.float8_e4m3fnuz, torch.float8_e5m2fnuz]


def pair(codes=torch.uint8, scales=torch.uint8):
    return (torch.zeros((3, 256), dtype=torch.uint8).view(codes),
            torch.zeros((2, 16), dtype=torch.uint8).view(scales))


@pytest.mark.parametrize("scales", [torch.uint8, E8M0])
@pytest.mark.parametrize("codes,fmt", [(torch.uint8, "fp8"), (torch.uint8, "fp8_e5m2"), (E4M3, "fp8"),
                                       (E5M2, "fp8_e5m2"), (E4M3, api.FP8_E4M3)])
def test_takes(codes, fmt, scales):
    c, s = pair(codes, scales)
    q = api.fp8_matrix(c, s, 3, 200, fmt)
    assert q.codes.dtype == q.scales.dtype == torch.uint8
    assert q.codes.data_ptr() == c.data_ptr() and q.scales.data_ptr() == s.data_ptr()
    assert q.fmt == api._fmt(fmt) and (q.rows, q.cols) == (3, 200)


@pytest.mark.parametrize("codes,fmt", [(E5M2, "fp8"), (E4M3, "fp8_e5m2"), (torch.int8, "fp8"),
                                       (torch.bool, "fp8"), (E8M0, "fp8")] +
                         [(f, fmt) for f in FNUZ for fmt in ("fp8", "fp8_e5m2")])
def test_refuses_codes_of_another_type(codes, fmt):
    """Their bytes would be read as values that they are not."""
    with pytest.raises(ValueError, match="codes"):
        api.fp8_matrix(*pair(codes), 3, 200, fmt)


@pytest.mark.parametrize("scales", [E4M3, E5M2, torch.int8, torch.bool] + FNUZ)
def test_refuses_scales_of_another_type(scales):
    with pytest.raises(ValueError, match="scales"):
        api.fp8_matrix(*pair(scales=scales), 3, 200)


@pytest.mark.parametrize("which", [0, 1])
def test_refuses_wider_elements(which):
    """(A view of them as bytes has another shape, but may have the right one.)"""
    c, s = pair()
    bad = ((torch.zeros((3, 64), dtype=torch.float32), s), (c, torch.zeros((2, 4), dtype=torch.float32)))[which]
    with pytest.raises(ValueError):
        api.fp8_matrix(*bad, 3, 200)
