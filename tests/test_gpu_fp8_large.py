"""The FP8 operators on matrices of more than 2^32 elements: the last tiles
against the same operator on the last rows alone, bit for bit."""
import pytest
import torch

from fp4_block_scaled_x16_amd import api
from fp8_check import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROWS, COLS = 65664, 65536               # 513 and 512 tiles of 128: 2^32 + 2^23 elements
TAIL = 128


def random(rows, cols, scale=1.0):
    x = torch.empty((rows, cols), dtype=BF, device=DEV)
    return x.normal_(0.0, scale)


def same_rows(whole, tail):
    """Rowwise codes of the last TAIL rows."""
    assert torch.equal(whole.codes[-TAIL:], tail.codes)
    assert torch.equal(whole.scales[:, whole.rows - TAIL:whole.rows], tail.scales[:, :TAIL])


def same_columns(whole, tail):
    """Codes of the transpose whose last block along the rows is the tail."""
    assert torch.equal(whole.codes[:, -TAIL:], tail.codes)
    assert torch.equal(whole.scales[-1, :whole.rows], tail.scales[0, :whole.rows])


def test_quantize_transpose_and_values():
    x = random(ROWS, COLS)
    q, qt = api.quantize_dual(x, "fp8")
    tail = x[-TAIL:].clone()
    t, tt = api.quantize_dual(tail, "fp8")
    same_rows(q, t)
    same_columns(qt, tt)
    del qt
    same_columns(api.requantize_t(q), api.requantize_t(t))
    del x
    assert torch.equal(api.dequantize(q, torch.bfloat16)[-TAIL:], api.dequantize(t, torch.bfloat16))


@pytest.mark.parametrize("act", ["swiglu", "relu2"])
def test_activation(act):
    F = COLS // 2 if act == "swiglu" else COLS
    h = random(ROWS, COLS)
    a, qh = api.act_quantize(h, act)
    ta, tqh = api.act_quantize(h[-TAIL:].clone(), act)
    del h
    same_rows(a, ta)
    same_rows(qh, tqh)
    del a
    da = random(ROWS, F, 1e-2)
    got = api.act_backward(qh, da, act, fmt="fp8_e5m2")
    want = api.act_backward(tqh, da[-TAIL:].clone(), act, fmt="fp8_e5m2")
    same_rows(got[0], want[0])
    same_columns(got[1], want[1])
    same_columns(got[2], want[2])


@pytest.mark.parametrize("out", [torch.float32, BF])
def test_product(out):
    """Small whole numbers, exact in every kernel."""
    K = 192
    x, w = (torch.randint(-3, 4, (n, K), device=DEV, dtype=torch.int8).to(BF) for n in (ROWS, COLS))
    b = api.quantize(w, "fp8")
    d = api.gemm(api.quantize(x, "fp8").operand(), b.operand(), ROWS, COLS, K, out_dtype=out)
    t = api.gemm(api.quantize(x[-TAIL:].clone(), "fp8").operand(), b.operand(), TAIL, COLS, K, out_dtype=out)
    assert torch.equal(d[-TAIL:], t)
    want = (x[-TAIL:].double() @ w[-256:].double().t()).to(out)
    assert torch.equal(d[-TAIL:, -256:], want)
