"""The attention layers around their kernels: what they keep, refuse and hand on.  The
kernels are stood in for by plain tensor operations, so this runs on the CPU."""
import pytest
import torch

from fp4_block_scaled_x16_amd import api, attention

BF = torch.bfloat16


@pytest.fixture
def plain_norm(monkeypatch):
    """Each head times its weight and the first angle's cosine, and what the calls got."""
    calls = []

    def forward(norm, q, k, positions=None):
        calls.append(norm)
        c = norm.table[positions, :1].unsqueeze(-1)
        return tuple(None if x is None else (x.float() * w.float() * c).to(BF)
                     for x, w in ((q, norm.q_weight), (k, norm.k_weight)))

    def backward(norm, q, k, positions, dq, dk, weight_grads):
        c = norm.table[positions, :1].unsqueeze(-1)
        got = [(d.float() * w.float() * c).to(BF) for d, w in ((dq, norm.q_weight), (dk, norm.k_weight))]
        return *got, None, None

    monkeypatch.setattr(api, "qk_norm_rope", forward)
    monkeypatch.setattr(api, "qk_norm_rope_backward", backward)
    return calls


def training(d=64):
    w = [torch.full((d,), 2.0 + i).requires_grad_() for i in range(2)]
    table = torch.arange(1.0, 9.0).unsqueeze(1).expand(8, 32).contiguous()
    layer = attention.QKNormRope(*w, table)
    q, k = (torch.ones((5, h, d), dtype=BF).requires_grad_() for h in (2, 1))
    return layer, table, q, k, torch.arange(5)


def test_a_table_that_changes_between_the_passes(plain_norm):
    """Its gradient would be that of other angles: refused, as changed weights are."""
    layer, table, q, k, pos = training()
    y = layer(q, k, pos)
    table.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.backward(y, [torch.ones_like(t) for t in y])
    y = layer(q, k, pos)
    torch.autograd.backward(y, [torch.ones_like(t) for t in y])
    assert torch.equal(q.grad[:, 0, 0].float(), 4.0 * torch.arange(1.0, 6.0))


def test_a_table_made_in_inference_mode(plain_norm):
    """It has no versions to go by and is used as it is."""
    with torch.inference_mode():
        table = torch.ones((8, 32))
    layer = attention.QKNormRope(torch.ones(64).requires_grad_(), torch.ones(64).requires_grad_(), table)
    q = torch.ones((5, 2, 64), dtype=BF).requires_grad_()
    y, k = layer(q, torch.ones((5, 1, 64), dtype=BF).requires_grad_(), torch.arange(5))
    torch.autograd.backward((y, k), (torch.ones_like(y), torch.ones_like(k)))
    assert torch.all(q.grad == 1)
