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


class Codes:
    """What a quantized matrix stands for here: its values."""

    def __init__(self, x):
        self.codes, self.scales = x.detach().clone(), torch.ones(1)

    def operand(self):
        op = api.Operand()
        op._owner = self
        return op


@pytest.fixture
def plain_layer(monkeypatch):
    """An attention layer of 2 heads on 1 of 64 whose attention gives the queries."""
    monkeypatch.setattr(api, "quantize", lambda x, fmt, block="1d": Codes(x))
    monkeypatch.setattr(api, "gemm", lambda a, b, m, n, k, out_dtype: (
        a._owner.codes.float() @ b._owner.codes.float().T).to(out_dtype))
    monkeypatch.setattr(api, "kv_cache_write", lambda *a, **kw: None)
    monkeypatch.setattr(api, "attention_decode", lambda q, *a: q.contiguous())
    g = torch.Generator().manual_seed(0)
    qkv, out = (torch.randn(s, generator=g).to(BF) for s in ((4 * 64, 32), (32, 2 * 64)))
    return attention.QuantizedAttention(qkv, out, 2, 1)


def test_the_generating_layer_has_no_backward_pass(plain_layer):
    """It takes an input under autograd, with the same result, and says so when a gradient
    is asked of it; it used to hand on a result that wanted none."""
    x = torch.randn((3, 32), generator=torch.Generator().manual_seed(1)).to(BF)
    y = plain_layer(x, None, None, None, None)
    assert not y.requires_grad
    leaf = x.clone().requires_grad_()
    got = plain_layer(leaf, None, None, None, None)
    assert torch.equal(got, y) and got.requires_grad
    got += 1                                            # a residual, say
    with pytest.raises(RuntimeError, match="QuantizedAttention has no backward pass"):
        (got.float() + leaf.sum()).sum().backward()
    with torch.no_grad():
        assert not plain_layer(leaf, None, None, None, None).requires_grad


@pytest.mark.parametrize("what", ["q_weight", "k_weight", "table"])
def test_a_norm_whose_tensors_data_is_replaced(monkeypatch, what):
    """The calls get the addresses of the new data: the old memory may be gone."""
    got = []

    def launch(name, fn, device, *args):
        assert norm._at in args
        d = api.QKNormDesc.from_address(norm._at)
        got.append((d.q_weight, d.k_weight, d.table, d.weight_f32, d.rotary_dim))

    monkeypatch.setattr(api, "_launch", launch)
    monkeypatch.setattr(api, "_norm_workspace", lambda device, d: 16)
    t = dict(q_weight=torch.ones(64), k_weight=torch.ones(64), table=torch.ones((8, 32)))
    norm = api.QKNorm(**t)
    cache = api.KVCache.empty(2, 16, 1, 64, device="cpu")
    x, pos = torch.ones((5, 1, 64), dtype=BF), torch.arange(5)
    calls = [lambda: api.qk_norm_rope(norm, x, x, pos), lambda: api.qk_norm_rope_backward(norm, x, x, pos, x, x),
             lambda: api.kv_cache_write(cache, x, x, pos, q=x, norm=norm, positions=pos)]
    for call in calls:
        t[what].data = t[what].data.clone()
        call()
        assert got[-1] == (t["q_weight"].data_ptr(), t["k_weight"].data_ptr(), t["table"].data_ptr(), 1, 32)
    t["table"].data = torch.ones((9, 64), dtype=torch.float64)
    with pytest.raises(ValueError, match="table must be"):
        calls[0]()


def test_refresh_writes_the_codes_in_place(plain_layer):
    """A step that has been captured reads them where they were."""
    before = [op._owner for op in (plain_layer._qkv, plain_layer._out)]
    at = [(o.codes.data_ptr(), o.scales.data_ptr()) for o in before]
    ops = plain_layer._qkv, plain_layer._out
    plain_layer.qkv.mul_(2)
    plain_layer.out.add_(1)
    plain_layer.refresh()
    assert (plain_layer._qkv, plain_layer._out) == ops
    for o, w, a in zip(before, (plain_layer.qkv, plain_layer.out), at):
        assert torch.equal(o.codes, w) and (o.codes.data_ptr(), o.scales.data_ptr()) == a
    # weights of another shape are other codes
    plain_layer.out = torch.ones((48, 128), dtype=BF)
    plain_layer.refresh()
    assert plain_layer._out._owner.codes.shape == (48, 128) and plain_layer._qkv is ops[0]


def test_refresh_of_a_layer_made_in_inference_mode(plain_layer):
    """Its codes may not be changed outside that mode, so they are changed in it; and those
    of a layer made outside may be changed inside."""
    with torch.inference_mode():
        inside = attention.QuantizedAttention(plain_layer.qkv, plain_layer.out, 2, 1)
        plain_layer.qkv.add_(1)
        plain_layer.refresh()
    at = inside._qkv._owner.codes.data_ptr()
    inside.refresh()
    assert inside._qkv._owner.codes.data_ptr() == at
    for layer in (inside, plain_layer):
        assert torch.equal(layer._qkv._owner.codes, plain_layer.qkv)
