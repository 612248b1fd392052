"""Norm and rotation of queries and keys on the GPU, forward and backward, against
the formulas in 64 bits (within the derived error of their fp32 steps and one
rounding), and the gradients against differences of the forward formula."""
import numpy as np
import pytest
import torch

import kv_check as C
from fp4_block_scaled_x16_amd import api, attention
from kv_check import DEV, DIMS, U
from oracle import attention as A

pytestmark = pytest.mark.gpu
EPS = 1e-5
SIZES = [(1, 1, 1), (1, 32, 8), (3, 5, 5), (67, 7, 1), (130, 8, 2)]


def setup(tokens, hq, hk, d, rot, w_dtype, seed):
    """(q, k, norm's tensors, positions) on the GPU, q and k parts of one projection."""
    x = C.rows((tokens, hq + hk + 1, d), seed).to(DEV)
    g = torch.Generator().manual_seed(seed)
    w = [None, None] if w_dtype is None else [(1 + 0.3 * torch.randn(d, generator=g)).to(w_dtype).to(DEV) for _ in range(2)]
    tab = torch.from_numpy(C.table(200, rot)).to(DEV) if rot else None
    pos = torch.randint(0, 200, (tokens,), generator=g).to(DEV) if rot else None
    return x[:, :hq], x[:, hq:hq + hk], w, tab, pos


def angles(tab, pos):
    if tab is None:
        return None, None
    t = C.as64(tab)[pos.cpu().numpy()][:, None]
    return np.split(t, 2, -1)


# fp32 steps of y = r (x (w c) + xp (wp s)): the sum of squares adds up at most 8 + 5
# terms per lane and step, half of which (with the mean, eps and the root) is in r:
# 9 roundings; the products and the sum 6 more; 16 in all
def forward_err(x, w, c, s, inter):
    size = np.abs(x) if w is None else np.abs(x * A.inv_rms(x, EPS) * w)
    return 16 * U * C.turned(size, c, s, inter)


@pytest.mark.parametrize("tokens,hq,hk", SIZES)
@pytest.mark.parametrize("rot,style,w_dtype", [(1, "half", torch.bfloat16), (0.5, "interleaved", torch.float32),
                                               (0.25, "half", torch.float32), (0, "half", torch.bfloat16),
                                               (1, "interleaved", None)])
@pytest.mark.parametrize("d", DIMS)
def test_forward_and_backward(d, rot, style, w_dtype, tokens, hq, hk):
    rot, inter = int(rot * d), style == "interleaved"
    q, k, w, tab, pos = setup(tokens, hq, hk, d, rot, w_dtype, tokens + d)
    norm = api.QKNorm(*w, tab, eps=EPS, style=style)
    c, s = angles(tab, pos)
    y = api.qk_norm_rope(norm, q, k, pos)
    dy = [(1e-2 * C.rows(tuple(t.shape), 77 + i).float()).to(torch.bfloat16).to(DEV) for i, t in enumerate((q, k))]
    got = api.qk_norm_rope_backward(norm, q, k, pos, *dy)
    for i, x in enumerate((q, k)):
        x64, w64 = C.as64(x), None if w[i] is None else C.as64(w[i])
        C.near(y[i], A.norm_rope(x64, w64, c, s, EPS, inter), forward_err(x64, w64, c, s, inter))
        dx, dw = A.norm_rope_grad(x64, w64, c, s, EPS, C.as64(dy[i]), inter)
        dz = C.turned(np.abs(C.as64(dy[i])), c, s, inter)            # sizes of dz's terms
        if w64 is None:
            C.near(got[i], dx, 4 * U * dz)
            assert got[2 + i] is None
            continue
        r = A.inv_rms(x64, EPS)
        xr, g = np.abs(x64 * r), dz * np.abs(w64)
        # dz 3 roundings, g one more, r 10, each term of the mean 14 and its sum 14,
        # the difference and the last product 12
        C.near(got[i], dx, r * (16 * U * g + 56 * U * xr * np.mean(g * xr, -1, keepdims=True)))
        # any order of adding n terms errs by n - 1 half steps of their sizes
        n = tokens * x.shape[1]
        err = (n + 64) * U * (dz * xr).reshape(-1, d).sum(0)
        assert np.all(np.abs(C.as64(got[2 + i]) - dw) <= err + U * np.abs(dw))


def test_gradients_against_differences():
    """The backward pass along random directions, against central differences of the
    64-bit forward: gradients in bf16 (rounded by 2^-8 of themselves at most)."""
    d, rot = 64, 32
    q, k, w, tab, pos = setup(5, 3, 2, d, rot, torch.float32, 9)
    norm = api.QKNorm(*w, tab, eps=EPS)
    c, s = angles(tab, pos)
    rng = np.random.default_rng(1)
    dy = [torch.from_numpy(rng.standard_normal(tuple(t.shape)).astype(np.float32)).to(torch.bfloat16).to(DEV) for t in (q, k)]
    got = api.qk_norm_rope_backward(norm, q, k, pos, *dy)
    for i, x in enumerate((q, k)):
        x64, w64, dy64 = C.as64(x), C.as64(w[i]), C.as64(dy[i])
        def loss(a, b):
            return (A.norm_rope(a, b, c, s, EPS) * dy64).sum()
        live = np.abs(x64).max(-1, keepdims=True) > 0                # at a zero row r is not smooth to this step
        for _ in range(4):
            t = rng.standard_normal(x64.shape) * live * np.abs(x64).max(-1, keepdims=True)
            h = 1e-5
            num = (loss(x64 + h * t, w64) - loss(x64 - h * t, w64)) / (2 * h)
            g = C.as64(got[i])
            # bf16's rounding of each element of the gradient; differences to 1e-6
            assert abs((g * t).sum() - num) <= 2.0 ** -8 * np.abs(g * t).sum() + 1e-6 * np.abs(dy64).sum()
            u = rng.standard_normal(d)
            num = (loss(x64, w64 + h * u) - loss(x64, w64 - h * u)) / (2 * h)
            assert abs((C.as64(got[2 + i]) * u).sum() - num) <= 1e-5 * np.abs(dy64).sum()


@pytest.mark.parametrize("which", ["q", "k"])
def test_one_of_them(which):
    q, k, w, tab, pos = setup(11, 4, 2, 128, 128, torch.bfloat16, 2)
    norm = api.QKNorm(*w, tab)
    both = api.qk_norm_rope(norm, q, k, pos)
    grads = api.qk_norm_rope_backward(norm, q, k, pos, *both)
    i = "qk".index(which)
    args = [q, k]
    args[1 - i] = None
    one = api.qk_norm_rope(norm, *args, pos)
    assert one[1 - i] is None and torch.equal(one[i], both[i])
    got = api.qk_norm_rope_backward(norm, *args, pos, *both)
    assert got[1 - i] is None and got[3 - i] is None
    assert torch.equal(got[i], grads[i])
    assert torch.allclose(got[2 + i], grads[2 + i], rtol=1e-4, atol=1e-4)     # other groups of the same sum
    none = api.qk_norm_rope_backward(norm, q, k, pos, *both, weight_grads=False)
    assert none[2] is none[3] is None and torch.equal(none[0], grads[0])


def test_in_place_and_into_one_buffer():
    """Outputs that are the inputs, and gradients that are parts of the projection's."""
    q, k, w, tab, pos = setup(19, 6, 2, 64, 64, torch.bfloat16, 4)
    norm = api.QKNorm(*w, tab)
    want = api.qk_norm_rope(norm, q, k, pos)
    grads = api.qk_norm_rope_backward(norm, q, k, pos, *want)
    buf = torch.full((19, 10, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    got = api.qk_norm_rope_backward(norm, q, k, pos, *want, out=(buf[:, 1:7], buf[:, 7:9]))
    assert torch.equal(got[0], grads[0]) and torch.equal(buf[:, 7:9], grads[1])
    assert torch.isnan(buf[:, 0]).all() and torch.isnan(buf[:, 9]).all()
    dq, dk = (t.clone() for t in want)
    api.qk_norm_rope_backward(norm, q, k, pos, dq, dk, out=(dq, dk))
    assert torch.equal(dq, grads[0]) and torch.equal(dk, grads[1])
    x = torch.cat([q, k], 1)
    api.qk_norm_rope(norm, x[:, :6], x[:, 6:], pos, out=(x[:, :6], x[:, 6:]))
    assert torch.equal(x[:, :6], want[0]) and torch.equal(x[:, 6:], want[1])
    heads_out = k.transpose(0, 1).contiguous().transpose(0, 1)       # heads outermost
    assert torch.equal(api.qk_norm_rope(norm, None, heads_out, pos, out=(None, torch.empty_like(heads_out)))[1], want[1])


def test_positions_outside_the_table():
    """Rotated elements of such a token are NaN, the others and other tokens as ever."""
    q, k, w, tab, pos = setup(6, 2, 1, 64, 32, torch.bfloat16, 6)
    norm = api.QKNorm(*w, tab)
    want = api.qk_norm_rope(norm, q, k, pos)
    bad = pos.clone()
    bad[1], bad[4] = -1, 200
    got = api.qk_norm_rope(norm, q, k, bad)
    for a, b in zip(got, want):
        ok = [0, 2, 3, 5]
        assert torch.equal(a[ok], b[ok]) and torch.equal(a[..., 32:], b[..., 32:])
        assert torch.isnan(a[[1, 4], :, :32]).all()


def test_zero_rows_and_no_tokens():
    w = [torch.ones(128, dtype=torch.float32, device=DEV) for _ in range(2)]
    norm = api.QKNorm(*w)
    zero = torch.zeros((3, 2, 128), dtype=torch.bfloat16, device=DEV)
    y, _ = api.qk_norm_rope(norm, zero, None)
    assert not y.any()
    none = torch.empty((0, 2, 128), dtype=torch.bfloat16, device=DEV)
    assert api.qk_norm_rope(norm, none, none)[0].shape == (0, 2, 128)
    dq, dk, dwq, dwk = api.qk_norm_rope_backward(norm, none, none, None, none, none)
    assert dq.shape == dk.shape == (0, 2, 128) and not dwq.any() and not dwk.any()


def test_large_and_small_rows():
    """Squares that would pass fp32's range do not: rows up to 2^60 and down to 2^-60
    (with eps = 0)."""
    x = torch.ones((2, 1, 64), dtype=torch.bfloat16)
    x[0] *= 2.0 ** 60
    x[1] *= 2.0 ** -60
    x[:, :, ::2] *= -1
    norm = api.QKNorm(*(torch.ones(64, device=DEV) for _ in range(2)), eps=0.0)
    y, _ = api.qk_norm_rope(norm, x.to(DEV), None)
    assert torch.equal(y.cpu(), torch.sign(x.float()).to(torch.bfloat16))


def layer_setup(tokens=13, seed=3):
    tab = attention.rotary_table(200, 64, device=DEV)
    q, k, w, _, pos = setup(tokens, 4, 2, 64, 64, torch.float32, seed)
    w = [t.clone().requires_grad_() for t in w]
    return q, k, w, tab, pos, attention.QKNormRope(*w, tab)


def test_autograd():
    """The layer under autograd gives what the two calls give; weight gradients are
    added to main_grad, and hooks on the weights run when they are."""
    q, k, w, tab, pos, layer = layer_setup()
    qkv = torch.cat([q, k], 1).requires_grad_()
    seen = []
    w[1].register_post_accumulate_grad_hook(lambda t: seen.append(layer.main_grad.clone()))
    want_w = 0
    for step in range(2):
        y = layer(qkv[:, :4], qkv[:, 4:], pos)
        plain = api.qk_norm_rope(layer.norm, q, k, pos)
        assert torch.equal(y[0], plain[0]) and torch.equal(y[1], plain[1])
        dy = [torch.randn_like(t.float()).to(torch.bfloat16) for t in plain]
        qkv.grad = None
        torch.autograd.backward(y, [t.transpose(0, 1).contiguous().transpose(0, 1) for t in dy])
        want = api.qk_norm_rope_backward(layer.norm, q, k, pos, *dy)
        assert torch.equal(qkv.grad, torch.cat(want[:2], 1))
        want_w = want_w + torch.stack(want[2:])
        assert torch.equal(layer.main_grad, want_w)
        assert len(seen) == step + 1 and torch.equal(seen[-1], want_w)
        assert w[0].grad is None
    with torch.no_grad():
        assert not layer(q, k, pos)[0].requires_grad


def test_rotation_alone_under_autograd():
    q, k, w, tab, pos = setup(7, 2, 2, 128, 64, None, 5)
    layer = attention.QKNormRope(table=tab)
    q = q.clone().requires_grad_()
    y, _ = layer(q, k, pos)
    (y.float() * C.rows((7, 2, 128), 8).to(DEV).float()).sum().backward()
    dy = C.rows((7, 2, 128), 8).to(DEV)
    want = api.qk_norm_rope_backward(layer.norm, q.detach(), None, pos, dy, None)
    assert torch.equal(q.grad, want[0]) and layer.main_grad is None


def test_table_of_far_positions():
    tab = attention.rotary_table(100000, 32, theta=5e5, device=DEV)
    p = np.arange(99000, 100000)[:, None]
    a = p * 5e5 ** (-np.arange(16) / 16.0)
    # 64-bit angles: an error of 2^-52 of 1e5 radians and fp32's half step
    assert np.abs(C.as64(tab)[99000:] - np.concatenate([np.cos(a), np.sin(a)], 1)).max() <= U + 1e-9


def test_captured_step_beside_an_eager_graph():
    """A forward and backward step that is captured while an eager graph of the same
    weights lives, replayed several times with eager work between."""
    q, k, w, tab, pos, layer = layer_setup(9)
    eager = layer(q.clone().requires_grad_(), k.clone().requires_grad_(), pos)        # kept alive
    dy = [torch.randn_like(t.float()).to(torch.bfloat16) for t in (q, k)]
    x = [q.clone(), k.clone()]
    grads = [torch.zeros_like(t) for t in x]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()

    def step():
        leaves = [t.detach().requires_grad_() for t in x]
        torch.autograd.backward(layer(*leaves, pos), dy)
        for g, t in zip(grads, leaves):
            g.copy_(t.grad)

    with torch.cuda.stream(side):
        step()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    for n in range(3):
        x[0].copy_(C.rows(tuple(q.shape), n).to(DEV))
        x[1].copy_(C.rows(tuple(k.shape), n + 9).to(DEV))
        layer.main_grad.zero_()
        graph.replay()
        want = api.qk_norm_rope_backward(layer.norm, *x, pos, *dy)
        torch.cuda.synchronize()
        assert torch.equal(grads[0], want[0]) and torch.equal(grads[1], want[1])
        assert torch.equal(layer.main_grad, torch.stack(want[2:]))
    torch.autograd.backward(eager, dy)
    torch.cuda.synchronize()
