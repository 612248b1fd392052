"""GPU parity of the feed-forward activation with its 8-bit checkpoint, forward
and backward, against the formulas in 64 bits: the checkpoint to the bit, what
passes through the fp32 sigmoid within its derived error and half a step of
the output's format; gradients also against differences of the forward."""
import numpy as np
import pytest
import torch

from fp4_block_scaled_x16_amd import api
from fp8_check import DEV, as64, bf16, encodes, same_matrix
from oracle import fp8

pytestmark = pytest.mark.gpu
ACTS = ["swiglu", "relu2"]
SIZES = [(1, 8), (1, 1000), (17, 128), (127, 136), (128, 256), (130, 264), (300, 520), (3, 21504)]
U = 2.0 ** -24       # half a step of fp32, relative


def hidden(rows, cols, act, seed):
    """Gate values from the saturated ends through zero, and an outlier."""
    rng = np.random.default_rng(seed)
    v = rng.standard_normal((rows, cols * (2 if act == "swiglu" else 1))) * 3
    v *= np.exp2(np.arange(rows) % 9 - 6.0)[:, None]
    v[0, 0] = -120.0
    v[-1, cols // 2] = 150.0
    if rows > 2:
        v[1] = 0.0
    return bf16(v)


def gradient(rows, cols, seed):
    rng = np.random.default_rng(seed)
    return bf16(np.exp2(rng.uniform(-24, -6, (rows, cols))) * rng.choice([-1, 1], (rows, cols)))


def act_err(h, act):
    """Absolute error of fp32 a: sigmoid's exponential has |g| log2 e roundings of
    its argument (half a step each, times ln 2: |g| U) and an ulp of its own (2 U),
    the sum, the reciprocal (2 U) and the products one each: (|g| + 8) U; and the
    smallest normal number, below which the hardware exp2 and reciprocal
    may give zero, times the factors."""
    a = np.abs(fp8.act(h, act))
    if act == "relu2":
        return a * U
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    return a * (np.abs(g) + 8) * U + np.abs(g * u) * 2.0 ** -125


def grad_err(h, da, act):
    """The same for dh: every factor's relative error, with the terms of
    1 + g (1 - s) taken in absolute value (1 - s has U of absolute error)."""
    if act == "relu2":
        return np.abs(fp8.act_grad(h, da, act)) * 2 * U
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    s = fp8._sigmoid(g)
    e = (np.abs(g) + 8) * U
    inner = 1 + np.abs(g) * (1 - s)
    dg = np.abs(da * u) * (s * inner * (e + 6 * U) + s * np.abs(g) * (s * e + 2 * U) + (1 + np.abs(g)) * 2.0 ** -125)
    du = np.abs(da * g) * (s * (e + 4 * U) + 2.0 ** -125)
    return np.concatenate([dg, du], 1)


def near(t, v, err):
    """bf16 t: values within err of v, rounded once (half a step: 2^-9 of the
    binade's top, a subnormal's 2^-134)."""
    mag = np.maximum(np.abs(v) + err, 2.0 ** -126)
    half = np.exp2(np.floor(np.log2(mag)) - 8)
    bad = np.abs(as64(t) - v) > half + err
    assert not bad.any(), np.argwhere(bad)[:5].tolist()


def device(t, cols):
    """The matrix as the first columns of rows of a multiple of 8."""
    w = torch.zeros((t.shape[0], -(-t.shape[1] // 8) * 8), dtype=torch.bfloat16, device=DEV)
    w[:, :t.shape[1]] = t.to(DEV)
    return w[:, :t.shape[1]]


@pytest.mark.parametrize("rows,cols", SIZES + [(40, 1003), (1, 1)])
@pytest.mark.parametrize("act", ACTS)
def test_act_quantize(act, rows, cols):
    if act == "swiglu" and cols % 8:
        with pytest.raises(api.Fp4Error):
            api.act_quantize(torch.zeros((rows, 2 * cols + 2), dtype=torch.bfloat16, device=DEV)[:, :2 * cols], act)
        return
    h = hidden(rows, cols, act, rows + cols)
    hd, h64 = device(h, cols), as64(h)
    a, qh = api.act_quantize(hd, act)
    same_matrix(qh, *fp8.encode(fp8.checkpoint_layout(h64, cols), "fp8"))
    encodes(a, fp8.act(h64, act), act_err(h64, act), "fp8")
    av, none = api.act_quantize(hd, act, a="bf16", checkpoint=False)
    assert none is None
    near(av, fp8.act(h64, act), act_err(h64, act))
    none, qh2 = api.act_quantize(hd, act, a=None)
    assert none is None and torch.equal(qh.codes, qh2.codes)


@pytest.mark.parametrize("rows,cols", SIZES + [(40, 1003), (1, 1)])
@pytest.mark.parametrize("fmt", ["fp8", "fp8_e5m2"])
@pytest.mark.parametrize("act", ACTS)
def test_act_backward(act, fmt, rows, cols):
    if act == "swiglu" and cols % 8:
        pytest.skip("SwiGLU halves are multiples of 8")
    h = hidden(rows, cols, act, rows + cols + 1)
    da = gradient(rows, cols, rows)
    _, qh = api.act_quantize(device(h, cols), act, a=None)
    qh.scales[:, rows:] = 255                   # padding of unspecified value
    held = fp8.values(qh.codes.cpu().numpy(), qh.scales.cpu().numpy(), "fp8")
    first = -(-cols // 128) * 128
    hv = held[:, :cols] if act == "relu2" else np.concatenate([held[:, :cols], held[:, first:first + cols]], 1)
    d64 = as64(da)
    dh, err = fp8.act_grad(hv, d64, act), grad_err(hv, d64, act)
    a, aerr = fp8.act(hv, act), act_err(hv, act)
    dev_da = device(da, cols)
    qdh, qdht, qat = api.act_backward(qh, dev_da, act, fmt=fmt)
    lay = lambda v: fp8.checkpoint_layout(v, cols)     # noqa: E731
    encodes(qdh, lay(dh), lay(err), fmt)
    encodes(qdht, dh.T, err.T, fmt)
    encodes(qat, a.T, aerr.T, "fp8")
    dhv, av = api.act_backward(qh, dev_da, act, out="bf16")
    near(dhv, dh, err)
    near(av, a, aerr)


@pytest.mark.parametrize("act", ACTS)
def test_gradient_is_the_forwards_difference_quotient(act):
    """Differences of the forward's own values: the checkpoint's values with one
    half moved by a step d of its own grid each way, through act_quantize."""
    rows, cols = 16, 128
    rng = np.random.default_rng(2)
    halves = 2 if act == "swiglu" else 1
    # multiples of 1/4 in [-3.5, 3.5]: held exactly by the checkpoint (scale 2^-6)
    h = rng.integers(-14, 15, (rows, halves * cols)) / 4.0
    h[:, ::128] = 3.5
    _, qh = api.act_quantize(bf16(h).to(DEV), act, a=None)
    assert np.array_equal(fp8.values(qh.codes.cpu().numpy(), qh.scales.cpu().numpy(), "fp8"), h)
    ones = torch.ones((rows, cols), dtype=torch.bfloat16, device=DEV)
    dh, _ = api.act_backward(qh, ones, act, out="bf16")
    for half in range(halves):
        d = 2.0 ** -4
        e = np.zeros_like(h)
        e[:, half * cols:(half + 1) * cols] = d
        up, _ = api.act_quantize(bf16(h + e).to(DEV), act, a="bf16", checkpoint=False)
        down, _ = api.act_quantize(bf16(h - e).to(DEV), act, a="bf16", checkpoint=False)
        diff = (as64(up) - as64(down)) / (2 * d)
        got = as64(dh)[:, half * cols:(half + 1) * cols]
        # bf16 rounding of both values (2^-8 of up to 13 each) over 2 d, of the
        # gradient (2^-8 of up to 7), the third derivative's term
        # (d^2 / 6, |third| <= 1 * 3.5), and the kink of max(h, 0)^2 within d of 0
        size = np.maximum(np.abs(as64(up)), np.abs(as64(down)))
        tol = size * 2.0 ** -8 / d + np.abs(got) * 2.0 ** -8 + d * d + (d if act == "relu2" else 0)
        assert np.all(np.abs(diff - got) <= tol)


@pytest.mark.parametrize("act", ACTS)
def test_strided_input_and_neighbours(act):
    """h and da as columns of wider matrices; what lies beside them, non-finite
    here, changes nothing."""
    rows, cols = 70, 264
    w = cols * (2 if act == "swiglu" else 1)
    h, da = hidden(rows, cols, act, 5), gradient(rows, cols, 6)
    big_h = torch.full((rows + 1, w + 24), float("nan"), dtype=torch.bfloat16, device=DEV)
    big_d = torch.full((rows + 1, cols + 16), float("inf"), dtype=torch.bfloat16, device=DEV)
    big_h[:rows, 8:8 + w], big_d[:rows, 8:8 + cols] = h.to(DEV), da.to(DEV)
    a0, q0 = api.act_quantize(h.to(DEV), act)
    a1, q1 = api.act_quantize(big_h[:rows, 8:8 + w], act)
    assert torch.equal(a0.codes, a1.codes) and torch.equal(q0.codes, q1.codes)
    for x, y in zip(api.act_backward(q0, da.to(DEV), act), api.act_backward(q1, big_d[:rows, 8:8 + cols], act)):
        assert torch.equal(x.codes, y.codes) and torch.equal(x.scales[:, :x.rows], y.scales[:, :y.rows])


@pytest.mark.parametrize("act", ACTS)
def test_non_finite_stay_in_their_place(act):
    rows, cols = 40, 128
    h = hidden(rows, cols, act, 8)
    clean = h.clone()
    h[7, 9] = float("nan")
    clean[7, 9] = 0.0
    a, qh = api.act_quantize(h.to(DEV), act, a="bf16")
    b, _ = api.act_quantize(clean.to(DEV), act, a="bf16")
    assert bool(torch.isnan(a[7, 9]))
    a[7, 9] = b[7, 9]
    assert torch.equal(a, b)
    dh, av = api.act_backward(qh, gradient(rows, cols, 3).to(DEV), act, out="bf16")
    assert bool(torch.isnan(dh[7, 9])) and bool(torch.isnan(av[7, 9]))
    dh[7, 9] = 0
    if act == "swiglu":
        dh[7, cols + 9] = 0
    assert bool(torch.isfinite(dh).all())


@pytest.mark.parametrize("act", ACTS)
def test_empty_geometry_and_graph(act):
    w = 2 if act == "swiglu" else 1
    a, qh = api.act_quantize(torch.empty((0, 64 * w), dtype=torch.bfloat16, device=DEV), act)
    assert a.codes.shape == (0, 128)
    out = api.act_backward(qh, torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), act)
    assert out[2].codes.shape == (64, 0)
    rows, cols = 390, 400
    hs = [hidden(rows, cols, act, k).to(DEV) for k in range(3)]
    da = gradient(rows, cols, 1).to(DEV)

    def both(h):
        a, qh = api.act_quantize(h, act)
        return [a, qh, *api.act_backward(qh, da, act, fmt="fp8_e5m2")]

    def same(p, q):
        return all(torch.equal(x.codes, y.codes) and torch.equal(x.scales[:, :x.rows], y.scales[:, :y.rows])
                   for x, y in zip(p, q))

    want = [both(h) for h in hs]
    try:
        for wgs in (1, 5):
            api.selftest_set_geometry(wgs)
            assert same(both(hs[0]), want[0])
    finally:
        api.selftest_set_geometry()
    h = hs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = both(h)
    for k in (1, 2, 0, 1):
        h.copy_(hs[k])
        g.replay()
        both(hs[2])
        torch.cuda.synchronize()
        assert same(got, want[k])
