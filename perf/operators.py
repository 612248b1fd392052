"""The 8-bit block-128 operators, each in a plain form and as the library's call.

An FP8 matrix here is E4M3 or E5M2 codes with one power-of-two scale (a UE8M0 byte) per block of 128 along the
blocked axis: a code row is padded with zero codes to a multiple of 128 bytes, and the scales lie K-major,
[blocks, rows rounded up to 16].  2D blocks are 128 x 128, their scale repeated for each row.

  gemm       D = A B^T of two such matrices (B's weights in 1D or 2D blocks), bf16 or fp32, also into an old fp32 D
  quantize   bf16 -> codes and scales: along rows, along columns (of the transpose), both, or 2D with the transpose
  transpose  an 8-bit checkpoint of rows re-encoded along its columns: the weight gradient's operand
  act        SwiGLU or squared ReLU of bf16 h, encoded for the next product, with h's 8-bit checkpoint
  act_grad   their backward pass from that checkpoint: the gradient along rows and columns, the activation along columns

Sizes are those of the 1.2B, 12B and 8B feed-forward layers of this repository (2048 -> 6144, 4608 -> 12288,
4096 -> 21504) at 8192 tokens, and smaller and ragged ones.
"""
import math

import torch

own = False

E4M3, E5M2 = "fp8", "fp8_e5m2"
# name: (torch type, largest value = 1.75 * 2^top, smallest normal exponent, mantissa bits)
TYPES = {E4M3: (torch.float8_e4m3fn, 8, -6, 3), E5M2: (torch.float8_e5m2, 15, -14, 2)}
LARGEST = 2.0 * 8192 * 21504 * 4096          # floating point operations of the largest product
LARGEST_ELEMS = 8192 * 21504                 # elements of the largest elementwise case


def listed():
    return [
        # one token through the 1.2B layer's up projection: latency
        dict(name="gemm decode 1 token", op="gemm", m=1, n=6144, k=2048, fa=E4M3, w="2d", out="bf16"),
        # a batch of decoding requests through the 8B layer's down projection: the weights' bytes
        dict(name="gemm decode 32 tokens", op="gemm", m=32, n=4096, k=21504, fa=E4M3, w="2d", out="bf16"),
        # a ragged prompt through the 12B layer's down projection
        dict(name="gemm ragged prompt", op="gemm", m=1000, n=4608, k=12288, fa=E4M3, w="2d", out="bf16"),
        # the 8B layer's forward product at one sequence: the largest
        dict(name="gemm 8B forward", op="gemm", m=8192, n=21504, k=4096, fa=E4M3, w="2d", out="bf16"),
        # the 1.2B layer's weight gradient, E5M2 gradients, added to the fp32 main gradient
        dict(name="gemm 1.2B weight grad", op="gemm", m=6144, n=2048, k=8192, fa=E5M2, w="1d", out="acc"),
        # an 8B layer's input, along rows for the forward product and along columns for the weight gradient
        dict(name="quantize 8B input dual", op="quantize", rows=8192, cols=4096, fmt=E4M3, mode="dual"),
        # the 12B layer's weights in 2D blocks, with the transpose for the input gradient
        dict(name="quantize 12B weights 2d", op="quantize", rows=12288, cols=4608, fmt=E4M3, mode="2d"),
        # an 8B layer's input checkpoint, as the weight gradient reads it
        dict(name="transpose 8B checkpoint", op="transpose", rows=8192, cols=4096, fmt=E4M3),
        # the 1.2B layer's activation, gated, one sequence
        dict(name="act swiglu 1.2B", op="act", rows=8192, cols=6144, act="swiglu"),
        # a few tokens of the 8B layer, squared ReLU
        dict(name="act relu2 17 tokens", op="act", rows=17, cols=21504, act="relu2"),
        # the backward pass of both
        dict(name="act grad swiglu 1.2B", op="act_grad", rows=8192, cols=6144, act="swiglu", fmt=E5M2),
        dict(name="act grad relu2 ragged", op="act_grad", rows=1001, cols=4104, act="relu2", fmt=E4M3),
    ]


def draw(rng):
    def size(lo, hi, step=1):
        v = round(math.exp(rng.uniform(math.log(lo), math.log(hi))))
        return max(lo, v // step * step)

    op = rng.choice(["gemm", "gemm", "gemm", "quantize", "transpose", "act", "act_grad"])
    if op == "gemm":
        while True:
            m, n, k = size(1, 8192), size(128, 21504), size(64, 21504)
            if rng.random() < 0.5:        # a layer's own widths are multiples of 128
                n, k = max(128, n // 128 * 128), max(128, k // 128 * 128)
            if 2.0 * m * n * k <= LARGEST:
                break
        return dict(op=op, m=m, n=n, k=k, fa=rng.choice([E4M3, E4M3, E5M2]), w=rng.choice(["2d", "2d", "1d"]),
                    out=rng.choice(["bf16", "bf16", "fp32", "acc"]))
    if op in ("quantize", "transpose"):
        rows, cols = size(1, 8192), size(64, 21504)
        c = dict(op=op, rows=rows, cols=cols, fmt=rng.choice([E4M3, E4M3, E5M2]))
        return dict(c, mode=rng.choice(["row", "col", "dual", "2d"])) if op == "quantize" else c
    act = rng.choice(["swiglu", "relu2"])
    while True:
        rows, cols = size(1, 8192), size(64, 21504, 8)
        if rows * cols * (2 if act == "swiglu" else 1) <= LARGEST_ELEMS:
            break
    c = dict(op=op, rows=rows, cols=cols, act=act)
    return dict(c, fmt=rng.choice([E4M3, E5M2])) if op == "act_grad" else c


def up(v, to):
    return -(-v // to) * to


# ------------------------------------------------------------- inputs ----
def gen(seed, k):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 16 + k)


def activations(rows, cols, seed, k):
    """N(0, 1) with one entry in a thousand 50 times as large; rows 8 elements aligned."""
    x = torch.randn((rows, up(cols, 8)), generator=gen(seed, k), device="cuda")
    x = torch.where(torch.rand(x.shape, generator=gen(seed, k + 1), device="cuda") < 0.001, x * 50, x)
    return x.to(torch.bfloat16)[:, :cols]


def weights(rows, cols, seed, k):
    x = torch.randn((rows, up(cols, 8)), generator=gen(seed, k), device="cuda") * 0.02
    return x.to(torch.bfloat16)[:, :cols]


def gradients(rows, cols, seed, k):
    """+-10^U, U uniform in [-8, -2]: the spread of output gradients."""
    u = torch.rand((rows, up(cols, 8)), generator=gen(seed, k), device="cuda") * 6 - 8
    s = torch.rand(u.shape, generator=gen(seed, k + 1), device="cuda") < 0.5
    x = torch.exp(u * math.log(10.0))
    return torch.where(s, x, -x).to(torch.bfloat16)[:, :cols]


# ------------------------------------------------- plain encode/decode ---
def exponents(amax, fmt):
    """The smallest e with largest * 2^e >= amax, in [-127, 127]; -127 for a zero block."""
    m, k = torch.frexp(amax)                       # amax = m 2^k, m in [0.5, 1)
    e = (k - 1 - TYPES[fmt][1] + (m > 0.875)).clamp(-127, 127)
    return torch.where(amax > 0, e, torch.full_like(e, -127))


def pow2(e):
    """2^e in fp32 for whole e in [-127, 127]."""
    bits = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 0x00400000))
    return bits.to(torch.int32).view(torch.float32)


def codes_of(v, e, fmt):
    return (v * pow2(-e)).to(TYPES[fmt][0]).view(torch.uint8)


def encode(x, fmt, two_d=False):
    """(codes [R, up(C, 128)], scales [KB, up(R, 16)]) of fp32 x [R, C] in blocks along its rows."""
    R, C = x.shape
    v = torch.nn.functional.pad(x.float(), (0, up(C, 128) - C)).view(R, -1, 128)
    amax = v.abs().amax(2)                         # [R, KB]
    if two_d:
        a = torch.nn.functional.pad(amax, (0, 0, 0, up(R, 128) - R)).view(-1, 128, amax.shape[1]).amax(1)
        amax = a.repeat_interleave(128, 0)[:R]
    e = exponents(amax, fmt)
    codes = codes_of(v, e.unsqueeze(2), fmt).view(R, -1)
    scales = torch.nn.functional.pad((e + 127).to(torch.uint8).t(), (0, up(R, 16) - R)).contiguous()
    return codes, scales


def decode(codes, scales, fmt):
    """fp32 values [R, Kp] of codes [R, Kp]."""
    R, Kp = codes.shape
    s = pow2(scales[:, :R].t().to(torch.int32) - 127)
    return (codes.view(TYPES[fmt][0]).float().view(R, -1, 128) * s.unsqueeze(2)).view(R, Kp)


def values(codes, scales, rows, fmt):
    """Codes and scales as the numbers that they stand for."""
    return codes.view(TYPES[fmt][0]), scales[:, :rows].view(torch.float8_e8m0fnu)


def plain_act(g, u, act):
    if act == "swiglu":
        return g * torch.sigmoid(g) * u
    r = g.clamp(min=0)
    return r * r


def plain_act_grad(g, u, da, act):
    """(the gradients of the halves of h, the activation)"""
    if act == "swiglu":
        s = torch.sigmoid(g)
        silu = g * s
        return [da * u * s * (1 + g * (1 - s)), da * silu], silu * u
    r = g.clamp(min=0)
    return [da * 2 * r], r * r


# ------------------------------------------------------------ prepare ----
def prepare(case, seed):
    op, s = case["op"], dict(case)
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        x = gradients(m, k, seed, 0) if case["fa"] == E5M2 else activations(m, k, seed, 0)
        w = weights(n, k, seed, 2) if case["w"] == "2d" else activations(n, k, seed, 2)
        s["a"], s["sa"] = encode(x, case["fa"])
        s["b"], s["sb"] = encode(w, E4M3, case["w"] == "2d")
        if case["out"] == "acc":
            s["d"] = torch.randn((m, n), generator=gen(seed, 4), device="cuda")
    elif op == "quantize":
        make = weights if case["mode"] == "2d" else gradients if case["fmt"] == E5M2 else activations
        s["x"] = make(case["rows"], case["cols"], seed, 0)
    elif op == "transpose":
        make = gradients if case["fmt"] == E5M2 else activations
        s["q"], s["sq"] = encode(make(case["rows"], case["cols"], seed, 0), case["fmt"])
    else:
        halves = 2 if case["act"] == "swiglu" else 1
        s["h"] = activations(case["rows"], halves * case["cols"], seed, 0)
        if op == "act_grad":
            s["q"], s["sq"] = encode(gapped(s.pop("h").float(), case["cols"]), E4M3)
            s["da"] = gradients(case["rows"], case["cols"], seed, 2)
    return s


def gapped(h, cols):
    """The halves of h, each from a multiple of 128 columns on."""
    gap = up(cols, 128) - cols
    parts = [torch.nn.functional.pad(p, (0, gap)) for p in h.split(cols, 1)]
    return torch.cat(parts, 1)[:, :h.shape[1] + (len(parts) - 1) * gap]


# ---------------------------------------------------------------- run ----
def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    from fp4_block_scaled_x16_amd import api

    op = s["op"]
    if op == "gemm":
        m, n, k = s["m"], s["n"], s["k"]
        if "w_op" not in s:                       # the weights' operand, laid out once
            s["w_op"] = api.fp8_matrix(s["b"], s["sb"], n, k).operand()
        a = api.fp8_matrix(s["a"], s["sa"], m, k, s["fa"]).operand()
        if s["out"] == "acc":
            return api.gemm(a, s["w_op"], m, n, k, out=s["d"], accumulate=True)
        return api.gemm(a, s["w_op"], m, n, k, device=s["a"].device,
                        out_dtype=torch.float32 if s["out"] == "fp32" else torch.bfloat16)
    if op == "quantize":
        mode = s["mode"]
        if mode in ("dual", "2d"):
            q = api.quantize_dual(s["x"], s["fmt"], block="2d" if mode == "2d" else "1d")
        else:
            q = [api.quantize(s["x"], s["fmt"], orient=mode)]
        return [values(p.codes, p.scales, p.rows, s["fmt"]) for p in q]
    if op == "transpose":
        q = api.requantize_t(api.fp8_matrix(s["q"], s["sq"], s["rows"], s["cols"], s["fmt"]))
        return values(q.codes, q.scales, q.rows, s["fmt"])
    if op == "act":
        return [values(p.codes, p.scales, p.rows, E4M3) for p in api.act_quantize(s["h"], s["act"])]
    cols = s["cols"] + (up(s["cols"], 128) if s["act"] == "swiglu" else 0)
    qh = api.fp8_matrix(s["q"], s["sq"], s["rows"], cols)
    dh, dh_t, a_t = api.act_backward(qh, s["da"], s["act"], fmt=s["fmt"])
    return [values(p.codes, p.scales, p.rows, f) for p, f in ((dh, s["fmt"]), (dh_t, s["fmt"]), (a_t, E4M3))]


def run_plain(s):
    op = s["op"]
    if op == "gemm":
        d = decode(s["a"], s["sa"], s["fa"]) @ decode(s["b"], s["sb"], E4M3).t()
        if s["out"] == "acc":
            return s["d"].add_(d)
        return d if s["out"] == "fp32" else d.to(torch.bfloat16)
    if op == "quantize":
        mode, fmt, x = s["mode"], s["fmt"], s["x"]
        got = [encode(x, fmt, mode == "2d")] if mode != "col" else []
        got += [encode(x.t(), fmt, mode == "2d")] if mode != "row" else []
        rows = [x.shape[0]] * (mode != "col") + [x.shape[1]] * (mode != "row")
        return [values(c, e, r, fmt) for (c, e), r in zip(got, rows)]
    if op == "transpose":
        v = decode(s["q"], s["sq"], s["fmt"])[:, :s["cols"]]
        return values(*encode(v.t(), s["fmt"]), s["cols"], s["fmt"])
    rows, cols = s["rows"], s["cols"]
    if op == "act":
        h = s["h"].float()
        a = encode(plain_act(h[:, :cols], h[:, cols:], s["act"]), E4M3)
        return [values(c, e, rows, E4M3) for c, e in (a, encode(gapped(h, cols), E4M3))]
    h = decode(s["q"], s["sq"], E4M3)
    g, u = h[:, :cols], h[:, up(cols, 128):][:, :cols]
    parts, a = plain_act_grad(g, u, s["da"].float(), s["act"])
    dh = torch.cat(parts, 1)
    return [values(*encode(gapped(dh, cols), s["fmt"]), rows, s["fmt"]),
            values(*encode(dh.t(), s["fmt"]), dh.shape[1], s["fmt"]),
            values(*encode(a.t(), E4M3), cols, E4M3)]


# --------------------------------------------------------------- work ----
def matrix_bytes(rows, cols):
    """Codes and scales of an FP8 matrix."""
    return rows * cols + rows * -(-cols // 128)


def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        out = {"bf16": 2, "fp32": 4, "acc": 8}[case["out"]]
        return {"bytes": matrix_bytes(m, k) + matrix_bytes(n, k) + out * m * n, "flops": 2.0 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    along, across = matrix_bytes(rows, cols), matrix_bytes(cols, rows)
    if op == "quantize":
        mode = case["mode"]
        return {"bytes": 2 * rows * cols + (mode != "col") * along + (mode != "row") * across, "flops": 2.0 * rows * cols}
    if op == "transpose":
        return {"bytes": along + across, "flops": 2.0 * rows * cols}
    halves = 2 if case["act"] == "swiglu" else 1
    if op == "act":
        return {"bytes": 2 * halves * rows * cols + (halves + 1) * along, "flops": 10.0 * halves * rows * cols}
    return {"bytes": halves * along + 2 * rows * cols + halves * (along + across) + across, "flops": 20.0 * halves * rows * cols}


# -------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    """The outputs from the formats' definitions in 64 bits: a table of the 256 codes' values, rounding by
    arithmetic, scales as powers of two found by comparison."""
    op, s = case["op"], prepare(case, seed)
    if op == "gemm":
        if 2.0 * case["m"] * case["n"] * case["k"] > 2e14:
            return None                     # minutes of 64-bit products
        d = torch.matmul(wide(s["a"], s["sa"], case["fa"]), wide(s["b"], s["sb"], E4M3).t().contiguous())
        return d + s["d"].double() if case["out"] == "acc" else d
    if op == "quantize":
        x, fmt, two = s["x"].double(), case["fmt"], case["mode"] == "2d"
        return [narrow(t, fmt, two) for t, on in ((x, case["mode"] != "col"), (x.t(), case["mode"] != "row")) if on]
    if op == "transpose":
        return narrow(wide(s["q"], s["sq"], case["fmt"])[:, :case["cols"]].t(), case["fmt"])
    cols, fmt = case["cols"], case.get("fmt")
    first = up(cols, 128)
    if op == "act":
        h = s["h"].double()
        g = h[:, :cols]
        a = g / (1 + torch.exp(-g)) * h[:, cols:] if case["act"] == "swiglu" else torch.where(g > 0, g, 0.0) ** 2
        return [narrow(a, E4M3), narrow(gapped(h, cols), E4M3)]
    h, da = wide(s["q"], s["sq"], E4M3), s["da"].double()
    g = h[:, :cols]
    if case["act"] == "swiglu":
        u, t = h[:, first:first + cols], torch.exp(-g)
        a = g * u / (1 + t)
        dh = torch.cat([da * u * (1 + t + g * t) / (1 + t) ** 2, da * g / (1 + t)], 1)
    else:
        a, dh = torch.where(g > 0, g, 0.0) ** 2, torch.where(g > 0, 2 * g * da, 0.0)
    return [narrow(gapped(dh, cols), fmt), narrow(dh.t(), fmt), narrow(a.t(), E4M3)]


def table(fmt):
    """The value of each code, from its sign, exponent and mantissa bits."""
    _, _, low, bits = TYPES[fmt]
    c = torch.arange(256, device="cuda")
    man, field = (c & ((1 << bits) - 1)).double(), ((c & 127) >> bits)
    scale = torch.exp2((field.clamp(min=1) - 1 + low).double())
    v = torch.where(field > 0, 1 + man / (1 << bits), man / (1 << bits)) * scale
    return torch.where(c > 127, -v, v)


def wide(codes, scales, fmt):
    e = scales[:, :codes.shape[0]].t().double() - 127
    return table(fmt)[codes.long()] * torch.exp2(e).repeat_interleave(128, 1)


def narrow(v, fmt, two_d=False):
    """(values of the codes [R, up(C, 128)], values of the scales [KB, R]) in 64 bits."""
    _, top, low, bits = TYPES[fmt]
    R, C = v.shape
    v = torch.nn.functional.pad(v, (0, up(C, 128) - C)).reshape(R, -1, 128)
    amax = v.abs().amax(2)
    if two_d:
        rows = torch.arange(R, device=v.device) // 128
        best = torch.zeros((rows[-1] + 1, amax.shape[1]), dtype=v.dtype, device=v.device)
        amax = best.index_reduce(0, rows, amax, "amax")[rows]
    e = torch.floor(torch.log2(amax.clamp(min=1e-300))) - top - 1
    e = e + (1.75 * torch.exp2(e + top) < amax)
    e = (e + (1.75 * torch.exp2(e + top) < amax)).clamp(-127, 127)
    y = v * torch.exp2(-e).unsqueeze(2)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** low))).clamp(min=low) - bits)
    return (torch.round(y / step) * step).view(R, -1), torch.exp2(e).t().contiguous()
