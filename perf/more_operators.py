"""Attention on a quantized key-value cache: each operator in a plain form and as the library's call.

The cache is paged: codes [pages, heads, page_size, bytes of a row], one byte per element (E4M3) or two E2M1 codes per
byte, element 2j in the low nibble; block scales [pages, heads, blocks of a row, page_size].  A block is 128 elements of
a row (fp8; a shorter row is one block), 32 (mxfp8, mxfp4) or 16 (nvfp4, ue5m3); the last two have a tensor scale from a
given amax each for K and V.  A slot is page * page_size + place in the page.

  norm       q and k: RMS norm of each head, times a weight, then rotation by the token's position (cos | sin rows of a table)
  norm_grad  its backward pass: the gradients of q and k and of both weights
  write      new tokens' K and V encoded into their slots; 8-bit formats: with norm and rotation of q and k in the same pass
             (q comes back); 4-bit formats: from K and V as they are, and read back as values
  read       slots back to values
  attend     attention of one new token per request over its pages, heads in groups that share a K and V head

Sizes: the model widths of this repository (2048, 4096) as heads of 64, 128 and 256, sequences of 8192 tokens as in its
feed-forward layers, and generic ones.
"""
import math

import torch

own = False
DEV = "cuda"

# name: (block, largest element, bytes per element x 2, tensor scale)
FORMATS = {"fp8": (128, 448.0, 2, False), "mxfp8": (32, 448.0, 2, False), "mxfp4": (32, 6.0, 1, False),
           "nvfp4": (16, 6.0, 1, True), "ue5m3": (16, 6.0, 1, True)}
SCALE_TOP = {"nvfp4": 448.0, "ue5m3": 122880.0}
TARGET = {"nvfp4": 448.0, "ue5m3": 2048.0}
EPS = 1e-6
LARGEST_TOKENS = 8192 * 40 * 128             # elements of the largest norm and write
LARGEST_CACHE = 4 * 120000 * 8 * 128         # elements of K in the largest attention
LARGEST_READ = 32768 * 8 * 128


def listed():
    return [
        # queries and keys of one training sequence of a layer 4096 wide, 8 key heads
        dict(name="norm 8192 tokens", op="norm", tokens=8192, hq=32, hk=8, d=128, rot=128, style="half"),
        # a ragged prompt, 2048 wide, every head its own key, half of each head rotated, neighbours paired
        dict(name="norm ragged prompt", op="norm", tokens=1001, hq=32, hk=32, d=64, rot=32, style="interleaved"),
        # their backward passes
        dict(name="norm grad 8192 tokens", op="norm_grad", tokens=8192, hq=32, hk=8, d=128, rot=128, style="half"),
        dict(name="norm grad ragged prompt", op="norm_grad", tokens=1001, hq=32, hk=32, d=64, rot=32, style="interleaved"),
        # one decoding step of 64 requests: a token each
        dict(name="write 64 requests", op="write", fmt="fp8", tokens=64, hq=32, hk=8, d=128, rot=128, style="half", page=16),
        # a prompt of 8192 tokens
        dict(name="write prompt", op="write", fmt="mxfp8", tokens=8192, hq=32, hk=8, d=128, rot=128, style="half", page=64),
        # a long prefix back to values, for a kernel that takes those
        dict(name="read 32768 tokens", op="read", fmt="nvfp4", tokens=32768, hk=8, d=128, page=64),
        # a short one, wide heads
        dict(name="read 1000 tokens", op="read", fmt="mxfp4", tokens=1000, hk=4, d=256, page=32),
        # one request early in its answer: latency
        dict(name="attend 1 request", op="attend", fmt="fp8", requests=1, longest=1000, ragged=False, hq=32, hk=8, d=128, page=16),
        # a serving batch of mixed lengths
        dict(name="attend 64 ragged requests", op="attend", fmt="mxfp8", requests=64, longest=8192, ragged=True, hq=32, hk=8,
             d=128, page=64),
        # few requests with long contexts: the largest
        dict(name="attend long contexts", op="attend", fmt="nvfp4", requests=4, longest=120000, ragged=False, hq=64, hk=8,
             d=128, page=128),
        # many short ones, 16 small query heads to a key head
        dict(name="attend 256 short requests", op="attend", fmt="mxfp4", requests=256, longest=1024, ragged=True, hq=64, hk=4,
             d=64, page=32),
    ]


def draw(rng):
    def size(lo, hi):
        return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    op = rng.choice(["norm", "norm_grad", "write", "read", "attend", "attend", "attend"])
    d = rng.choice([64, 128, 128, 256])
    hk = rng.choice([1, 2, 4, 8, 8, 16])
    hq = hk * rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 12, 16])
    c = dict(op=op, hk=hk, d=d)
    if op in ("norm", "norm_grad", "write"):
        hq = min(hq, 64 - hk)
        while True:
            t = size(1, 8192)
            if t * (hq + hk) * d <= LARGEST_TOKENS:
                break
        c.update(tokens=t, hq=hq, rot=rng.choice([d, d, d // 2]), style=rng.choice(["half", "half", "interleaved"]))
    if op == "read":
        while True:
            c["tokens"] = size(1, 32768)
            if c["tokens"] * hk * d <= LARGEST_READ:
                break
    if op in ("write", "read", "attend"):
        c.update(fmt=rng.choice(list(FORMATS)), page=rng.choice([16, 32, 64, 128]))
    if op == "attend":
        while True:
            n, longest = size(1, 256), size(1, 120000)
            if n * longest * hk * d <= LARGEST_CACHE:
                break
        c.update(hq=hq, requests=n, longest=longest, ragged=rng.random() < 0.6)
    return c


def lengths(case):
    """Tokens of each request: all alike, or spread over (0, longest] by the golden ratio's multiples, the first the longest."""
    n, longest = case["requests"], case["longest"]
    if not case["ragged"]:
        return [longest] * n
    return [max(1, math.ceil(longest * (1 - i * 0.6180339887498949 % 1))) for i in range(n)]


def row_bytes(fmt, d):
    """Codes and scales of a row of d."""
    block, _, halves, _ = FORMATS[fmt]
    return d * halves // 2 + -(-d // block)


# ------------------------------------------------------------- inputs ----
def gen(seed, k):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 16 + k)


def normal(shape, seed, k):
    return torch.randn(shape, generator=gen(seed, k), device=DEV)


def projected(shape, seed, k):
    """Rows as a projection gives them: normal, a few channels several times as large."""
    x = normal(shape, seed, k)
    far = torch.rand(shape[-2:], generator=gen(seed, k + 1), device=DEV) < 0.03
    return (x * torch.where(far, 6.0, 1.0)).to(torch.bfloat16)


def rotations(tokens, rot):
    """cos | sin of the angles of positions 0 .. tokens - 1, made in 64 bits."""
    f = torch.exp(torch.arange(rot // 2, device=DEV, dtype=torch.float64) * (-2.0 / rot * math.log(1e4)))
    a = torch.arange(tokens, device=DEV, dtype=torch.float64).unsqueeze(1) * f
    return torch.cat([torch.cos(a), torch.sin(a)], 1).float()


# ------------------------------------------------- plain encode/decode ---
def pow2(e):
    """2^e in fp32 for whole e in [-127, 127]."""
    bits = torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 0x00400000))
    return bits.to(torch.int32).view(torch.float32)


def tensor_scales(amax, fmt):
    """(encode, decode) of a tensor amax: fp32, every operation rounded by itself."""
    e = torch.where(amax > 0, amax.new_full((), 6.0) * TARGET[fmt] / amax, torch.ones_like(amax))
    return e, torch.ones_like(e) / e


def scale_codes(t, fmt):
    """fp32 t as the nearest code of a two-level format's scale, and its value."""
    t = t.clamp(max=SCALE_TOP[fmt])
    if fmt == "nvfp4":
        c = t.to(torch.float8_e4m3fn)
        return c.view(torch.uint8), c.float()
    k = torch.frexp(t)[1].clamp(min=-13) - 1                        # floor(log2 t), at least -14
    q = torch.round(t * pow2(3 - k))                                # steps of 2^(k - 3), up to 16
    return ((k + 14) * 8 + q).to(torch.uint8), q * pow2(k - 3)


def e2m1(y):
    """E2M1 codes (sign in bit 3) of fp32 y, to nearest, ties to even."""
    m = y.abs()
    c = (m > 0.25).to(torch.uint8)
    c += m >= 0.75
    c += m > 1.25
    c += m >= 1.75
    c += m > 2.5
    c += m >= 3.5
    c += m > 5.0
    return c | (torch.signbit(y).to(torch.uint8) << 3)


def encode(x, fmt, amax=None):
    """(codes, scales [.., blocks]) of fp32 rows x."""
    block, top, halves, two = FORMATS[fmt]
    d = x.shape[-1]
    v = x.unflatten(-1, (-1, min(block, d)))
    big = v.abs().amax(-1)
    if two:
        enc, dec = tensor_scales(amax, fmt)
        scales, s = scale_codes((big.double() / 6).float() * enc, fmt)
        inv = torch.where(scales > 0, torch.ones_like(s) / (s * dec), torch.zeros_like(s))
    else:
        m, k = torch.frexp(big)
        e = (k - (9 if top == 448.0 else 3) + (m > (0.875 if top == 448.0 else 0.75))).clamp(-127, 127)
        e = torch.where(big > 0, e, torch.full_like(e, -127))
        scales, inv = (e + 127).to(torch.uint8), pow2(-e)
    y = (v * inv.unsqueeze(-1)).flatten(-2)
    if halves == 2:
        return y.to(torch.float8_e4m3fn).view(torch.uint8), scales
    c = e2m1(y)
    return c[..., 0::2] | (c[..., 1::2] << 4), scales


def e2m1_values():
    v = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    return torch.cat([v, -v])


def decode(codes, scales, fmt, amax=None):
    """fp32 values of rows of codes with their scales [.., blocks]."""
    block, _, halves, two = FORMATS[fmt]
    if halves == 2:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        t = e2m1_values()
        v = torch.stack([t[(codes & 15).int()], t[(codes >> 4).int()]], -1).flatten(-2)
    if fmt == "nvfp4":
        s = scales.view(torch.float8_e4m3fn).float()
    elif fmt == "ue5m3":
        k, f = scales.int() >> 3, (scales & 7).float()
        s = torch.where(k > 0, (1 + f / 8) * pow2(k - 15), f * 2.0 ** -17)
    else:
        s = pow2(scales.int() - 127)
    v = v * s.repeat_interleave(v.shape[-1] // s.shape[-1], -1)
    return v * tensor_scales(amax, fmt)[1] if two else v


def pool(s, k, v, pages, fmt):
    """The cache's tensors, from the values of its pages [pages, heads, page_size, d]."""
    s["amax"] = torch.stack([k.abs().amax(), v.abs().amax()]) if FORMATS[fmt][3] else None
    for i, (name, x) in enumerate((("k", k), ("v", v))):
        codes, scales = encode(x, fmt, None if s["amax"] is None else s["amax"][i])
        s[name + "_codes"], s[name + "_scales"] = codes, scales.transpose(2, 3).contiguous()


def rows_of(s, name, slots):
    """The codes and scales of slots, as [slots, heads, ..]."""
    ps = s["page"]
    page, place = slots // ps, slots % ps
    return s[name + "_codes"][page, :, place], s[name + "_scales"][page, :, :, place]


# ------------------------------------------------------------ prepare ----
def prepare(case, seed):
    op, s = case["op"], dict(case)
    hk, d = case["hk"], case["d"]
    if op in ("norm", "norm_grad", "write"):
        t, hq = case["tokens"], case["hq"]
        qkv = projected((t, hq + 2 * hk, d), seed, 0)            # one projection's output: q, k and v beside each other
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["wq"], s["wk"] = ((1 + 0.2 * normal((d,), seed, 2 + i)).to(torch.bfloat16) for i in range(2))
        s["table"] = rotations(8192, case["rot"])
        s["positions"] = torch.arange(t, device=DEV)
        if op == "write" and t <= 256:                           # a decoding batch: requests at places of their own
            s["positions"] = torch.randint(0, 8192, (t,), generator=gen(seed, 4), device=DEV)
    if op == "norm_grad":
        s["dq"], s["dk"] = ((1e-3 * normal((t, h, d), seed, 5 + i)).to(torch.bfloat16) for i, h in enumerate((hq, hk)))
    if op in ("write", "read"):
        t, ps = case["tokens"], case["page"]
        pages = -(-t // ps) + 3
        x = normal((2, pages, hk, ps, d), seed, 8)
        pool(s, x[0], x[1], pages, case["fmt"])
        order = torch.randperm(pages, generator=gen(seed, 9), device=DEV)
        place = torch.arange(t, device=DEV)
        s["slots"] = order[place // ps] * ps + place % ps
    if op == "write" and s["amax"] is not None:
        s["amax"] = torch.stack([s[n].float().abs().amax() for n in "kv"])
    if op == "attend":
        n, ps = case["requests"], case["page"]
        s["lens"] = torch.tensor(lengths(case), dtype=torch.int32, device=DEV)
        width = -(-case["longest"] // ps)
        pages = sum(-(-length // ps) for length in lengths(case)) + 2
        k = normal((pages, hk, ps, d), seed, 8)
        k *= torch.where(torch.rand((hk, 1, d), generator=gen(seed, 7), device=DEV) < 0.03, 4.0, 1.0)
        pool(s, k, normal((pages, hk, ps, d), seed, 10), pages, case["fmt"])
        order = torch.randperm(pages, generator=gen(seed, 9), device=DEV).int()
        used = (s["lens"] + ps - 1) // ps
        at = (torch.cumsum(used, 0) - used).unsqueeze(1) + torch.arange(width, device=DEV)
        s["page_table"] = torch.where(torch.arange(width, device=DEV) < used.unsqueeze(1),
                                      order[at.clamp(max=pages - 1)], -1).int()
        s["q"] = (1.5 * normal((n, case["hq"], d), seed, 11)).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------- run ----
def run(s):
    return run_own(s) if own else run_plain(s)


def stored(s):
    """The cache's contents, as the numbers that 8-bit codes stand for."""
    scale = torch.float8_e8m0fnu
    return [(s[n + "_codes"].view(torch.float8_e4m3fn), s[n + "_scales"].view(scale)) for n in "kv"]


def run_own(s):
    from fp4_block_scaled_x16_amd import api

    op = s["op"]
    if "q" in s and "table" in s and "norm" not in s:             # weights and table: once
        s["norm"] = api.QKNorm(s["wq"], s["wk"], s["table"], eps=EPS, style=s["style"])
    if "k_codes" in s and "cache" not in s:
        s["cache"] = api.KVCache(s["fmt"], s["k_codes"], s["k_scales"], s["v_codes"], s["v_scales"], amax=s["amax"],
                                 target=TARGET.get(s["fmt"], 448.0))
    if op == "norm":
        return api.qk_norm_rope(s["norm"], s["q"], s["k"], s["positions"])
    if op == "norm_grad":
        return api.qk_norm_rope_backward(s["norm"], s["q"], s["k"], s["positions"], s["dq"], s["dk"])
    if op == "write":
        if FORMATS[s["fmt"]][2] == 2:
            q = api.kv_cache_write(s["cache"], s["k"], s["v"], s["slots"], q=s["q"], norm=s["norm"], positions=s["positions"])
            return q, stored(s)
        api.kv_cache_write(s["cache"], s["k"], s["v"], s["slots"])
        return api.kv_cache_read(s["cache"], s["slots"])
    if op == "read":
        return api.kv_cache_read(s["cache"], s["slots"])
    return api.attention_decode(s["q"], s["cache"], s["page_table"], s["lens"])


def rotate(z, cos, sin, style):
    """Rotated rows z [tokens, heads, d] (fp32 or wider); cos and sin [tokens, pairs]."""
    n = cos.shape[1]
    c, si = cos.unsqueeze(1), sin.unsqueeze(1)
    if style == "half":
        a, b, rest = z[..., :n], z[..., n:2 * n], z[..., 2 * n:]
        return torch.cat([a * c - b * si, b * c + a * si, rest], -1)
    a, b, rest = z[..., 0:2 * n:2], z[..., 1:2 * n:2], z[..., 2 * n:]
    return torch.cat([torch.stack([a * c - b * si, b * c + a * si], -1).flatten(-2), rest], -1)


def angles(s, dtype):
    t = s["table"][s["positions"]].to(dtype)
    return t.chunk(2, 1)


def plain_norm(x, w, s):
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return rotate(x * r * w.float(), *angles(s, torch.float32), s["style"])


def plain_norm_grad(x, w, dy, s):
    x, (cos, sin) = x.float(), angles(s, torch.float32)
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    dz = rotate(dy.float(), cos, -sin, s["style"])
    g = dz * w.float()
    dx = r * (g - x * r * r * (g * x).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (dz * x * r).sum((0, 1))


def run_plain(s):
    op = s["op"]
    if op == "norm":
        return [plain_norm(s[n], s["w" + n], s).to(torch.bfloat16) for n in "qk"]
    if op == "norm_grad":
        (dq, dwq), (dk, dwk) = (plain_norm_grad(s[n], s["w" + n], s["d" + n], s) for n in "qk")
        return dq, dk, dwq, dwk
    if op == "write":
        fmt, page, place = s["fmt"], s["slots"] // s["page"], s["slots"] % s["page"]
        eight = FORMATS[fmt][2] == 2
        amax = s["amax"] if s["amax"] is not None else [None, None]
        for i, (n, x) in enumerate((("k", plain_norm(s["k"], s["wk"], s) if eight else s["k"].float()), ("v", s["v"].float()))):
            codes, scales = encode(x, fmt, amax[i])
            s[n + "_codes"][page, :, place] = codes
            s[n + "_scales"][page, :, :, place] = scales
        if eight:
            return plain_norm(s["q"], s["wq"], s).to(torch.bfloat16), stored(s)
    if op in ("write", "read"):
        amax = s["amax"] if s["amax"] is not None else [None, None]
        return [decode(*rows_of(s, n, s["slots"]), s["fmt"], amax[i]).to(torch.bfloat16) for i, n in enumerate("kv")]
    n, hk, d = s["requests"], s["hk"], s["d"]
    k, v = (values_of(s, i) for i in range(2))                      # [requests, heads, places, d]
    q = s["q"].float().view(n, hk, -1, d)
    w = (q @ k.transpose(2, 3).contiguous()) / math.sqrt(d)
    off = torch.arange(w.shape[-1], device=DEV) >= s["lens"].view(n, 1, 1, 1)
    w = w.masked_fill(off, float("-inf"))
    p = torch.exp(w - w.amax(-1, keepdim=True))
    return ((p @ v) / p.sum(-1, keepdim=True)).view(n, -1, d).to(torch.bfloat16)


def values_of(s, i):
    """K (0) or V (1) of every place of the requests' pages, [requests, heads, places, d]; absent pages are page 0."""
    table = s["page_table"].clamp(min=0).long()
    codes = s["kv"[i] + "_codes"][table].transpose(1, 2).flatten(2, 3)
    scales = s["kv"[i] + "_scales"][table].transpose(3, 4).transpose(1, 2).flatten(2, 3)
    return decode(codes, scales, s["fmt"], None if s["amax"] is None else s["amax"][i])


# --------------------------------------------------------------- work ----
def work(case):
    op, hk, d = case["op"], case["hk"], case["d"]
    if op == "attend":
        total, hq = sum(lengths(case)), case["hq"]
        return {"bytes": 2 * total * hk * row_bytes(case["fmt"], d) + 4 * case["requests"] * hq * d, "flops": 4.0 * total * hq * d}
    t = case["tokens"]
    if op == "read":
        return {"bytes": 2 * t * hk * (row_bytes(case["fmt"], d) + 2 * d) + 8 * t, "flops": 2.0 * t * hk * d}
    heads, row = case["hq"] + hk, 8 + 4 * case["rot"]               # a token's position and angles
    if op == "norm":
        return {"bytes": t * (4 * heads * d + row), "flops": 10.0 * t * heads * d}
    if op == "norm_grad":
        return {"bytes": t * (6 * heads * d + row), "flops": 25.0 * t * heads * d}
    codes = 2 * hk * row_bytes(case["fmt"], d)
    if FORMATS[case["fmt"]][2] == 2:
        return {"bytes": t * (4 * case["hq"] * d + 4 * hk * d + codes + row + 8), "flops": 12.0 * t * heads * d}
    return {"bytes": t * (4 * hk * d + 2 * codes + 4 * hk * d + 16), "flops": 8.0 * t * hk * d}


# -------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    """The outputs in 64 bits: rotation as a product of complex numbers, codes through tables of their values."""
    op, s = case["op"], prepare(case, seed)
    if op == "norm":
        return [turn(unit(s[n])[0] * s["w" + n].double(), s, 1) for n in "qk"]
    if op == "norm_grad":
        dx, dw = zip(*(unit_grad(s[n], s["w" + n].double(), turn(s["d" + n].double(), s, -1)) for n in "qk"))
        return [*dx, *dw]
    if op in ("write", "read"):
        fmt, ps = case["fmt"], case["page"]
        eight = FORMATS[fmt][2] == 2
        if op == "read":
            return [wide(*rows_of(s, n, s["slots"]), s, i) for i, n in enumerate("kv")]
        k = turn(unit(s["k"])[0] * s["wk"].double(), s, 1) if eight else s["k"].double()
        got = [narrow(x, s, i) for i, x in enumerate((k, s["v"].double()))]
        if not eight:
            return [(v.unflatten(-1, (e.shape[-1], -1)) * e.unsqueeze(-1)).flatten(-2) for v, e in got]
        page, place = s["slots"] // ps, s["slots"] % ps
        pools = []
        for n, (v, e) in zip("kv", got):
            codes, scales = s[n + "_codes"].view(torch.float8_e4m3fn).double(), torch.exp2(s[n + "_scales"].double() - 127)
            codes[page, :, place], scales[page, :, :, place] = v, e
            pools.append((codes, scales))
        return turn(unit(s["q"])[0] * s["wq"].double(), s, 1), pools
    n, hk, d, ps = case["requests"], case["hk"], case["d"], case["page"]
    out = torch.zeros((n, case["hq"], d), dtype=torch.float64, device=DEV)
    for r, length in enumerate(lengths(case)):
        place = torch.arange(length, device=DEV)
        slots = s["page_table"][r][place // ps].long() * ps + place % ps
        k, v = (wide(*rows_of(s, name, slots), s, i).transpose(0, 1).contiguous() for i, name in enumerate("kv"))
        w = torch.matmul(k, s["q"][r].double().view(hk, -1, d).transpose(1, 2).contiguous()) * d ** -0.5
        w = torch.softmax(w, 1).transpose(1, 2).contiguous()
        out[r] = torch.matmul(w, v).reshape(-1, d)
    return out


def unit(x):
    """(x over its root mean square, that)"""
    x = x.double()
    r = torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS)
    return x / r, r


def unit_grad(x, w, dz):
    u, r = unit(x)
    g = dz * w
    return (g - u * (g * u).sum(-1, keepdim=True) / x.shape[-1]) / r, (dz * u).sum((0, 1))


def turn(z, s, sign):
    """Rows with their pairs multiplied by cos + sign i sin."""
    t = s["table"].double()[s["positions"]]
    n = t.shape[1] // 2
    by = torch.complex(t[:, :n], sign * t[:, n:]).unsqueeze(1)
    head, rest = z[..., :2 * n], z[..., 2 * n:]
    pairs = head.unflatten(-1, (2, n)).transpose(-1, -2) if s["style"] == "half" else head.unflatten(-1, (n, 2))
    got = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * by)
    got = got.transpose(-1, -2) if s["style"] == "half" else got
    return torch.cat([got.flatten(-2), rest], -1)


def steps(y, low, bits):
    """y to nearest on a grid of `bits` mantissa bits, subnormal below 2^low."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** low))).clamp(min=low) - bits)
    return torch.round(y / step) * step


def held(x):
    """64-bit x where the format's definition has an fp32 number."""
    return x.float().double()


def both_scales(s, i):
    """The tensor's encode and decode scale."""
    e = held(6 * TARGET[s["fmt"]] / s["amax"][i].double())
    return e, held(1 / e)


def narrow(x, s, i):
    """(values of the codes, scales) of rows x, in 64 bits; the two-level formats name an fp32 number at each of their
    steps, which decides ties of inputs that are short fractions themselves."""
    fmt = s["fmt"]
    block, top, halves, two = FORMATS[fmt]
    v = x.unflatten(-1, (-1, min(block, x.shape[-1])))
    big = v.abs().amax(-1)
    if two:
        enc, dec = both_scales(s, i)
        e = steps(held(held(big / 6) * enc).clamp(max=SCALE_TOP[fmt]), -6 if fmt == "nvfp4" else -14, 3)
        by = e * dec
        y = held(v * torch.where(e > 0, held(1 / held(by)), torch.zeros_like(e)).unsqueeze(-1)).clamp(-top, top)
    else:
        by = torch.exp2(torch.ceil(torch.log2((big / top).clamp(min=2.0 ** -127))).clamp(-127, 127))
        y = v / by.unsqueeze(-1)
    y = steps(y, -6, 3) if halves == 2 else steps(y, 0, 1)
    return y.flatten(-2), by


def wide(codes, scales, s, i):
    """Values of rows of codes in 64 bits, from a table of what each code stands for."""
    fmt = s["fmt"]
    c = torch.arange(256, device=DEV)
    eight = torch.where((c & 127) > 7, (8 + (c & 7)).double() * torch.exp2(((c & 127) >> 3).double() - 10), (c & 7).double() / 512)
    if FORMATS[fmt][2] == 2:
        v = torch.where(c > 127, -eight, eight)[codes.long()]
    else:
        m = c & 7
        four = torch.where(m > 1, (2 + (m & 1)).double() * torch.exp2((m >> 1).double() - 2), m.double() / 2)
        four = torch.where((c & 8) > 0, -four, four)
        v = torch.stack([four[(codes & 15).long()], four[(codes >> 4).long()]], -1).flatten(-2)
    if fmt == "nvfp4":
        e = eight[scales.long()]
    elif fmt == "ue5m3":
        e = torch.where(c > 7, (8 + (c & 7)).double() * torch.exp2((c >> 3).double() - 18), c.double() * 2.0 ** -17)[scales.long()]
    else:
        e = torch.exp2(scales.double() - 127)
    v = v * e.repeat_interleave(v.shape[-1] // e.shape[-1], -1)
    return v * both_scales(s, i)[1] if FORMATS[fmt][3] else v
