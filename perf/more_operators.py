"""Performance cases of the dense FP4 operators of a decoder layer.

The products of a layer that are not routed (projections, a shared expert, the
logits) on matrices in block-scaled FP4, and what stands between them:

  quantize  fp4_quantize, fp4_dequantize   rows to FP4 and back to the values the codes stand for
  swiglu    fp4_swiglu                     SiLU(gate) * up
  linear    fp4_linear_rows                rows of 16 or 32 bits, quantised, times an FP4 weight matrix
  norm      fp4_block_norm                 norm behind a block, gate, residual scale and sum, norm before the next block
  ffn       all of them                    a shared expert between two residual sums, FP4 from each operator to the next

FP4 is e2m1 with an E4M3 scale per 16 elements and a power of two per row
(nvfp4), or with a power of two per 32 elements (mxfp4).

A case is a dict of plain values.  ``run`` computes it with elementary torch
operations in FP32, or, when ``own`` is set, with the library's calls.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BLOCK = {"nvfp4": 16, "mxfp4": 32}
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a token's hidden state before a projection: latency
        dict(name="quantize_token", op="quantize", type="bf16", format="nvfp4", rows=1, cols=2560, strided=False),
        # eight prompts, the attention's part of a packed projection
        dict(name="quantize_prompts", op="quantize", type="fp16", format="mxfp4", rows=19608, cols=4096, strided=True),
        # the shared expert of a decoded batch: latency
        dict(name="swiglu_batch", op="swiglu", type="bf16", rows=32, cols=2880, out="bf16", strided=True),
        # the shared expert of eight prompts, gate and up side by side in a row
        dict(name="swiglu_prompts", op="swiglu", type="bf16", rows=19608, cols=5760, out="bf16", strided=True),
        # one token through a projection: the weights' bytes
        dict(name="linear_token", op="linear", type="bf16", format="nvfp4", rows=1, cols=2560, outs=8192, bias=False,
             out="bf16"),
        # logits of a small batch over an odd vocabulary
        dict(name="linear_logits", op="linear", type="bf16", format="nvfp4", rows=7, cols=2560, outs=50257, bias=False,
             out="fp32"),
        # eight trees of 63 drafts, with a bias
        dict(name="linear_drafts", op="linear", type="fp16", format="mxfp4", rows=504, cols=4096, outs=5120, bias=True,
             out="fp16"),
        # many prompts at once through a wide layer: matrix work
        dict(name="linear_wide", op="linear", type="bf16", format="nvfp4", rows=16384, cols=8192, outs=8192, bias=False,
             out="bf16"),
        # between two blocks of a decoded token: latency
        dict(name="norm_token", op="norm", type="bf16", block="bf16", rows=1, cols=2560, post=True, gate="channel",
             out="bf16"),
        # behind the routed experts of eight prompts (their sums are in FP32), a gate for each element
        dict(name="norm_prompts", op="norm", type="bf16", block="fp32", rows=19608, cols=4096, post=True, gate="full",
             out="bf16"),
        # the shared expert of one decoded token: five launches' latency
        dict(name="ffn_token", op="ffn", type="bf16", format="nvfp4", rows=1, cols=2560, inter=640),
        # the shared expert of a prompt
        dict(name="ffn_prompt", op="ffn", type="bf16", format="mxfp4", rows=2451, cols=4096, inter=2880),
    ]


def _spread(rng, low, high):
    """An integer from low to high, even in its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    def one(op):
        c = dict(op=op, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), rows=_spread(rng, 1, 20000),
                 cols=32 * _spread(rng, 2, 512))
        if op in ("quantize", "linear", "ffn"):
            c["format"] = rng.choice(["nvfp4", "mxfp4"])
        if op in ("quantize", "swiglu"):
            c["strided"] = rng.random() < 0.5
        if op in ("swiglu", "norm"):
            c["out"] = rng.choice(["bf16", "fp16"])
        if op == "linear":
            c.update(outs=_spread(rng, 1, 50257), bias=rng.random() < 0.4, out=rng.choice(["bf16", "fp16", "fp32"]))
        elif op == "norm":
            c.update(block=rng.choice([c["type"], "bf16"]), post=rng.random() < 0.6,
                     gate=rng.choice(["none", "channel", "token", "full"]))
        elif op == "ffn":
            c["inter"] = 32 * _spread(rng, 2, 256)
        return c

    def size(c):
        return c["rows"] * c["cols"] * max(1, c.get("inter", 0) + c.get("outs", 0))

    def fits(c):
        top = [k for k in listed() if k["op"] == c["op"]]
        return (size(c) <= max(size(k) for k in top)
                and work(c)["bytes"] <= max(work(k)["bytes"] for k in top)
                and c["rows"] * c.get("outs", 0) <= 1 << 28)

    op = rng.choice(["quantize", "swiglu", "linear", "linear", "norm", "ffn"])
    c = one(op)
    while not fits(c):
        c = one(op)
    return c


def _width(kind):
    return 4 if kind == "fp32" else 2


def work(case):
    n, e = case["rows"] * case["cols"], _width(case["type"])
    # of an element in FP4 with its share of the scales
    held = 0.5 + 1 / BLOCK[case.get("format", "nvfp4")]
    if case["op"] == "quantize":  # the matrix, and once more as values of 16 bits
        return {"bytes": n * (e + held + 2), "flops": 0}
    if case["op"] == "swiglu":
        return {"bytes": n * (2 * e + 2), "flops": 0}
    if case["op"] == "linear":
        outs = case["outs"]
        return {"bytes": n * e + outs * case["cols"] * held + case["rows"] * outs * _width(case["out"]),
                "flops": 2 * n * outs}
    if case["op"] == "ffn":
        weights = 3 * case["cols"] * case["inter"]
        return {"bytes": n * (2 * e + 2 + 2) + weights * held, "flops": 2 * case["rows"] * weights}
    gate = {"none": 0, "channel": case["cols"], "token": case["rows"], "full": n}[case["gate"]]
    return {"bytes": n * (2 * e + _width(case["block"]) + 2) + gate * _width(case["block"]), "flops": 0}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols, dt = case["rows"], case["cols"], TYPES[case["type"]]

    def normal(*shape, type=torch.float32, mean=0.0, std=1.0):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=gen).to(type)

    def hidden(n, type):
        """Rows of different size with a few channels that stand out, as hidden states have them."""
        x = torch.empty(rows, n, device="cuda").normal_(generator=gen)
        x.mul_(normal(rows, 1).mul_(0.5).exp_())
        loud = torch.randperm(n, generator=gen, device="cuda")[:max(1, n // 256)]
        x[:, loud] *= 12
        return x.to(type)

    def weights(outs, n):
        w = torch.empty(outs, n, device="cuda").normal_(0.0, 0.02, generator=gen)
        return _packed(w.mul_(normal(outs, 1).mul_(0.3).exp_()), case["format"])

    s = {"case": case, "keep": {}}
    if case["op"] == "quantize":
        x = hidden(cols + (512 if case["strided"] else 0), dt)
        s["x"] = x[:, :cols]
    elif case["op"] == "swiglu":
        both = hidden(2 * cols, dt)
        s["gate"], s["up"] = both[:, :cols], both[:, cols:]
        if not case["strided"]:
            s["gate"], s["up"] = s["gate"].contiguous(), s["up"].contiguous()
    elif case["op"] == "linear":
        s["x"] = hidden(cols, dt)
        s["w"] = weights(case["outs"], cols)
        s["bias"] = normal(case["outs"]) if case["bias"] else None
    else:
        kind, block = case.get("gate", "none"), TYPES[case.get("block", "bf16")]
        s["r"], s["y"] = hidden(cols, dt).mul_(4), hidden(cols, block)
        shape = {"none": None, "channel": (cols,), "token": (rows, 1), "full": (rows, cols)}[kind]
        s["gate"] = None if shape is None else normal(*shape, type=block)
        s["post_weight"] = normal(cols, mean=1.0, std=0.1) if case.get("post") else None
        s["weight"], s["scale"] = normal(cols, mean=1.0, std=0.1), 0.75
        s["r_out"] = torch.zeros_like(s["r"])
        if case["op"] == "ffn":
            s["in"], s["out"] = weights(2 * case["inter"], cols), weights(cols, case["inter"])
            s["next_weight"] = normal(cols, mean=1.0, std=0.1)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    from block_scaled_fp4_softmax_gb300 import fp4

    c, keep = s["case"], s["keep"]
    kind = {"nvfp4": fp4.NVFP4, "mxfp4": fp4.MXFP4, None: None}[c.get("format")]
    if not keep:  # what a serving loop makes once: laid-out weights, workspaces, the matrices between the operators
        keep[""] = None
        if c["op"] == "quantize":
            keep["m"] = fp4.fp4_empty(c["rows"], c["cols"], kind)
        elif c["op"] == "linear":
            keep["w"] = fp4.fp4_matrix(*s["w"], format=kind)
            keep["ws"] = fp4.fp4_linear_rows_workspace(keep["w"], c["rows"])
        elif c["op"] == "ffn":
            keep["in"], keep["out"] = fp4.fp4_matrix(*s["in"], format=kind), fp4.fp4_matrix(*s["out"], format=kind)
            keep["h"], keep["a"] = (fp4.fp4_empty(c["rows"], n, kind) for n in (c["cols"], c["inter"]))
    if c["op"] == "quantize":
        return fp4.fp4_dequantize(fp4.fp4_quantize(s["x"], kind, out=keep["m"]))
    if c["op"] == "swiglu":
        return fp4.fp4_swiglu(s["gate"], s["up"], dtype=TYPES[c["out"]])[0]
    if c["op"] == "linear":
        return fp4.fp4_linear_rows(s["x"], keep["w"], bias=s["bias"], dtype=TYPES[c["out"]], workspace=keep["ws"])
    if c["op"] == "norm":
        r, h, _ = fp4.fp4_block_norm(s["r"], s["y"], post_weight=s["post_weight"], gate=s["gate"], scale=s["scale"],
                                     weight=s["weight"], eps=1e-6, dtype=TYPES[c["out"]], r_out=s["r_out"])
        return {"r": r, "h": h}
    i = c["inter"]
    r, _, h = fp4.fp4_block_norm(s["r"], s["y"], scale=s["scale"], weight=s["weight"], eps=1e-6, dtype=None,
                                 format=kind, r_out=s["r_out"], matrix=keep["h"])
    both = fp4.fp4_linear(h, keep["in"])
    _, a = fp4.fp4_swiglu(both[:, :i], both[:, i:], dtype=None, format=kind, matrix=keep["a"])
    y = fp4.fp4_linear(a, keep["out"])
    r, h, _ = fp4.fp4_block_norm(r, y, scale=s["scale"], weight=s["next_weight"], eps=1e-6, r_out=r)
    return {"r": r, "h": h}


def _plain(s):
    return {"quantize": _plain_quantize, "swiglu": _plain_swiglu, "linear": _plain_linear, "norm": _plain_norm,
            "ffn": _plain_ffn}[s["case"]["op"]](s)


def _power(e):
    """2^e of whole numbers from -126 to 127 in FP32."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _times(x, e):
    """x * 2^e for e from -127 to 127, in two steps: 2^-127 is no normal number."""
    half = torch.div(e, 2, rounding_mode="floor")
    return x * _power(half) * _power(e - half)


def _codes(q):
    """The nearest e2m1 magnitude's number, ties to the even one, of q in FP32."""
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=q.device)
    up = torch.tensor([False, True, False, True, False, True, False], device=q.device)
    ties = torch.where(up, torch.nextafter(ties, torch.zeros_like(ties)), ties)
    return torch.bucketize(q.abs(), ties, out_int32=True)


def _quantized(x, kind):
    """Codes' signs and numbers [rows, blocks, block], scales [rows, blocks, 1]
    as E4M3 values or exponents, and row exponents [rows, 1] or None."""
    x = x.float()
    if kind == "nvfp4":
        m, e = torch.frexp(x.abs().amax(-1, keepdim=True))  # 2688 = 448 * 6 = 0.65625 * 2^12
        row = (e - 12 + (m > 0.65625)).clamp(min=-126).masked_fill(m == 0, -126)
        x = (x * _power(-row)).unflatten(-1, (-1, 16))
        scale = (x.abs().amax(-1, keepdim=True) / 6).to(torch.float8_e4m3fn)
        real = scale.float()
        q = torch.where(real == 0, torch.zeros_like(x), x / real)
    else:
        x, row = x.unflatten(-1, (-1, 32)), None
        m, e = torch.frexp(x.abs().amax(-1, keepdim=True))  # 6 = 0.75 * 2^3
        scale = (e - 3 + (m > 0.75)).clamp(-127, 127).masked_fill(m == 0, -127)
        q = _times(x, -scale)
    return torch.signbit(q), _codes(q), scale, row


def _packed(x, kind):
    """A matrix's parts as a checkpoint holds them: codes, two to a byte and the
    even column in the low half, a byte of scale for each block, a factor for each row."""
    sign, code, scale, row = _quantized(x, kind)
    code = (code | sign.to(torch.int32) << 3).flatten(-2).to(torch.uint8)
    bits = scale.view(torch.uint8) if kind == "nvfp4" else (scale + 127).to(torch.uint8)
    return (code[:, ::2] | code[:, 1::2] << 4).contiguous(), bits.squeeze(-1).contiguous(), \
        None if row is None else _power(row).squeeze(-1).contiguous()


def _values(sign, code, scale, row, kind):
    v = torch.tensor(VALUES, device=code.device)[code]
    v = torch.where(sign, -v, v)
    v = v * scale.float() if kind == "nvfp4" else _times(v, scale)
    v = v.flatten(-2)
    return v if row is None else v * _power(row)


def _plain_quantize(s):
    kind = s["case"]["format"]
    return _values(*_quantized(s["x"], kind), kind).to(torch.bfloat16)


def _swiglu(gate, up):
    g = gate.float()
    return g / (1 + torch.exp(-g)) * up.float()


def _plain_swiglu(s):
    return _swiglu(s["gate"], s["up"]).to(TYPES[s["case"]["out"]])


def _product(x, parts, kind):
    """x [rows, cols], quantised, times the matrix of these parts."""
    codes, scales, row_scale = parts
    x = _values(*_quantized(x, kind), kind)
    byte = codes.to(torch.int32)
    code = torch.stack((byte & 15, byte >> 4), -1).flatten(-2).unflatten(-1, (-1, BLOCK[kind]))
    scale = scales.view(torch.float8_e4m3fn) if kind == "nvfp4" else scales.to(torch.int32) - 127
    w = _values((code & 8) != 0, code & 7, scale[..., None], None, kind)
    return x @ (w if row_scale is None else w * row_scale[:, None]).T


def _plain_linear(s):
    y = _product(s["x"], s["w"], s["case"]["format"])
    return (y if s["bias"] is None else y + s["bias"]).to(TYPES[s["case"]["out"]])


def _normed(x, weight):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight


def _residual(s, r, y):
    y = y.float()
    if s["post_weight"] is not None:
        y = _normed(y, s["post_weight"])
    if s["gate"] is not None:
        y = y * s["gate"].float()
    return r.float() + s["scale"] * y


def _plain_norm(s):
    r = _residual(s, s["r"], s["y"])
    s["r_out"].copy_(r)
    return {"r": s["r_out"], "h": _normed(r, s["weight"]).to(TYPES[s["case"]["out"]])}


def _plain_ffn(s):
    # what one operator hands to the next is of the type it has there: BF16, the residual's, or FP4
    kind = s["case"]["format"]
    r = _residual(s, s["r"], s["y"])
    both = _product(_normed(r, s["weight"]), s["in"], kind).to(torch.bfloat16)
    y = _product(_swiglu(*both.chunk(2, -1)), s["out"], kind).to(torch.bfloat16)
    r = _residual(s, r.to(s["r"].dtype), y)
    s["r_out"].copy_(r)
    return {"r": s["r_out"], "h": _normed(r, s["next_weight"]).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# The definitions in FP64
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    kind = case.get("format")

    def nearest(x, step):
        return torch.round(x / step) * step  # half way: to the even multiple

    def exponent(x):
        """floor(log2 x) of x > 0."""
        return torch.frexp(x)[1].double() - 1

    def fp4(x):
        """The values that the rows of x have in FP4."""
        size = x.abs()
        if kind == "nvfp4":
            top = size.amax(-1, keepdim=True)
            row = torch.ceil(torch.log2(top / 2688)).clamp(min=-126)
            row = torch.where(2688 * torch.exp2(row - 1) >= top, row - 1, row)  # log2 may be off at a border
            row = torch.exp2(torch.where(2688 * torch.exp2(row) < top, row + 1, row).clamp(min=-126))
            a = (size / row).unflatten(-1, (-1, 16))
            want = a.amax(-1, keepdim=True) / 6
            scale = nearest(want, torch.exp2(exponent(want.clamp(min=2.0 ** -6)) - 3))  # E4M3: 3 bits, subnormal below 2^-6
        else:
            row = 1.0
            a = size.unflatten(-1, (-1, 32))
            want = a.amax(-1, keepdim=True) / 6
            up = torch.exp2(exponent(want.clamp(min=2.0 ** -127)))
            scale = torch.where(want > up, 2 * up, up).clamp(max=2.0 ** 127)
        q = a / torch.where(scale == 0, 1.0, scale)
        q = nearest(q, torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0))).clamp(max=6)
        return torch.copysign((q * scale).flatten(-2) * row, x)

    value = torch.tensor(VALUES + tuple(-v for v in VALUES), dtype=torch.float64, device="cuda")

    def product(x, codes, scales, row_scale):
        even, odd = value[(codes & 15).int()], value[(codes >> 4).int()]
        b = scales.double()
        if kind == "nvfp4":
            e, m = torch.div(b, 8, rounding_mode="floor"), b % 8
            b = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2(e - 10))
        else:
            b = torch.exp2(b - 127)
        b = b if row_scale is None else b * row_scale.double()[:, None]
        x, b = fp4(x), b.repeat_interleave(BLOCK[kind] // 2, 1)
        return x[:, ::2] @ (even * b).T + x[:, 1::2] @ (odd * b).T

    def swiglu(g, u):
        g = g.double()
        return g * torch.sigmoid(g) * u.double()

    def norm(x, w):
        return x / ((x * x).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()

    def residual(r, y):
        y = y.double() if s["post_weight"] is None else norm(y.double(), s["post_weight"])
        return r.double() + s["scale"] * (y if s["gate"] is None else y * s["gate"].double())

    if case["op"] == "quantize":
        return fp4(s["x"].double())
    if case["op"] == "swiglu":
        return swiglu(s["gate"], s["up"])
    if case["op"] == "linear":
        y = product(s["x"].double(), *s["w"])
        return y if s["bias"] is None else y + s["bias"].double()
    r = residual(s["r"], s["y"])
    if case["op"] == "norm":
        return {"r": r, "h": norm(r, s["weight"])}
    both = product(norm(r, s["weight"]), *s["in"]).to(torch.bfloat16)
    y = product(swiglu(*both.chunk(2, -1)), *s["out"]).to(torch.bfloat16)
    r = residual(r.to(s["r"].dtype), y)
    return {"r": r, "h": norm(r, s["next_weight"])}
