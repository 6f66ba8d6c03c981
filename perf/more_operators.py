"""A decoder's 4-bit linear layers and its heads' rotation, each in its plain form and as the library runs it.

* linear: y = x W^T + bias with both operands in microscaled 4-bit floating point: the tokens are quantized in the
          call, the weights were quantized when the model was loaded;
* gated:  act(x G^T + bias_g) * (x U^T + bias_u), the first half of a gated feed-forward block, the same way;
* normed: h = x + residual, the root-mean-square norm of h with a gain, quantized, and the product that reads it;
* rotate: the root-mean-square norm of each query and key head and the rotation by its token's position.

The 4-bit formats: codes are E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte, the even element in
the low half.  "nvfp4": a scale S in E4M3 for each 16 elements of a row and a power of two s for each row, the smallest
with max|row| <= 6 * 448 * s; S = E4M3(max|block| / s / 6), code = E2M1(x / s / S).  "mxfp4": a power of two for each 32
elements, the smallest with max|block| <= 6 * scale (held as exponent + 127), code = E2M1(x / scale).  Both round to
nearest, ties to even.  Behind a norm, what is quantized is t = h * gain, and the row's scale takes the norm's factor.

`prepare` makes what a program has in hand before the call, `run` is one call, and `exact` is the same result from the
definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = {"nvfp4": 16, "mxfp4": 32}


# ------------------------------------------------------------------ cases
def _linear(name, tokens, width, out, fmt, bias):
    return {"name": name, "op": "linear", "tokens": tokens, "width": width, "out": out, "fmt": fmt, "bias": bias}


def _gated(name, tokens, width, out, fmt, bias, activation):
    return {"name": name, "op": "gated", "tokens": tokens, "width": width, "out": out, "fmt": fmt, "bias": bias,
            "activation": activation}


def _normed(name, tokens, width, out, fmt):
    return {"name": name, "op": "normed", "tokens": tokens, "width": width, "out": out, "fmt": fmt}


def _rotate(name, tokens, q_heads, kv_heads, head_dim, rotary, axes, interleaved, norm, far):
    return {"name": name, "op": "rotate", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "rotary": rotary, "axes": axes, "interleaved": interleaved, "norm": norm, "far": far}


def listed():
    return [
        # one request's decode step, a fused QKV projection: the weights' stream and launch latency
        _linear("linear_step_1x4096x6144_nvfp4", 1, 4096, 6144, "nvfp4", True),
        # a decode batch of an odd count, a projection back to the model's width
        _linear("linear_batch_61x5120x2080_mxfp4", 61, 5120, 2080, "mxfp4", True),
        # a chunk of a prompt; neither side a whole number of tiles
        _linear("linear_chunk_777x2592x4104_nvfp4", 777, 2592, 4104, "nvfp4", False),
        # a long prefill, the feed-forward's way down: products
        _linear("linear_prefill_8192x8192x4096_mxfp4", 8192, 8192, 4096, "mxfp4", False),
        # four requests decode through a gated feed-forward block
        _gated("gated_step_4x4096x11008_nvfp4", 4, 4096, 11008, "nvfp4", False, "silu"),
        # a mixed step of a smaller model, with biases
        _gated("gated_mixed_300x2048x5640_mxfp4", 300, 2048, 5640, "mxfp4", True, "gelu"),
        # a long prefill
        _gated("gated_prefill_4096x4096x12288_nvfp4", 4096, 4096, 12288, "nvfp4", False, "silu"),
        # a decode batch enters an attention block: residual, norm, QKV
        _normed("normed_batch_8x5120x7168_mxfp4", 8, 5120, 7168, "mxfp4"),
        # a prefill enters it
        _normed("normed_prefill_4095x4096x6144_nvfp4", 4095, 4096, 6144, "nvfp4"),
        # a decode step of 64 requests far into their contexts: launch latency
        _rotate("rotate_step_64x32x8x128", 64, 32, 8, 128, 128, 1, False, True, 131071),
        # a long prefill: bandwidth
        _rotate("rotate_prefill_16384x32x8x128", 16384, 32, 8, 128, 128, 1, False, True, 131071),
        # frames of patches with three axes, half of each head rotated, neighbours paired
        _rotate("rotate_patches_5001x24x24x96_3axes", 5001, 24, 24, 96, 48, 3, True, True, 700),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "gated", "gated", "normed", "normed", "rotate", "rotate"])
    if op == "rotate":
        head_dim = rng.choice([64, 80, 96, 128, 128, 256])
        rotary = rng.choice([head_dim, head_dim, head_dim // 32 * 16])
        kv_heads = rng.choice([1, 2, 4, 8, 24])
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 8])
        tokens = _log(rng, 1, min(16384, 16384 * 40 * 128 // ((q_heads + kv_heads) * head_dim)))
        case = _rotate("", tokens, q_heads, kv_heads, head_dim, rotary, rng.choice([1, 1, 2, 3]), rng.random() < 0.4,
                       rng.random() < 0.75, _log(rng, 100, 1 << 20))
    else:
        fmt = rng.choice(["nvfp4", "mxfp4"])
        width, out = 32 * _log(rng, 8, 256), 8 * _log(rng, 16, 1500)
        products = 4 if op == "gated" else 2
        tokens = _log(rng, 1, max(1, min(8192, 500_000_000_000 // (products * width * out))))
        if op == "linear":
            case = _linear("", tokens, width, out, fmt, rng.random() < 0.5)
        elif op == "gated":
            case = _gated("", tokens, width, out, fmt, rng.random() < 0.3, rng.choice(["silu", "gelu"]))
        else:
            case = _normed("", tokens, width, out, fmt)
    del case["name"]
    return case


# ------------------------------------------------------------------ work
def work(case):
    tokens = case["tokens"]
    if case["op"] == "rotate":
        n = tokens * (case["q_heads"] + case["kv_heads"]) * case["head_dim"]
        return {"bytes": 4 * n + 4 * tokens * case["axes"] + 2 * case["rotary"] + 4 * case["head_dim"], "flops": 8 * n}
    width, out = case["width"], case["out"]
    products = 2 if case["op"] == "gated" else 1
    weights = products * out * width
    size = weights // 2 + weights // BLOCK[case["fmt"]] + 4 * products * out  # codes, scales, rows' scales
    size += 2 * tokens * width + 2 * tokens * out
    if case["op"] == "normed":
        size += 4 * tokens * width + 2 * width  # the residual in and out, the gains
    elif case["bias"]:
        size += 2 * products * out
    return {"bytes": size, "flops": 2 * tokens * weights}


# ------------------------------------------------------------------ the formats, in 32 bits
def _e2m1(x):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with x's sign; ties to the even code; 6 from 5 on."""
    a = x.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((a / step).round() * step, x)


def _row_scale(most):
    """The smallest power of two with most <= 6 * 448 * 2^k, not below 2^-126; 0 for 0."""
    mantissa, exponent = torch.frexp(most)  # 6 * 448 = 0.65625 * 2^12
    k = (exponent - 12 + (mantissa > 0.65625).int()).clamp(min=-126)
    return torch.where(most > 0, torch.ldexp(torch.ones_like(most), k), 0.0)


def _quantize(x, fmt):
    """fp32 rows -> values of the codes times their blocks' scales [rows, width], those codes, the blocks' scales
    [rows, width / block], and the rows' scales [rows]."""
    blocks = x.unflatten(1, (-1, BLOCK[fmt]))
    if fmt == "nvfp4":
        row = _row_scale(x.abs().amax(1))
        inverse = torch.where(row > 0, 1 / row, 0.0)
        blocks = blocks * inverse[:, None, None]
        scale = (blocks.abs().amax(2) / 6).to(torch.float8_e4m3fn).float()
    else:
        row = torch.ones_like(x[:, 0])
        mantissa, exponent = torch.frexp(blocks.abs().amax(2))  # 6 = 0.75 * 2^3
        k = exponent - 3 + (mantissa > 0.75).int()
        scale = torch.ldexp(torch.ones_like(mantissa), torch.where(mantissa > 0, k.clamp(min=-127), -127))
    codes = _e2m1(torch.where(scale[:, :, None] > 0, blocks / scale[:, :, None], 0.0))
    return (codes * scale[:, :, None]).flatten(1), codes.flatten(1), scale, row


def _pack(codes, scale, row, fmt):
    """The library's layout: bytes of two codes; scales in tiles of 128 rows and 256 elements, in which those of four
    neighbouring blocks of a row lie together and rows r, r + 32, r + 64, r + 96 beside one another."""
    magnitude = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    nibble = torch.bucketize(codes.abs(), magnitude).to(torch.uint8) | (torch.signbit(codes).to(torch.uint8) << 3)
    packed = nibble[:, 0::2] | (nibble[:, 1::2] << 4)
    if fmt == "nvfp4":
        held = scale.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        held = (torch.frexp(scale)[1] + 126).to(torch.uint8)
    rows, groups = held.shape
    per = 256 // BLOCK[fmt]
    tiles, deep = -(-rows // 128), -(-groups // per)
    padded = torch.zeros(tiles * 128, deep * per, dtype=torch.uint8, device=codes.device)
    padded[:rows, :groups] = held
    tiled = padded.view(tiles, 4, 32, deep, per // 4, 4).permute(0, 3, 4, 2, 1, 5).reshape(tiles, deep, 128 * per)
    return {"codes": packed, "block_scales": tiled, "row_scales": row if fmt == "nvfp4" else None}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _hidden(g, tokens, width, loud):
    """Rows of a hidden state: a few channels are far louder than the others."""
    x = _randn(g, tokens, width)
    x[:, torch.randperm(width, generator=g, device="cuda")[: max(1, width // 100)]] *= loud
    return x.bfloat16()


def _weight(g, out, width, fmt):
    w = (_randn(g, out, width) * 0.02).bfloat16()
    values, codes, scale, row = _quantize(w.float(), fmt)
    return {"w": w, "values": values, "row": row, "packed": _pack(codes, scale, row, fmt)}


def prepare(case, seed):
    g = _generator(seed)
    tokens, op = case["tokens"], case["op"]
    if op == "rotate":
        heads, dim, half = case["q_heads"] + 2 * case["kv_heads"], case["head_dim"], case["rotary"] // 2
        qkv = (_randn(g, tokens, heads, dim) * 3).bfloat16()  # the fused projection's output: q and k are views
        q, k, _ = qkv.split((case["q_heads"], case["kv_heads"], case["kv_heads"]), dim=1)
        axes = case["axes"]
        positions = torch.randint(0, case["far"] + 1, (axes, tokens), generator=g, device="cuda", dtype=torch.int32)
        # each axis has its share of the pairs, and frequencies of its own from 1 down
        sections = [half // axes + (1 if a < half % axes else 0) for a in range(axes)]
        inv_freq = torch.cat([10000.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / n) for n in sections])
        weights = [(1 + 0.1 * _randn(g, dim)).bfloat16() if case["norm"] else None for _ in range(2)]
        return {"op": op, "q": q, "k": k, "positions": positions if axes > 1 else positions[0], "inv_freq": inv_freq.float(),
                "sections": sections, "interleaved": case["interleaved"], "q_weight": weights[0], "k_weight": weights[1],
                "eps": 1e-6}
    width, out, fmt = case["width"], case["out"], case["fmt"]
    s = {"op": op, "fmt": fmt, "x": _hidden(g, tokens, width, 20 if op != "normed" else 1)}
    if op == "gated":
        s["gate"], s["up"] = _weight(g, out, width, fmt), _weight(g, out, width, fmt)
        s["activation"] = case["activation"]
        for name in ("gate_bias", "up_bias"):
            s[name] = (0.1 * _randn(g, out)).bfloat16() if case["bias"] else None
        return s
    s["weight"] = _weight(g, out, width, fmt)
    if op == "normed":
        s["residual"] = _hidden(g, tokens, width, 20)
        s["gain"], s["eps"] = (1 + 0.1 * _randn(g, width)).bfloat16(), 1e-6
    else:
        s["bias"] = (0.1 * _randn(g, out)).bfloat16() if case["bias"] else None
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _RUN[state["op"]](state)
    return _PLAIN[state["op"]](state)


def _run_linear(s):
    import w8a8_int8_quantized_i8_gb300 as i8
    return i8.linear_fp4(s["x"], i8.FP4Rows(**s["weight"]["packed"]), s["bias"])


def _run_gated(s):
    import w8a8_int8_quantized_i8_gb300 as i8
    return i8.gated_linear_fp4(s["x"], i8.FP4Rows(**s["gate"]["packed"]), i8.FP4Rows(**s["up"]["packed"]),
                               s["gate_bias"], s["up_bias"], activation=s["activation"])


def _run_normed(s):
    import w8a8_int8_quantized_i8_gb300 as i8
    rows, h = i8.add_rmsnorm_quant_fp4(s["x"], s["residual"], s["gain"], eps=s["eps"], fmt=s["fmt"])
    return {"y": i8.gemm_fp4_bias_bf16(rows, i8.FP4Rows(**s["weight"]["packed"])), "h": h}


def _run_rotate(s):
    import w8a8_int8_quantized_i8_gb300 as i8
    q, k = i8.heads_rmsnorm_rotate(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"],
                                   eps=s["eps"], sections=s["sections"], interleaved=s["interleaved"])
    return {"q": q, "k": k}


# ------------------------------------------------------------------ plain forms
def _product(values, row, weight, bias):
    y = torch.matmul(values, weight["values"].T) * row[:, None] * weight["row"]
    return y if bias is None else y + bias.float()


def _plain_linear(s):
    values, _, _, row = _quantize(s["x"].float(), s["fmt"])
    return _product(values, row, s["weight"], s["bias"]).bfloat16()


def _activate(g, activation):
    if activation == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * torch.special.erfc(-g * math.sqrt(0.5))


def _plain_gated(s):
    values, _, _, row = _quantize(s["x"].float(), s["fmt"])
    g = _product(values, row, s["gate"], s["gate_bias"])
    return (_activate(g, s["activation"]) * _product(values, row, s["up"], s["up_bias"])).bfloat16()


def _plain_normed(s):
    h = s["x"].float() + s["residual"].float()
    values, _, _, row = _quantize(h * s["gain"].float(), s["fmt"])
    row = row / torch.sqrt((h * h).mean(1) + s["eps"])
    return {"y": _product(values, row, s["weight"], None).bfloat16(), "h": h.bfloat16()}


def _rotated(x, weight, cos, sin, s):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + s["eps"]) * weight.float()
    half = cos.shape[1]
    if s["interleaved"]:
        a, b = x[:, :, 0: 2 * half: 2], x[:, :, 1: 2 * half: 2]
    else:
        a, b = x[:, :, :half], x[:, :, half: 2 * half]
    c, d = cos[:, None], sin[:, None]
    pair = (a * c - b * d, b * c + a * d)
    front = torch.stack(pair, 3).flatten(2) if s["interleaved"] else torch.cat(pair, 2)
    return torch.cat((front, x[:, :, 2 * half:]), 2).bfloat16()


def _plain_rotate(s):
    where = s["positions"] if s["positions"].dim() == 2 else s["positions"][None]
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=sum(s["sections"]))
    angle = where[axis].T.double() * s["inv_freq"].double()  # far positions: 64 bits
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    return {"q": _rotated(s["q"], s["q_weight"], cos, sin, s), "k": _rotated(s["k"], s["k_weight"], cos, sin, s)}


_PLAIN = {"linear": _plain_linear, "gated": _plain_gated, "normed": _plain_normed, "rotate": _plain_rotate}
_RUN = {"linear": _run_linear, "gated": _run_gated, "normed": _run_normed, "rotate": _run_rotate}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "gated": _exact_gated, "normed": _exact_normed, "rotate": _exact_rotate}[case["op"]](s)


def _nearest(x, mantissa_bits, least, most):
    """The nearest value with so many bits behind the leading one, a least exponent and a most value; ties to even."""
    size = x.abs()
    exponent = torch.floor(torch.log2(size.clamp(min=2.0 ** (least - 8)))).clamp(min=least)
    step = torch.exp2(exponent - mantissa_bits)
    return torch.sign(x) * ((size / step).round() * step).clamp(max=most)


def _power_above(x):
    """The exponent of the smallest power of two that is at least x (log2 alone may be off in its last digit)."""
    k = torch.floor(torch.log2(x)) - 1
    for _ in range(3):
        k = torch.where(torch.exp2(k) < x, k + 1, k)
    return k


def _exact_values(t, fmt):
    """What rows in 64 bits stand for once they are held in the format."""
    size = t.abs()
    if fmt == "nvfp4":
        most = size.amax(1, keepdim=True)
        row = torch.where(most > 0, torch.exp2(_power_above(most / 2688).clamp(min=-126)), 1.0)
        top = (size / row).reshape(t.shape[0], -1, 16).amax(2).repeat_interleave(16, 1)
        scale = _nearest(top / 6, 3, -6, 448.0) * row
    else:
        top = size.reshape(t.shape[0], -1, 32).amax(2).repeat_interleave(32, 1)
        scale = torch.exp2(_power_above(top / 6).clamp(min=-127))
    full = torch.where(scale > 0, scale, 1.0)
    return torch.where(scale > 0, _nearest(t / full, 1, 0, 6.0) * scale, 0.0)


def _exact_product(t, weight, bias, fmt):
    y = t @ _exact_values(weight["w"].double(), fmt).T
    return y if bias is None else y + bias.double()


def _exact_linear(s):
    return _exact_product(_exact_values(s["x"].double(), s["fmt"]), s["weight"], s["bias"], s["fmt"])


def _exact_gated(s):
    t = _exact_values(s["x"].double(), s["fmt"])
    g = _exact_product(t, s["gate"], s["gate_bias"], s["fmt"])
    u = _exact_product(t, s["up"], s["up_bias"], s["fmt"])
    return u * (torch.nn.functional.silu(g) if s["activation"] == "silu" else torch.nn.functional.gelu(g))


def _exact_normed(s):
    h = s["x"].double() + s["residual"].double()
    t = _exact_values(h * s["gain"].double(), s["fmt"]) / (h.square().sum(1, keepdim=True) / h.shape[1] + s["eps"]).sqrt()
    return {"y": _exact_product(t, s["weight"], None, s["fmt"]), "h": h}


def _exact_rotate(s):
    where = s["positions"].reshape(-1, s["q"].shape[0]).double()
    turn = torch.cat([p[:, None] * f for p, f in zip(where, s["inv_freq"].double().split(s["sections"]))], 1)
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        if s[name + "_weight"] is not None:
            x = x / (x.square().sum(2, keepdim=True) / x.shape[2] + s["eps"]).sqrt() * s[name + "_weight"].double()
        n = turn.shape[1]
        first = torch.arange(n, device=x.device) * (2 if s["interleaved"] else 1)
        second = first + (1 if s["interleaved"] else n)
        z = torch.complex(x[:, :, first], x[:, :, second]) * torch.polar(torch.ones_like(turn), turn)[:, None]
        y = x.clone()
        y[:, :, first], y[:, :, second] = z.real, z.imag
        out[name] = y
    return out
