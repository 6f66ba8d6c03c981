"""The serving operators beside the W8A8 linear layer, each in its plain form and as the library runs it.

Four operators that a decoder built on 8-bit linear layers calls at every step:

* norm:   h = x + residual, the root-mean-square norm of h with a gain, and the norm's output in 8 bits with one
          scale a token (what the next linear layer reads);
* tables: the step's block tables, slot map, positions and offsets from the requests' lengths;
* append: the step's new keys and values into a paged cache held in 8 bits, one scale for each block and head;
* attend: causal attention of the new tokens over that cache.

`prepare` makes what a program has in hand before the call, `run` is one call, and `exact` is the same result from
the definition in 64 bits.  Lengths come from the case alone (`lens_seed`), values from the seed.
"""
import math
import random

import torch

own = False

INT8_MAX, E4M3_MAX = 127.0, 448.0


# ------------------------------------------------------------------ cases
def _norm(name, tokens, width, fmt):
    return {"name": name, "op": "norm", "tokens": tokens, "width": width, "fmt": fmt}


def _tables(name, requests, context, new, share, block, lens_seed):
    return {"name": name, "op": "tables", "requests": requests, "context": context, "new": new, "share": share,
            "block": block, "lens_seed": lens_seed}


def _append(name, requests, context, new, block, q_heads, kv_heads, head_dim, fmt, lens_seed):
    return {"name": name, "op": "append", "requests": requests, "context": context, "new": new, "block": block,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "fmt": fmt, "lens_seed": lens_seed}


def _attend(name, requests, context, new, block, q_heads, kv_heads, head_dim, fmt, lens_seed):
    return {"name": name, "op": "attend", "requests": requests, "context": context, "new": new, "block": block,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "fmt": fmt, "lens_seed": lens_seed}


def listed():
    return [
        # one request's decode step at the library's DiT width: launch latency
        _norm("norm_step_1x3072_int8", 1, 3072, "int8"),
        # a decode batch with an odd count of tokens
        _norm("norm_batch_333x4096_int8", 333, 4096, "int8"),
        # a long prefill: bandwidth
        _norm("norm_prefill_16384x3072_e4m3", 16384, 3072, "e4m3"),
        # a decode step: one new token a request
        _tables("tables_decode_64", 64, 4000, 1, 0.0, 16, 11),
        # a full scheduler step: most requests decode, some bring chunks of a prompt
        _tables("tables_mixed_2048", 2048, 8192, 777, 0.12, 64, 12),
        # a decode step's keys and values
        _append("append_decode_128_e4m3", 128, 30, 1, 16, 32, 8, 128, "e4m3", 21),
        # prompts' keys and values, some into blocks that are begun
        _append("append_prefill_5_int8", 5, 200, 2047, 64, 24, 8, 128, "int8", 22),
        # one request's decode step
        _attend("attend_step_1x777_int8", 1, 777, 1, 16, 24, 8, 128, "int8", 31),
        # a decode batch of ragged contexts
        _attend("attend_decode_64x8k_int8", 64, 8192, 1, 16, 32, 8, 128, "int8", 32),
        # one long context
        _attend("attend_long_1x131071_e4m3", 1, 131071, 1, 64, 64, 8, 128, "e4m3", 33),
        # drafted tokens are checked, every head with keys of its own
        _attend("attend_verify_16x2k_e4m3", 16, 2000, 5, 32, 24, 24, 64, "e4m3", 34),
        # chunks of prompts against their contexts: products
        _attend("attend_chunks_4x8k_int8", 4, 8000, 2048, 64, 32, 8, 128, "int8", 35),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "tables", "append", "append", "attend", "attend", "attend"])
    fmt = rng.choice(["int8", "e4m3"])
    seed = rng.randrange(1 << 30)
    if op == "norm":
        width = 16 * _log(rng, 16, 1024)
        tokens = _log(rng, 1, max(1, min(16384, 16384 * 3072 // width)))
        return {k: v for k, v in _norm("", tokens, width, fmt).items() if k != "name"}
    if op == "tables":
        c = _tables("", _log(rng, 1, 2048), _log(rng, 1, 8192), _log(rng, 1, 777), rng.choice([0.0, 0.05, 0.12]),
                    rng.choice([16, 32, 64, 128]), seed)
        return {k: v for k, v in c.items() if k != "name"}
    head_dim = rng.choice([64, 128, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 16])
    block = rng.choice([16, 32, 64, 128])
    if op == "append":
        new = _log(rng, 1, 2047)
        requests = _log(rng, 1, max(1, min(256, 5 * 2047 * 1024 // (new * kv_heads * head_dim))))
        c = _append("", requests, rng.randrange(0, 300), new, block, kv_heads * group, kv_heads, head_dim, fmt, seed)
        return {k: v for k, v in c.items() if k != "name"}
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    if kind == "decode":
        new = 1
        context = _log(rng, 1, 65536)
    elif kind == "verify":
        new = rng.randrange(2, 9)
        context = _log(rng, new, 16384)
    else:
        new = _log(rng, 9, 1024)
        context = _log(rng, new, 8000)
    # no more than the listed cases' bytes (contexts) and products (scores)
    most = min(64, 64 * 8192 * 1024 // (context * kv_heads * head_dim),
               4 * 2048 * 8000 * 32 * 128 // (new * context * kv_heads * group * head_dim))
    c = _attend("", _log(rng, 1, max(1, most)), context, new, block, kv_heads * group, kv_heads, head_dim, fmt, seed)
    return {k: v for k, v in c.items() if k != "name"}


def _lengths(case):
    """(tokens before the step, new tokens) of each request: ragged, the first one the longest."""
    rng = random.Random(case["lens_seed"])
    before, new = [], []
    for i in range(case["requests"]):
        if case["op"] == "tables":
            before.append(0 if rng.random() < 0.05 else rng.randrange(case["context"] + 1))
            new.append(rng.randrange(case["new"] + 1) if rng.random() < case["share"] else 1)
        elif case["op"] == "append":
            before.append(rng.randrange(case["context"] + 1))
            new.append(case["new"] if i == 0 else rng.randrange(1, case["new"] + 1))
        else:  # the context counts the new tokens
            whole = case["context"] if i == 0 else rng.randrange(1, case["context"] + 1)
            n = min(whole, case["new"] if i == 0 or case["new"] <= 8 else rng.randrange(1, case["new"] + 1))
            before.append(whole - n)
            new.append(n)
    return before, new


def _blocks(tokens, block):
    return -(-tokens // block)


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "norm":
        n = case["tokens"] * case["width"]
        # x and residual read, h and codes written; int8 codes come back as bf16 values
        return {"bytes": n * (2 + 2 + 2 + (1 if case["fmt"] == "e4m3" else 2)) + 2 * case["width"] + 4 * case["tokens"],
                "flops": 8 * n}
    before, new = _lengths(case)
    block, requests = case["block"], case["requests"]
    if case["op"] == "tables":
        tokens = sum(new)
        fresh = sum(_blocks(b + n, block) - _blocks(b, block) for b, n in zip(before, new))
        # lengths read, offsets and lengths written; a slot (8 bytes) and a position a token; new blocks read and written
        return {"bytes": 16 * requests + 12 * tokens + 8 * fresh, "flops": 8 * tokens + 8 * requests}
    heads, dim = case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        n = 2 * sum(new) * heads * dim
        touched = sum(_blocks(b + n_, block) - b // block for b, n_ in zip(before, new))
        return {"bytes": n * (2 + (1 if case["fmt"] == "e4m3" else 2)) + 8 * sum(new) + 16 * touched * heads, "flops": 4 * n}
    pairs = sum(n * b + n * (n + 1) // 2 for b, n in zip(before, new))
    cached = sum(b + n for b, n in zip(before, new))
    read = 2 * cached * heads * dim + sum(8 * heads + 4 for b, n in zip(before, new) for _ in range(_blocks(b + n, block)))
    return {"bytes": read + 4 * sum(new) * case["q_heads"] * dim, "flops": 4 * dim * case["q_heads"] * pairs}


# ------------------------------------------------------------------ inputs
def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _limit(fmt):
    return INT8_MAX if fmt == "int8" else E4M3_MAX


def _to_codes(x, fmt):
    """Codes of values that are already divided by their scale."""
    if fmt == "int8":
        return x.round().clamp(-INT8_MAX, INT8_MAX).to(torch.int8)
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float32).to(torch.float8_e4m3fn)


def _filled(g, blocks, heads, block, dim, fmt, spread):
    """A pool of blocks as earlier steps left it: codes [blocks, heads, block, dim] and scales [blocks, heads]."""
    x = _randn(g, blocks, heads, block, dim) * spread
    scale = x.abs().amax(dim=(2, 3)) / _limit(fmt)
    return _to_codes(x / scale[:, :, None, None], fmt), scale


def _tables_of(g, before, new, block, spare=0):
    """Block tables over a shuffled pool for requests of these lengths, and the pool's size."""
    need = [_blocks(b + n, block) for b, n in zip(before, new)]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(need), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at, rows, cols = 0, [], []
    for r, n in enumerate(need):
        rows += [r] * n
        cols += range(n)
    table[_ints(rows, torch.int64), _ints(cols, torch.int64)] = order[: len(rows)]
    return table, pool


def prepare(case, seed):
    g = _generator(seed)
    if case["op"] == "norm":
        tokens, width = case["tokens"], case["width"]
        x = _randn(g, tokens, width)
        residual = _randn(g, tokens, width) * 4
        residual[:, torch.randperm(width, generator=g, device="cuda")[: max(1, width // 100)]] *= 20  # outlier channels
        weight = 1 + 0.1 * _randn(g, width)
        return {"op": "norm", "fmt": case["fmt"], "x": x.bfloat16(), "residual": residual.bfloat16(),
                "weight": weight.bfloat16(), "eps": 1e-6}
    before, new = _lengths(case)
    block, requests = case["block"], case["requests"]
    if case["op"] == "tables":
        held = [_blocks(b, block) for b in before]
        need = [_blocks(b + n, block) for b, n in zip(before, new)]
        width = max(1, max(need)) + 3
        pool = sum(need) + 17
        order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
        table = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
        rows = [r for r, n in enumerate(held) for _ in range(n)]
        cols = [c for n in held for c in range(n)]
        table[_ints(rows, torch.int64), _ints(cols, torch.int64)] = order[: len(rows)]
        tokens = sum(new) + 5  # the buffers are a little larger than the step
        out = {"cu_new": _ints([0] * (requests + 1)), "seq_lens": _ints([0] * requests),
               "slots": torch.zeros(tokens, dtype=torch.int64, device="cuda"),
               "positions": torch.zeros(tokens, dtype=torch.int32, device="cuda"), "counts": _ints([0, 0, 0])}
        return {"op": "tables", "context_lens": _ints(before), "new_lens": _ints(new), "block_tables": table,
                "free_blocks": order[len(rows):].contiguous(), "taken": _ints([3]), "block": block, "tokens": tokens,
                "out": out}
    heads, q_heads, dim, fmt = case["kv_heads"], case["q_heads"], case["head_dim"], case["fmt"]
    table, pool = _tables_of(g, before, new, block)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    if case["op"] == "append":
        # the cache as the earlier steps left it, quieter than some of the new tokens: blocks that are begun get new scales
        k, k_scale = _filled(g, pool, heads, block, dim, fmt, 0.8)
        v, v_scale = _filled(g, pool, heads, block, dim, fmt, 0.8)
        qkv = _randn(g, cu[-1], (q_heads + 2 * heads) * dim).bfloat16()  # the fused projection's output: k and v are views
        keys = qkv[:, q_heads * dim: (q_heads + heads) * dim].unflatten(1, (heads, dim))
        values = qkv[:, (q_heads + heads) * dim:].unflatten(1, (heads, dim))
        request = torch.repeat_interleave(torch.arange(requests, device="cuda"), _ints(new, torch.int64), output_size=cu[-1])
        position = torch.arange(cu[-1], device="cuda") - _ints(cu, torch.int64)[request] + _ints(before, torch.int64)[request]
        slots = table[request, position // block].long() * block + position % block
        return {"op": "append", "fmt": fmt, "keys": keys, "values": values, "slots": slots, "k": k, "v": v,
                "k_scale": k_scale, "v_scale": v_scale}
    k, k_scale = _filled(g, pool, heads, block, dim, fmt, 1.0)
    v, v_scale = _filled(g, pool, heads, block, dim, fmt, 1.0)
    q = (_randn(g, cu[-1], q_heads, dim) * 2).bfloat16()
    return {"op": "attend", "fmt": fmt, "q": q, "k": k, "v": v, "k_scale": k_scale, "v_scale": v_scale, "block_tables": table,
            "seq_lens": _ints([b + n for b, n in zip(before, new)]), "cu_new": _ints(cu), "max_new": max(new)}


# ------------------------------------------------------------------ one pass
def run(state):
    if own:
        return _RUN[state["op"]](state)
    return _PLAIN[state["op"]](state)


def _values(codes, scale):
    """int8 codes as the bf16 values they stand for (e4m3 codes are a floating type already)."""
    if codes.dtype != torch.int8:
        return codes
    return torch.mul(codes, scale, out=torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device))


def _run_norm(s):
    import w8a8_int8_quantized_i8_gb300 as i8
    codes, scale, h = i8.add_rmsnorm_quant_act_pertoken(s["x"], s["residual"], s["weight"], eps=s["eps"], fmt=s["fmt"])
    return {"values": _values(codes, scale[:, None]), "scale": scale, "h": h}


def _run_tables(s):
    import w8a8_int8_quantized_i8_gb300 as i8
    plan = i8.build_block_tables(s["context_lens"], s["new_lens"], s["block_tables"], s["free_blocks"], s["block"],
                                 s["tokens"], taken=s["taken"], out=i8.BlockPlan(**s["out"]))
    return {"cu_new": plan.cu_new, "seq_lens": plan.seq_lens, "slots": plan.slots, "positions": plan.positions,
            "counts": plan.counts, "block_tables": s["block_tables"]}


def _cache_out(s):
    wide = lambda t: t[:, :, None, None]  # noqa: E731
    return {"k": _values(s["k"], wide(s["k_scale"])), "v": _values(s["v"], wide(s["v_scale"])),
            "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _run_append(s):
    import w8a8_int8_quantized_i8_gb300 as i8
    i8.kv_cache_append(s["keys"], s["values"], s["slots"], i8.QuantKVCache(s["k"], s["v"], s["k_scale"], s["v_scale"]))
    return _cache_out(s)


def _run_attend(s):
    import w8a8_int8_quantized_i8_gb300 as i8
    return i8.paged_attention(s["q"], i8.QuantKVCache(s["k"], s["v"], s["k_scale"], s["v_scale"]), s["block_tables"],
                              s["seq_lens"], s["cu_new"], max_new=s["max_new"])


# ------------------------------------------------------------------ plain forms
def _plain_norm(s):
    h = s["x"].float() + s["residual"].float()
    y = h * torch.rsqrt((h * h).mean(dim=1, keepdim=True) + s["eps"]) * s["weight"].float()
    scale = y.abs().amax(dim=1, keepdim=True) / _limit(s["fmt"])
    codes = _to_codes(torch.where(scale > 0, y / scale, 0.0), s["fmt"])
    return {"values": _values(codes, scale), "scale": scale[:, 0], "h": h.bfloat16()}


def _plain_tables(s):
    block, table, free = s["block"], s["block_tables"], s["free_blocks"]
    requests, width = table.shape
    before, new = s["context_lens"].long(), s["new_lens"].long()
    after = before + new
    cu = torch.zeros(requests + 1, dtype=torch.int64, device=table.device)
    cu[1:] = torch.cumsum(new, 0)
    held, need = (before + block - 1) // block, (after + block - 1) // block
    fresh = need - held
    first = s["taken"].long() + torch.cumsum(fresh, 0) - fresh  # each request's first new block in the free list
    column = torch.arange(width, device=table.device)
    at = first[:, None] + column - held[:, None]
    mine = (column >= held[:, None]) & (column < need[:, None])
    table.copy_(torch.where(mine, free[at.clamp(0, free.numel() - 1)], table))
    token = torch.arange(s["tokens"], device=table.device)
    real = token < cu[-1]
    request = torch.searchsorted(cu[1:], token, right=True).clamp(max=requests - 1)
    position = torch.where(real, before[request] + token - cu[request], 0)
    slots = torch.where(real, table[request, position // block].long() * block + position % block, -1)
    counts = torch.stack([cu[-1], s["taken"][0].long() + fresh.sum(), torch.zeros_like(cu[-1])])
    return {"cu_new": cu.int(), "seq_lens": after.int(), "slots": slots, "positions": position.int(),
            "counts": counts.int(), "block_tables": table}


def _plain_append_one(x, slots, codes, scale, fmt):
    block, limit = codes.shape[2], _limit(fmt)
    at, offset = slots // block, slots % block
    x = x.float()
    most = torch.zeros_like(scale).index_reduce_(0, at, x.abs().amax(dim=2), "amax")
    first = torch.full((scale.shape[0],), block, dtype=torch.int64, device=x.device).index_reduce_(0, at, offset, "amin")
    touched = torch.unique(at)
    base = torch.where(first[touched, None] > 0, scale[touched], 0.0)  # the scale of what the block holds already
    fresh = torch.maximum(base, most[touched] / torch.full_like(base, limit))
    ratio = torch.where(fresh > 0, base / fresh, 0.0)
    old = torch.arange(block, device=x.device) < first[touched, None]
    held = codes[touched]
    again = _to_codes(held.float() * ratio[:, :, None, None], fmt)
    bits = torch.int8 if fmt == "int8" else torch.uint8
    keep = torch.where(old[:, None, :, None], again.view(bits), held.view(bits))
    codes.view(bits)[touched] = keep
    scale[touched] = fresh
    over = scale[at][:, :, None]
    codes.view(bits)[at, :, offset] = _to_codes(torch.where(over > 0, x / over, 0.0), fmt).view(bits)


def _plain_append(s):
    _plain_append_one(s["keys"], s["slots"], s["k"], s["k_scale"], s["fmt"])
    _plain_append_one(s["values"], s["slots"], s["v"], s["v_scale"], s["fmt"])
    return _cache_out(s)


def _dense(codes, scale, table):
    """The blocks of a table as values [requests, heads, tokens, dim]."""
    at = table.clamp(min=0).long()
    x = codes[at].float() * scale[at][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attend(s):
    q, cu, lens, table = s["q"], s["cu_new"].long(), s["seq_lens"].long(), s["block_tables"]
    tokens, q_heads, dim = q.shape
    heads, requests, most = s["k"].shape[1], table.shape[0], s["max_new"]
    k, v = _dense(s["k"], s["k_scale"], table), _dense(s["v"], s["v_scale"], table)
    new = cu[1:] - cu[:-1]
    row = torch.arange(most, device=q.device)
    padded = q.float()[(cu[:-1, None] + row).clamp(max=tokens - 1)]  # [requests, most, q_heads, dim]
    padded = padded.unflatten(2, (heads, q_heads // heads)).permute(0, 2, 3, 1, 4).flatten(2, 3)
    scores = torch.matmul(padded, k.transpose(2, 3)) * dim ** -0.5  # [requests, heads, group * most, tokens]
    last = (lens - new)[:, None] + row  # the position of each new token
    seen = (torch.arange(k.shape[2], device=q.device) <= last[:, :, None]) & (row < new[:, None])[:, :, None]
    seen = seen.repeat(1, q_heads // heads, 1)[:, None]
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(dim=3, keepdim=True)
    scores.sub_(torch.where(top > -math.inf, top, 0.0)).exp_()
    total = scores.sum(dim=3, keepdim=True)
    out = torch.matmul(scores, v) / torch.where(total > 0, total, 1.0)
    out = out.unflatten(2, (q_heads // heads, most)).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [requests, most, q_heads, dim]
    token = torch.arange(tokens, device=q.device)
    request = torch.searchsorted(cu[1:], token, right=True)
    return out[request, token - cu[request]].bfloat16()


_PLAIN = {"norm": _plain_norm, "tables": _plain_tables, "append": _plain_append, "attend": _plain_attend}
_RUN = {"norm": _run_norm, "tables": _run_tables, "append": _run_append, "attend": _run_attend}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _nearest(x, fmt):
    """The values of the format nearest to x, in 64 bits, ties to the even one."""
    if fmt == "int8":
        return x.round().clamp(-INT8_MAX, INT8_MAX)
    exponent = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(exponent - 3)  # three bits after the leading one; below 2^-6 the steps stay 2^-9
    return ((x / step).round() * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_norm(s):
    h = s["x"].double() + s["residual"].double()
    y = h / (h.square().sum(1, keepdim=True) / h.shape[1] + s["eps"]).sqrt() * s["weight"].double()
    scale = y.abs().amax(1) / _limit(s["fmt"])
    codes = _nearest(y / scale[:, None], s["fmt"])
    return {"values": codes * scale[:, None] if s["fmt"] == "int8" else codes, "scale": scale, "h": h}


def _exact_append(s):
    fmt, out = s["fmt"], {}
    for name, x in (("k", s["keys"]), ("v", s["values"])):
        codes, scale = s[name].double(), s[name + "_scale"].double()
        block = codes.shape[2]
        at, offset = s["slots"] // block, s["slots"] % block
        # a block that begins with this step has nothing before it; the others keep at least the scale they have
        begun = torch.ones_like(scale[:, 0], dtype=torch.bool)
        begun[at[offset == 0]] = False
        written = torch.zeros_like(begun)
        written[at] = True
        target = torch.where((written & ~begun)[:, None], 0.0, scale)
        target = target.index_reduce(0, at, x.double().abs().amax(2) / _limit(fmt), "amax")
        again = _nearest(codes * (scale / target)[:, :, None, None], fmt)
        fresh = codes.clone()
        grown = (written & begun)[:, None] & (target > scale)
        is_new = torch.zeros(codes.shape[0], block, dtype=torch.bool, device=codes.device)
        is_new[at, offset] = True
        first = torch.where(is_new, torch.arange(block, device=codes.device), block).amin(1)
        before = torch.arange(block, device=codes.device) < first[:, None]
        fresh = torch.where(grown[:, :, None, None] & before[:, None, :, None], again, fresh)
        fresh[at, :, offset] = _nearest(x.double() / target[at][:, :, None], fmt)
        out[name] = fresh * target[:, :, None, None] if fmt == "int8" else fresh
        out[name + "_scale"] = target
    return out


def _exact_attend(s):
    q, cu, lens = s["q"].double(), s["cu_new"].tolist(), s["seq_lens"].tolist()
    heads, block = s["k"].shape[1], s["k"].shape[2]
    group = q.shape[1] // heads
    out = torch.zeros_like(q)
    for r, n in enumerate(lens):
        ids = s["block_tables"][r, : _blocks(n, block)].long()
        new = cu[r + 1] - cu[r]
        limit = torch.arange(n - new, n, device=q.device)[:, None] >= torch.arange(n, device=q.device)
        for head in range(heads):
            k = (s["k"][ids, head].double() * s["k_scale"][ids, head].double()[:, None, None]).reshape(-1, q.shape[2])[:n]
            v = (s["v"][ids, head].double() * s["v_scale"][ids, head].double()[:, None, None]).reshape(-1, q.shape[2])[:n]
            for j in range(head * group, (head + 1) * group):
                p = (q[cu[r]: cu[r + 1], j] @ k.T / math.sqrt(q.shape[2])).masked_fill(~limit, -math.inf)
                out[cu[r]: cu[r + 1], j] = torch.softmax(p, 1) @ v
    return out
