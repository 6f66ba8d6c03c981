"""Plain 64-bit forms of the serving operators, for their tests."""
import math

import torch

LIMIT = {"int8": 127.0, "f16codes": 127.0, "e4m3": 448.0}


def nearest(x, fmt):
    """The format's value nearest to x (fp64), ties to even."""
    if fmt != "e4m3":
        return x.round().clamp(-127, 127)
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -40))).clamp(min=-6) - 3)
    return ((x / step).round() * step).clamp(-448, 448)


def f32_div(a, b):
    """The fp32 quotient of fp32 values, correctly rounded (53 bits are enough
    for the double rounding to be harmless)."""
    return (a.double() / b.double()).float()


def norm_reference(x, residual, weight, eps, fmt):
    """codes (as values), scale and h of add_rmsnorm_quant, by its definition's
    fp32 steps; the scale from the fp64 mean."""
    h = x.float() + residual.float() if residual is not None else x.float()
    t = h * weight.float() if weight is not None else h
    amax = t.abs().amax(1)
    s_t = f32_div(amax, torch.tensor(LIMIT[fmt]))
    codes = torch.where(s_t[:, None] > 0, f32_div(t, s_t[:, None]).double(), 0.0)
    rstd = 1.0 / (h.double().square().mean(1) + eps).sqrt()
    scale = torch.where(amax > 0, s_t.double() * rstd, 0.0)
    return nearest(codes, fmt), scale, h


def tables_reference(context, new, table, free, taken, block, max_tokens):
    """build_block_tables with Python integers (lists in, lists out)."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    cu, lens, slots, positions = [0], [], [], []
    used, lost = taken, 0
    for r, (c, n) in enumerate(zip(context, new)):
        c, n = max(0, c), max(0, n)
        held, need = min(-(-c // block), width), min(-(-(c + n) // block), width)
        for col in range(held, need):
            table[r][col] = free[used] if used < len(free) else -1
            used += 1
        for p in range(c, c + n):
            b = table[r][p // block] if p // block < width else -1
            # a missing block counts as lost only where the free list or the width ran out
            if p // block >= width or (p // block >= held and used - (need - held) + p // block - held >= len(free)):
                lost += 1
            slots.append(b * block + p % block if b >= 0 else -1)
            positions.append(p)
        cu.append(cu[-1] + n)
        lens.append(c + n)
    counts = [cu[-1], min(used, max(taken, len(free))), lost]
    slots += [-1] * (max_tokens - len(slots))
    positions += [0] * (max_tokens - len(positions))
    return table, cu, lens, slots[:max_tokens], positions[:max_tokens], counts


def append_reference(x, slots, codes, scale, fmt):
    """kv_cache_append of one tensor, token run by token run, in the
    definition's fp32 steps; codes (values, fp64) and scale (fp32) in place."""
    block = codes.shape[2]
    runs = []                                  # (first slot, tokens), skipped tokens left out
    for t, s in enumerate(slots):
        if s < 0:
            continue
        if runs and runs[-1][0] // block == s // block:
            runs[-1][1].append(t)
        else:
            runs.append((s, [t]))
    for s, tokens in runs:
        b, off = divmod(s, block)
        n = len(tokens)
        run = x[tokens].float()                                    # [n, heads, D]
        old = scale[b].clone() if off else torch.zeros_like(scale[b])
        fresh = torch.maximum(old, f32_div(run.abs().amax(dim=(0, 2)), torch.tensor(LIMIT[fmt])))
        for h in range(codes.shape[1]):
            if off and fresh[h] > old[h]:
                ratio = f32_div(old[h], fresh[h])
                codes[b, h, :off] = nearest((codes[b, h, :off].float() * ratio).double(), fmt)
            q = f32_div(run[:, h], fresh[h]).double() if fresh[h] > 0 else torch.zeros_like(run[:, h]).double()
            codes[b, h, off:off + n] = nearest(q, fmt)
        scale[b] = fresh


def code_values(t):
    """Codes as fp64 values on the CPU."""
    return t.detach().cpu().float().double()


def attention_reference(q, k, v, k_scale, v_scale, table, lens, cu, scale):
    """(out, lse, bound on out, bound on lse) in fp64; k, v are code values
    [blocks, heads, B, D].  Ids out of range are left out.  The bounds count
    roundings: the result's to bf16 (half a step), P's to fp16 (half a step of
    each term, and the fp16 subnormals' spacing 2^-24 of the largest 2^10), the
    fp32 sums of D products, and the exponential's few units."""
    T, Hq, D = q.shape
    P, Hkv, B, _ = k.shape
    q = q.double()
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=q.device)
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    for r, n in enumerate(lens):
        new = cu[r + 1] - cu[r]
        if new <= 0 or n <= 0:
            continue
        ids = table[r][: -(-n // B)]
        keep = [0 <= i < P for i in ids]
        at = torch.tensor([i if ok else 0 for i, ok in zip(ids, keep)], device=q.device)
        ok = torch.tensor(keep, device=q.device).repeat_interleave(B)[:n]
        seen = (torch.arange(n, device=q.device) <= torch.arange(n - new, n, device=q.device)[:, None]) & ok
        for h in range(Hkv):
            ks = k_scale[at, h].double().repeat_interleave(B)[:n, None]
            vs = v_scale[at, h].double().repeat_interleave(B)[:n, None]
            kk = (k[at, h].reshape(-1, D)[:n] * ks).masked_fill(~ok[:, None], 0.0)
            vv = (v[at, h].reshape(-1, D)[:n] * vs).masked_fill(~ok[:, None], 0.0)
            used = seen.any(0)
            kk, vv = kk.masked_fill(~used[:, None], 0.0), vv.masked_fill(~used[:, None], 0.0)
            for g in range(Hq // Hkv):
                j = h * (Hq // Hkv) + g
                qq = q[cu[r]:cu[r + 1], j]
                s = (qq @ kk.T * scale).masked_fill(~seen, -math.inf)
                live = seen.any(1)
                top = s.amax(1, keepdim=True)
                p = torch.where(seen, (s - torch.where(live[:, None], top, 0.0)).exp(), 0.0)
                l = p.sum(1, keepdim=True)
                l1 = torch.where(l > 0, l, 1.0)
                o = p @ vv / l1
                delta = ((qq.abs() @ kk.abs().T * abs(scale)) * (D + 8) * 2.0 ** -24).masked_fill(~seen, 0).amax(1, keepdim=True) \
                    + 2.0 ** -20
                a = p @ vv.abs() / l1
                bound[cu[r]:cu[r + 1], j] = (2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * delta) * a
                                             + n * 2.0 ** -35 * vv.abs().amax())
                out[cu[r]:cu[r + 1], j] = o
                lse[cu[r]:cu[r + 1], j] = torch.where(live, (top + l.log())[:, 0], -math.inf)
                lse_bound[cu[r]:cu[r + 1], j] = delta[:, 0] * 2 + 2.0 ** -22 * lse[cu[r]:cu[r + 1], j].abs().clamp(max=1e6) \
                    + n * 2.0 ** -24
    return out, lse, bound, lse_bound


def attention_definition(q, k, v, k_scale, v_scale, table, lens, cu, scale, code_max):
    """(out, lse, bound on out, bound on lse) in fp64, as attention_reference,
    for values far apart and for NaN: a row's result depends on the tokens that
    it sees and on nothing else.  A sequence's tokens past its table, or without
    a block, are absent; rows keep their positions.  code_max is the format's
    largest code.  What P's fp16 loses is counted from the row's own largest
    term: half the spacing 2^-24 of fp16's subnormals, of at least 2^6."""
    T, Hq, D = q.shape
    P, Hkv, B, _ = k.shape
    dev = q.device
    q = q.double()
    out = torch.zeros(T, Hq, D, dtype=torch.float64, device=dev)
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device=dev)
    bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
    for r, n in enumerate(lens):
        new = cu[r + 1] - cu[r]
        if new <= 0:
            continue
        end = min(max(n, 0), len(table[r]) * B)
        pos = torch.arange(n - new, n, device=dev)
        if end == 0:
            continue
        ids = table[r][: -(-end // B)]
        keep = [0 <= i < P for i in ids]
        at = torch.tensor([i if ok else 0 for i, ok in zip(ids, keep)], device=dev)
        ok = torch.tensor(keep, device=dev).repeat_interleave(B)[:end]
        seen = (torch.arange(end, device=dev) <= pos[:, None]) & ok
        for h in range(Hkv):
            ks = k_scale[at, h].double().repeat_interleave(B)[:end, None]
            vs = v_scale[at, h].double().repeat_interleave(B)[:end, None]
            kk, vv = k[at, h].reshape(-1, D)[:end] * ks, v[at, h].reshape(-1, D)[:end] * vs
            spoilt = (seen.double() @ torch.isnan(vv).double()) > 0
            vv = torch.nan_to_num(vv, nan=0.0)
            top_v = torch.nan_to_num(vs[:, 0], nan=0.0) * code_max
            for g in range(Hq // Hkv):
                j, rows = h * (Hq // Hkv) + g, slice(cu[r], cu[r + 1])
                qq = q[rows, j]
                s = (qq @ kk.T * scale).masked_fill(~seen, -math.inf)
                live = seen.any(1)
                top = s.amax(1, keepdim=True)
                p = torch.where(seen, (s - torch.where(live[:, None], top, 0.0)).exp(), 0.0)
                l = p.sum(1, keepdim=True)
                l1 = torch.where(live[:, None], l, 1.0)
                o = torch.where(spoilt, math.nan, p @ vv / l1)
                delta = ((qq.abs() @ kk.abs().T * abs(scale)) * (D + 8) * 2.0 ** -24).masked_fill(~seen, 0).amax(1, keepdim=True) \
                    + 2.0 ** -19
                a = p @ vv.abs() / l1
                bound[rows, j] = (2.0 ** -8 * o.abs() + (2.0 ** -11 + 2 * delta) * a
                                  + end * 2.0 ** -31 * (p * top_v / l1).amax(1, keepdim=True) + 2.0 ** -134)
                out[rows, j] = o
                lse[rows, j] = torch.where(live, (top + l.log())[:, 0], -math.inf)
                lse_bound[rows, j] = delta[:, 0] * 2 + 2.0 ** -22 * lse[rows, j].abs().clamp(max=1e6) + end * 2.0 ** -24
    return out, lse, bound, lse_bound


def check_attention(out, lse, want):
    """NaN exactly where the definition has it, the rest within its bound."""
    o, l, bound, lse_bound = want
    out, lse = out.double(), lse.double()
    nan = torch.isnan(o)
    assert torch.equal(torch.isnan(out), nan)
    err = (out - o).abs()[~nan]
    assert (err <= bound[~nan]).all(), f"worst {float((err - bound[~nan]).max()):.3g} over the bound"
    assert torch.equal(torch.isnan(lse), torch.isnan(l))
    assert torch.equal(torch.isinf(lse) & (lse < 0), torch.isinf(l))
    assert (out[torch.isinf(l)] == 0).all()
    plain = torch.isfinite(l)
    assert ((lse - l).abs()[plain] <= lse_bound[plain]).all()
