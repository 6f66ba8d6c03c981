"""kv_cache_append against its definition: codes and scales bit for bit, and
nothing else of the cache touched."""
import random

import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _serving as ref

pytestmark = pytest.mark.gpu


def _pool(blocks, heads, block, D, fmt, g):
    bits = torch.randint(0, 256, (blocks, heads, block, D), generator=g, dtype=torch.int32).to(torch.uint8)
    if fmt == "e4m3":
        bits[(bits & 0x7F) == 0x7F] = 0x38          # no NaN codes among the older tokens
        codes = bits.view(torch.float8_e4m3fn)
    else:
        codes = bits.view(torch.int8).clamp(min=-127)
    return codes, torch.rand(blocks, heads, generator=g) * (0.02 if fmt == "int8" else 0.006) + 1e-4


def _slots(requests, block, rng):
    """Slots of requests (context, new) over shuffled blocks."""
    ids = list(range(sum(-(-(c + n) // block) for c, n in requests) + 2))
    rng.shuffle(ids)
    out = []
    for c, n in requests:
        mine = [ids.pop() for _ in range(-(-(c + n) // block))]
        out += [mine[p // block] * block + p % block for p in range(c, c + n)]
    return out


def _check(x, cache_cpu, slots, cache, fmt):
    for name, src in zip("kv", x):
        codes, scale = cache_cpu[name]
        want, ws = ref.code_values(codes), scale.clone()
        ref.append_reference(src, slots, want, ws, fmt)
        got, gs = getattr(cache, name), getattr(cache, name + "_scale").cpu()
        assert torch.equal(gs.view(torch.int32), ws.view(torch.int32))
        assert torch.equal(ref.code_values(got), want)


def _case(requests, block, heads, D, fmt, seed, spread=1.0, q_heads=None, slots=None):
    g, rng = torch.Generator().manual_seed(seed), random.Random(seed)
    slots = _slots(requests, block, rng) if slots is None else slots
    T = len(slots)
    blocks = max([s // block for s in slots] + [0]) + 2
    (kc, ks), (vc, vs) = _pool(blocks, heads, block, D, fmt, g), _pool(blocks, heads, block, D, fmt, g)
    if q_heads is None:
        k, v = (torch.randn(T, heads, D, generator=g).mul(spread).bfloat16() for _ in range(2))
        dk, dv = k.cuda(), v.cuda()
    else:                                              # views of the fused projection's output
        qkv = torch.randn(T, (q_heads + 2 * heads) * D, generator=g).mul(spread).bfloat16()
        cut = lambda t, a: t[:, a * D:(a + heads) * D].unflatten(1, (heads, D))  # noqa: E731
        k, v = cut(qkv, q_heads), cut(qkv, q_heads + heads)
        dq = qkv.cuda()
        dk, dv = cut(dq, q_heads), cut(dq, q_heads + heads)
    cache = i8.QuantKVCache(kc.view(torch.uint8).cuda().view(kc.dtype), vc.view(torch.uint8).cuda().view(vc.dtype),
                            ks.cuda(), vs.cuda())
    i8.kv_cache_append(dk, dv, torch.tensor(slots, dtype=torch.int64, device="cuda"), cache)
    i8.sync_check()
    _check((k, v), {"k": (kc, ks), "v": (vc, vs)}, slots, cache, fmt)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("block,heads,D", [(16, 1, 64), (16, 8, 128), (48, 3, 64), (64, 2, 256), (128, 2, 128)])
def test_steps(block, heads, D, fmt):
    _case([(5, 1)], block, heads, D, fmt, 1)                                     # one token
    _case([(c, 1) for c in range(40)], block, heads, D, fmt, 2, q_heads=3 * heads)   # a decode step
    _case([(0, 200), (3, 2), (17, 1), (block - 1, 2), (block, 130), (30, 3)], block, heads, D, fmt, 3, q_heads=heads)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("spread", [0.0, 1e-3, 30.0, 1e-38])
def test_loud_and_quiet(spread, fmt):
    """New tokens far louder or quieter than the block, zeros, and subnormals."""
    _case([(3, 1), (20, 5), (0, 1), (0, 40)], 16, 2, 64, fmt, 5, spread)


def test_many_requests_and_long_prompt():
    _case([(c % 37, 1) for c in range(3000)], 16, 2, 64, "int8", 6)
    _case([(7, 2047), (0, 512)], 64, 2, 128, "e4m3", 7)


def test_skipped_tokens():
    slots = [-1, 35, -1, 36, 37, -1, -1, 0, 1, -1]
    _case(None, 16, 2, 64, "int8", 8, slots=slots)
    _case(None, 16, 2, 64, "int8", 9, slots=[-1] * 40)


def test_token_by_token_keeps_the_older_codes():
    """The same tokens one step at a time: the scale only grows, and equals the
    whole block's in the end."""
    g = torch.Generator().manual_seed(11)
    block, heads, D, fmt = 16, 2, 64, "int8"
    x = torch.randn(block, heads, D, generator=g).bfloat16()
    cache = i8.QuantKVCache.empty(2, heads, block, D, fmt)
    want, scale = ref.code_values(cache.k), cache.k_scale.cpu().clone()
    for t in range(block):
        i8.kv_cache_append(x[t:t + 1].cuda(), x[t:t + 1].cuda(), torch.tensor([block + t], device="cuda"), cache)
        ref.append_reference(x[t:t + 1], [block + t], want, scale, fmt)
    i8.sync_check()
    assert torch.equal(ref.code_values(cache.k), want) and torch.equal(cache.v_scale.cpu(), scale)
    assert torch.equal(scale[1], ref.f32_div(x.float().abs().amax(dim=(0, 2)), torch.tensor(127.0)))
    # a begun block starts over when its offset 0 is written again
    y = (x[:1] * 0.01).bfloat16()
    i8.kv_cache_append(y.cuda(), y.cuda(), torch.tensor([block], device="cuda"), cache)
    i8.sync_check()
    assert torch.equal(cache.k_scale.cpu()[1], ref.f32_div(y.float().abs().amax(dim=(0, 2)), torch.tensor(127.0)))


def test_slots_out_of_range_are_reported():
    """Past the pool, or a block's tokens out of order: not written, and
    sync_check says so."""
    g = torch.Generator().manual_seed(12)
    k = torch.randn(3, 1, 64, generator=g).bfloat16().cuda()
    for slots in ([48, 0, 1], [1 << 40, -5, 1], [4, 3, 0]):
        cache = i8.QuantKVCache.empty(3, 1, 16, 64, "int8")
        i8.kv_cache_append(k, k, torch.tensor(slots, device="cuda"), cache)
        with pytest.raises(i8.I8Error) as e:
            i8.sync_check()
        assert e.value.status == 7
        i8.sync_check()                                   # read and cleared
        written = {s for i, s in enumerate(slots) if 0 <= s < 48 and slots != [4, 3, 0]} | ({4} if slots == [4, 3, 0] else set())
        rows = cache.k.cpu().reshape(48, 64).ne(0).any(1).nonzero()[:, 0].tolist()
        assert set(rows) == written


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_nan_shows_in_the_scale(fmt):
    """A NaN among a block's new tokens makes that block's scale of that head
    NaN, and it stays so until the block is begun again; nothing else differs
    from the same step without it, and attention over it is NaN."""
    g = torch.Generator().manual_seed(13)
    heads, block, D = 2, 16, 64
    x = torch.randn(40, heads, D, generator=g).bfloat16()
    bad = x.clone()
    bad[20, 1, 9] = float("nan")                          # block 1, head 1
    bad[39, 0, 0] = float("-nan")                         # block 2, head 0, with older tokens before it
    caches = []
    for k in (x, bad):
        cache = i8.QuantKVCache.empty(3, heads, block, D, fmt)
        for lo, hi in ((0, 36), (36, 40)):
            i8.kv_cache_append(k[lo:hi].cuda(), x[lo:hi].cuda(), torch.arange(lo, hi, device="cuda"), cache)
        caches.append(cache)
    i8.sync_check()
    good, spoilt = caches
    nan = torch.zeros(3, heads, dtype=torch.bool)
    nan[1, 1] = nan[2, 0] = True
    assert torch.equal(torch.isnan(spoilt.k_scale).cpu(), nan)
    assert torch.equal(spoilt.k_scale.cpu()[~nan], good.k_scale.cpu()[~nan])
    assert torch.equal(spoilt.k.view(torch.uint8).cpu()[~nan], good.k.view(torch.uint8).cpu()[~nan])
    assert torch.equal(spoilt.v.view(torch.uint8), good.v.view(torch.uint8)) and torch.equal(spoilt.v_scale, good.v_scale)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.randn(2, heads, D, generator=g).bfloat16().cuda()
    o = i8.paged_attention(q, spoilt, i32([[0, 1, 2], [0, 1, 2]]), i32([40, 10]), i32([0, 1, 2]), max_new=1)
    i8.sync_check()
    assert torch.isnan(o[0]).all() and torch.isfinite(o[1]).all()
    # more tokens do not hide it, a new beginning does
    i8.kv_cache_append(x[:2].cuda(), x[:2].cuda(), torch.tensor([40, 41], device="cuda"), spoilt)
    i8.sync_check()
    assert torch.isnan(spoilt.k_scale[2, 0])
    i8.kv_cache_append(x[:2].cuda(), x[:2].cuda(), torch.tensor([32, 33], device="cuda"), spoilt)
    i8.sync_check()
    assert torch.isfinite(spoilt.k_scale[2]).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("gap", [31, 32, 255, 256, 257, 5000, 100000])
def test_long_stretches_of_skipped_tokens(gap, fmt):
    """Skipped tokens before, inside and between runs: a run goes on behind them,
    and what begins behind them begins a run."""
    slots = [-1] * gap + [35, 36] + [-1] * gap + [37, 0] + [-1] * gap + [1, 2, 64] + [-1] * gap
    g = torch.Generator().manual_seed(gap)
    T, heads, D = len(slots), 1, 64
    (kc, ks), (vc, vs) = _pool(5, heads, 16, D, fmt, g), _pool(5, heads, 16, D, fmt, g)
    rows = torch.randn(T, heads, D, generator=g).bfloat16()
    cache = i8.QuantKVCache(kc.view(torch.uint8).cuda().view(kc.dtype), vc.view(torch.uint8).cuda().view(vc.dtype),
                            ks.cuda(), vs.cuda())
    i8.kv_cache_append(rows.cuda(), rows.cuda(), torch.tensor(slots, dtype=torch.int64, device="cuda"), cache)
    i8.sync_check()
    _check((rows, rows), {"k": (kc, ks), "v": (vc, vs)}, slots, cache, fmt)
