"""The decoder's attention over its caches, prompt against single tokens.

The residual stream hides what attention gives (a row's cosine stays above 0.99
with the attention left out), so the attention's own output is compared, token
by token of the cache, and the same comparisons are shown to fail for an
attention that lost or shifted tokens.
"""
import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _serving as ref
from w8a8_int8_quantized_i8_gb300 import decoder

pytestmark = pytest.mark.gpu


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("cache_fmt", ["int8", "e4m3"])
def test_the_last_token_s_attention_however_the_prompt_came(cache_fmt):
    """48 tokens as one prompt, as 47 and one, and in three parts.

    What the cache holds at a token's place is that token's key and value within
    half a code of its block's scale s each time it is coded, at most twice here
    (when it came, and when the block's last token raised the scale): s for
    int8, 2 * 2^-4 of the value or 2 * 2^-10 s for E4M3, the second of the once
    rounded value; a relative 2^-10 covers the fp32 quotients.  The last
    token's output is the attention over those values, within the roundings that
    attention_reference counts."""
    shape = decoder.Shape(blocks=1, width=512, q_heads=8, kv_heads=2, head_dim=64, mlp=1024, block_size=16,
                          cache_fmt=cache_fmt)
    x = torch.randn(48, shape.width, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    for parts in ([48], [47, 1], [16, 31, 1]):
        model = decoder.Decoder(shape, 4)
        reqs = decoder.Requests(1, 4, 4, shape.block_size)
        came, at = [], 0
        for n in parts:
            seen = {}
            model.step(x[at:at + n], reqs.plan(_ints([n]), n), reqs.block_tables, n,
                       record=lambda b, name, t: seen.setdefault(b, t))
            i8.sync_check()
            came.append(seen[0])
            at += n
        cache, table = model.caches[0], reqs.block_tables
        ids, place = table[0].long()[torch.arange(48) // 16], torch.arange(48) % 16
        for codes, scale, put in ((cache.k, cache.k_scale, torch.cat([c[1] for c in came])),
                                  (cache.v, cache.v_scale, torch.cat([c[2] for c in came]))):
            s = scale[ids].double()[..., None]
            got = codes.float().double()[ids, :, place] * s
            put = put.double()
            bound = s.expand_as(put) if cache_fmt == "int8" else 2 * (2.0 ** -4 * (1 + 2.0 ** -4) * put.abs()).clamp(min=2.0 ** -10 * s)
            bound = bound * (1 + 2.0 ** -10)
            assert ((got - put).abs() <= bound).all(), parts
            assert not ((got.roll(1, 0) - put).abs() <= bound).all()
        q, o = came[-1][0], came[-1][3][-1].double()

        def attention(k=cache.k.float().double(), v=cache.v.float().double(), vs=cache.v_scale):
            want, _, bound, _ = ref.attention_reference(q[-1:], k, v, cache.k_scale, vs, table.tolist(), [48], [0, 1],
                                                        shape.head_dim ** -0.5)
            return want[0], bound[0]

        want, bound = attention()
        assert ((o - want).abs() <= bound).all(), parts
        v = cache.v.float().double()
        lost = v.clone()
        lost[table[0, 0].long()] = 0                                       # the first block
        for wrong in (torch.zeros_like(want), attention(v=lost)[0], attention(v=v.roll(1, 2))[0]):
            assert not ((wrong - want).abs() <= bound).all()
