"""CPU model of the paged attention's reads.

The TMA boxes of a half tile (16 tokens) land swizzled in shared memory: the
lanes' reads cover each code of K and of V exactly once, and a quarter warp's
16-byte reads meet no bank twice.  The fragments' head dimensions are a
permutation.  The columns and offsets that a warp steps through are those of
its tiles, and every 16-token half stays inside a block.
"""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _source():
    with open(os.path.join(ROOT, "w8a8_int8_quantized_i8_gb300", "csrc", "kv_attention.cuh")) as fh:
        return " ".join(re.sub(r"//[^\n]*", " ", fh.read()).split())


def _place(D, row, byte):
    tokens = 16 if D == 256 else 32
    if D == 64:
        return row * 64 + (byte ^ (((row >> 1) & 3) << 4))
    return (byte >> 7) * (tokens * 128) + row * 128 + ((byte & 127) ^ ((row & 7) << 4))


def _k_dim(D, j, c):
    return c * 16 if D == 64 else (j >> 1) * 128 + (2 * c + (j & 1)) * 16


def _swizzled(D, row, byte):
    """Where TMA puts it: 16-byte chunks of the address xor-ed with address bits
    7..9 (128-byte swizzle) or 7..8 (64-byte)."""
    tokens = 16 if D == 256 else 32
    box = min(D, 128)
    a = byte // box * (tokens * 128) + row * box + byte % box
    return a ^ (((a >> 7) & (7 if box == 128 else 3)) << 4)


def test_the_model_is_the_source():
    src = _source()
    assert "if constexpr (D == 64) return row * 64 + (byte ^ (((row >> 1) & 3) << 4));" in src
    assert "return (byte >> 7) * (AttnTile<D>::TOKENS * 128) + row * 128 + ((byte & 127) ^ ((row & 7) << 4));" in src
    assert "return D == 64 ? c * 16 : (j >> 1) * 128 + (2 * c + (j & 1)) * 16;" in src
    assert "lds_16(stage + h * 16 * Tile::BOX + attn_place<D>(g + 8 * i, attn_k_dim<D>(j, c)))" in src
    assert "lds_16(half + attn_place<D>(tk, j * 128 + g * 16))" in src
    assert "lds_8(half + attn_place<D>(tk, g * 8))" in src
    # every innermost TMA coordinate is a multiple of a box, 64 or 128 bytes
    assert src.count("tma_load_3d(") == 2 and src.count("bar, b * Tile::BOX, f.next_off[h], row)") == 2


@pytest.mark.parametrize("D", [64, 128, 256])
def test_reads_cover_each_code_once_without_conflicts(D):
    assert all(_place(D, r, b) == _swizzled(D, r, b) for r in range(16) for b in range(D))
    k, v = {}, {}
    for j in range(D // 64):
        for row_add in (0, 8):
            for q in range(4):
                banks = set()
                for lane in range(8 * q, 8 * q + 8):
                    g, c = lane >> 2, lane & 3
                    a = _place(D, g + row_add, _k_dim(D, j, c))
                    assert a % 16 == 0
                    banks.add(a // 16 % 8)
                    for b in range(16):
                        k[a + b] = k.get(a + b, 0) + 1
                assert len(banks) == 8
    size = min(16, D // 8)
    for i in range(4):
        for j in range(max(1, D // 128)):
            for q in range(4):
                banks = set()
                for lane in range(8 * q, 8 * q + 8):
                    g, c = lane >> 2, lane & 3
                    tk = 2 * c + (i & 1) + 8 * (i >> 1)
                    a = _place(D, tk, j * 128 + g * size)
                    assert a % size == 0
                    banks.add(a // 16 % 8)
                    for b in range(size):
                        v[a + b] = v.get(a + b, 0) + 1
                assert D == 64 or len(banks) == 8
    assert len(k) == len(v) == 16 * D and set(k.values()) == set(v.values()) == {1}


@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_dimensions_are_permutations(D):
    vb = min(16, D // 8)
    dims = sorted((2 * j + half) // vb * 128 + g * vb + (2 * j + half) % vb
                  for j in range(D // 16) for half in range(2) for g in range(8))
    assert dims == list(range(D))
    assert sorted(_k_dim(D, j >> 2, c) + (j & 3) * 4 + b for j in range(D // 16) for c in range(4) for b in range(4)) \
        == list(range(D))


@pytest.mark.parametrize("block", [16, 32, 48, 64, 112, 128, 160, 1024])
@pytest.mark.parametrize("tokens", [16, 32])
def test_columns_and_offsets_follow_the_tiles(block, tokens):
    unit = 4 * tokens
    for warp in range(4):
        for begin in (0, unit, 7 * unit):
            t = begin + warp * tokens
            col, off = t // block, t % block
            for _ in range(40):
                for h in range(tokens // 16):
                    wraps = off + 16 * h >= block
                    c, o = col + wraps, off + 16 * h - (block if wraps else 0)
                    assert (c, o) == ((t + 16 * h) // block, (t + 16 * h) % block)
                    assert o % 16 == 0 and o + 16 <= block
                if block % 32 == 0 and tokens == 32:      # one box of 32: both halves in one block
                    assert off + 32 <= block
                t += unit
                col, off = col + unit // block, off + unit % block
                if off >= block:
                    off, col = off - block, col + 1
