"""CPU model of the paged attention's global reads: the lanes' addresses of a
16-token half tile cover each code of K and of V exactly once, inside the
block; tiles of a sequence cover every token once, in blocks of its table; and
the fragments' head dimensions are a permutation."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _source():
    with open(os.path.join(ROOT, "w8a8_int8_quantized_i8_gb300", "csrc", "kv_attention.cuh")) as fh:
        return " ".join(re.sub(r"//[^\n]*", " ", fh.read()).split())


@pytest.mark.parametrize("D", [64, 128, 256])
def test_half_tile_reads_each_code_once(D):
    src = _source()
    assert "ld_stream_v4(kp + (g + 8 * i) * D + j * 64 + c * 16)" in src
    assert "ld_stream_v4(vp + tk * D + j * 128 + g * 16)" in src
    k, v = [0] * (16 * D), [0] * (16 * D)
    for lane in range(32):
        g, c = lane >> 2, lane & 3
        for i in range(2):
            for j in range(D // 64):
                a = (g + 8 * i) * D + j * 64 + c * 16
                assert a % 16 == 0
                for b in range(16):
                    k[a + b] += 1
        size = min(16, D // 8)
        for i in range(4):
            tk = 2 * c + (i & 1) + 8 * (i >> 1)
            for j in range(max(1, D // 128)):
                a = tk * D + j * 128 + g * size
                assert a % size == 0
                for b in range(size):
                    v[a + b] += 1
    assert set(k) == {1} and set(v) == {1}


@pytest.mark.parametrize("D", [64, 128, 256])
def test_output_rows_are_a_permutation_of_the_head_dimension(D):
    vb = min(16, D // 8)
    dims = sorted((2 * j + half) // vb * 128 + g * vb + (2 * j + half) % vb
                  for j in range(D // 16) for half in range(2) for g in range(8))
    assert dims == list(range(D))
    assert sorted((j >> 2) * 64 + c * 16 + (j & 3) * 4 + b for j in range(D // 16) for c in range(4) for b in range(4)) \
        == list(range(D))


@pytest.mark.parametrize("block", [16, 48, 64, 1024])
def test_halves_stay_inside_a_block(block):
    for t in range(0, 4 * block, 16):
        off = t - t // block * block
        assert off % 16 == 0 and off + 16 <= block
