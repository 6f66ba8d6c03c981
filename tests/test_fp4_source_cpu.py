"""Source guards of the 4-bit route's and the rotation's kernels: they may begin
while the kernel before them still runs, so their loads are ordinary ones; every
wait is bounded, nothing traps, and a CTA that gives up ends after its copies."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w8a8_int8_quantized_i8_gb300", "csrc")
SOURCES = ["fp4_format.cuh", "fp4_quant.cuh", "fp4_mma.cuh", "fp4_stream.cuh", "fp4_pair.cuh", "heads_rotate.cuh"]


def _code(name):
    """The source with comments removed and whitespace collapsed."""
    with open(os.path.join(CSRC, name)) as fh:
        text = fh.read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    text = re.sub(r"//[^\n]*", " ", text)
    return " ".join(text.split())


@pytest.mark.parametrize("name", SOURCES)
def test_loads_are_ordinary(name):
    for promise in ("__ldg", "ld.global.nc", "ld_stream_v4", "__restrict__"):
        assert promise not in _code(name), (name, promise)


@pytest.mark.parametrize("name", SOURCES)
def test_every_wait_is_bounded_and_nothing_traps(name):
    src = _code(name)
    for word in ("mbar_try_wait", "for (;;)", "do {", "__trap", "trap;", "while ("):
        assert word not in src, (name, word)
    assert not re.search(r"(?<!static_)\bassert\(", src), name


@pytest.mark.parametrize("name", ["fp4_stream.cuh", "fp4_pair.cuh"])
def test_a_kernel_touches_global_memory_behind_the_wait(name):
    """What comes before pdl_wait() is descriptors and prefetches into L2."""
    kernel = re.search(r"__global__.*", _code(name)).group(0)
    before = kernel[: kernel.index("pdl_wait();")]
    before = re.sub(r"bulk_prefetch_l2\(p\.w\[\d\]\.scales \+ ws0, ahead\);", "", before)
    for load in ("p.w[", "p.scales", "p.row_scales", "p.y", "tma_load", "bulk_load"):
        assert load not in before, (name, load)


@pytest.mark.parametrize("name", ["fp4_stream.cuh", "fp4_pair.cuh"])
def test_what_is_on_its_way_ends_before_the_cta_does(name):
    src = _code(name)
    assert re.search(r"if \(!ok(?: && rank == 0)?\) for \(int \w = max\(0, issued - Cfg::STAGES\); \w < issued; \+\+\w\) "
                     r"mbar_wait_bounded\(", src)
    assert re.search(r"mbar_wait_bounded\((?:smem_u32\(&done\)|done), 0u, 100000000ull\);", src)


def test_co_resident_ctas_share_tensor_memory():
    """Two CTAs of the streaming kernel share an SM, and a cluster's CTAs wait for one another: their tensor
    memory fits together, or they do not fit together at all."""
    assert "static_assert(STAGES >= 2 && (COLS <= 256 || SMEM > 120 * 1024));" in _code("fp4_stream.cuh")
