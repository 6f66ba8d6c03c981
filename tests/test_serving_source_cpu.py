"""Source guards of the serving operators' kernels.

Their kernels are launched so that they may begin while the kernel before them
in the stream still runs, and h of the norm may lie where x or the residual
does.  So the loads after the wait are ordinary ones: the read-only path
(ld.global.nc: __ldg, and what the compiler makes of const __restrict__) is for
memory that nobody writes while the kernel lives.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w8a8_int8_quantized_i8_gb300", "csrc")


def _code(name):
    """The source with comments removed and whitespace collapsed."""
    with open(os.path.join(CSRC, name)) as fh:
        text = fh.read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    text = re.sub(r"//[^\n]*", " ", text)
    return " ".join(text.split())


@pytest.mark.parametrize("name", ["rmsnorm.cuh", "block_tables.cuh", "kv_append.cuh", "kv_attention.cuh",
                                  "kv_prefill.cuh"])
def test_loads_are_ordinary(name):
    """The norm's gains, a model's parameters, are the exception."""
    src = _code(name).replace("g = __ldg(reinterpret_cast<const uint4*>(weight + e));", "")
    for promise in ("__ldg", "ld.global.nc", "ld_stream_v4", "__restrict__"):
        assert promise not in src, (name, promise)


SOURCES = ["rmsnorm.cuh", "block_tables.cuh", "kv_append.cuh", "kv_attention.cuh", "kv_prefill.cuh"]


@pytest.mark.parametrize("name", SOURCES)
def test_every_wait_is_bounded_and_nothing_traps(name):
    src = _code(name)
    for word in ("mbar_try_wait", "for (;;)", "do {", "__trap", "trap;"):
        assert word not in src, (name, word)
    assert not re.search(r"\bwhile\s*\((?!off|a\.box)", src), name
    assert not re.search(r"(?<!static_)\bassert\(", src), name


def test_what_is_on_its_way_ends_before_the_cta_does():
    """A CTA that gives up waits, bounded, for its own copies and products: a copy
    that lands later writes another CTA's shared memory.  Whichever role gave up,
    the copying and the issuing warp of the chunks' kernel drain after the last
    barrier; a warp of the few-row kernel drains its ring where it gives up."""
    few, many = _code("kv_attention.cuh"), _code("kv_prefill.cuh")
    m = re.search(r"if \(!mbar_wait\(bars \+ 8 \* slot, \(parity >> slot\) & 1u, abort_flag\)\) \{(.*?)break; \}", few)
    assert m and "for (int i = 0; i < S - 1; ++i, t0 += Tile::UNIT)" in m.group(1)
    assert "mbar_wait_bounded(bars + 8 * at, (parity >> at) & 1u, kDrainLimitNs);" in m.group(1)
    end = many[many.index("copied = item;"):]
    m = re.search(r"__syncthreads\(\); if \(abort_flag\) \{(.*?)\} pdl_trigger\(\);", end)
    assert m, "the drain does not follow the last barrier"
    assert "at = max(0, copied - kPreSlots); at < copied;" in m.group(1)
    assert "mbar_wait_bounded(smem_u32(&raw_full[at % kPreSlots]), (at / kPreSlots) & 1, kDrainLimitNs);" in m.group(1)
    assert "mma_commit_warp(smem_u32(&drained)); mbar_wait_bounded(smem_u32(&drained), 0, kDrainLimitNs);" in m.group(1)
    assert "tmem_dealloc(tmem, 512);" in end[m.end():]


def test_a_run_s_vectors_are_counted_in_64_bits():
    """Skipped tokens count into a run's span: 2^26 of them are 2^31 vectors of a
    256-wide head, so the loops over them count in 64 bits."""
    src = _code("kv_append.cuh")
    assert "const int64_t n = static_cast<int64_t>(run.span) << vs;" in src
    assert not re.search(r"for \(int i = me \+ kAppendKeep \* threads; i < n;", src)
    assert len(re.findall(r"for \(int64_t i = me \+ kAppendKeep \* threads; i < n;", src)) == 2
