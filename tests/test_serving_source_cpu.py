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
