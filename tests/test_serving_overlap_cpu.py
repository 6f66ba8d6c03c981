"""build_block_tables refuses operands that share memory, on the host: every CTA
reads the inputs for itself, so an output in their place is a race.  (Only
refusals here: the addresses are no memory.)"""
import ctypes

import pytest

from w8a8_int8_quantized_i8_gb300 import binding

R, WIDTH, LD, FREE, T = 6, 4, 10, 20, 32
SIZES = dict(context=4 * R, new=4 * R, table=4 * (LD * (R - 1) + WIDTH), free=4 * FREE, taken=4, cu=4 * (R + 1),
             lens=4 * R, slots=8 * T, positions=4 * T, counts=12)
INPUTS, OUTPUTS = ("context", "new", "free", "taken"), ("table", "cu", "lens", "slots", "positions", "counts")
BASE = {name: 0x100000 + 0x1000 * i for i, name in enumerate(SIZES)}


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def _call(lib, **at):
    a = {name: ctypes.c_void_p(v) for name, v in {**BASE, **at}.items()}
    return lib.i8_build_block_tables(a["context"], a["new"], R, a["table"], WIDTH, LD, a["free"], FREE, a["taken"], 16, T,
                                     a["cu"], a["lens"], a["slots"], a["positions"], a["counts"], None)


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("other", INPUTS + OUTPUTS)
def test_shared_memory_is_refused(lib, out, other):
    """The same address, the other's last bytes, and the other's end over the
    beginning of this one."""
    if out == other:
        pytest.skip("an operand is itself")
    grain = 8 if out == "slots" or other == "slots" else 4
    last = -(-SIZES[other] // grain) * grain - grain
    for shift in (0, last, -(-(-SIZES[out] // grain) * grain - grain)):
        assert _call(lib, **{out: BASE[other] + shift}) == 1, shift


def test_step_kept_in_place_is_refused(lib):
    """Last step's seq_lens as this step's context_lens, its counts[1] as taken,
    with the same outputs again."""
    assert _call(lib, context=BASE["lens"]) == 1
    assert _call(lib, taken=BASE["counts"] + 4) == 1


def test_every_row_of_the_table_counts(lib):
    for row in range(R):
        for col in (0, WIDTH - 1):
            assert _call(lib, taken=BASE["table"] + 4 * (row * LD + col)) == 1


def _attention(lib, T, Hq, ot, oh, D=64):
    ok = ctypes.c_void_p(0x10000)
    info = binding.KVCacheInfo(0x10000, 0x10000, 0x10000, 0x10000, 4, 16, 1, D, 0)
    # (max_new 0: nothing is queued where the strides are fine)
    return lib.i8_paged_attention(ok, Hq * D, D, T, Hq, ctypes.byref(info), ok, 4, 4, ok, ok, 2, 0, 0.1, ok, ot, oh, None,
                                  ok, 1 << 30, None)


def test_out_whose_rows_share_elements_is_refused(lib):
    """Every pair of strides, counted out on the host."""
    D = 64
    seen = {0: 0, 1: 0}
    for T in (1, 2, 3, 5):
        for Hq in (1, 2, 3, 4):
            for ot in range(0, 9 * D, 24):
                for oh in (0, 8, 56, 64, 72, 128, 136, 192, 200, 320):
                    starts = [t * ot + h * oh for t in range(T) for h in range(Hq)]
                    starts.sort()
                    shared = any(b - a < D for a, b in zip(starts, starts[1:]))
                    got = _attention(lib, T, Hq, ot, oh)
                    assert got == int(shared), (T, Hq, ot, oh)
                    seen[got] += 1
    assert min(seen.values()) > 100


def test_h_over_other_rows_of_the_inputs_is_refused(lib):
    """h beside x and the residual, counted out on the host by rows; refused
    exactly where row i of h shares memory with row j != i of an input."""
    K, far = 64, 1 << 30
    x0 = 0x100000

    def call(at, M, ldx, ldh, which):
        x, r = (x0, far) if which == "x" else (far, x0)
        return lib.i8_add_rmsnorm_quant_act_pertoken(ctypes.c_void_p(x), M, K, ldx if which == "x" else K, ctypes.c_void_p(r),
                                                     ldx if which == "r" else K, None, 1e-6, 0, ctypes.c_void_p(2 * far), K,
                                                     ctypes.c_void_p(3 * far), ctypes.c_void_p(at), ldh, None)

    refused = 0
    for M in (2, 3, 5):
        for ldx in (64, 72, 136, 200):
            for ldh in (64, 72, 136, 200):
                for shift in range(-6 * 200, 6 * 200, 40):
                    cross = any(abs(shift + i * ldh - j * ldx) < K for i in range(M) for j in range(M) if i != j)
                    if not cross:
                        continue                    # (it would be queued)
                    refused += 1
                    for which in "xr":
                        assert call(x0 + 2 * shift - (2 * shift) % 16, M, ldx, ldh, which) == 1, (M, ldx, ldh, shift)
    assert refused > 500
