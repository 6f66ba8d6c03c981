"""paged_attention where values lie far apart, are NaN, or lengths leave the
table: against the definition in 64 bits, in which a row depends on the tokens
that it sees and on nothing else."""
import random

import pytest
import torch

import w8a8_int8_quantized_i8_gb300 as i8
from tests import _serving as ref

pytestmark = pytest.mark.gpu

# one token a request (a row or two a kv head, and 16 rows), and chunks on tcgen05
FORMS = [pytest.param(1, 2, 2, 64, id="step64"), pytest.param(1, 8, 2, 128, id="step128"),
         pytest.param(4, 8, 2, 128, id="rows16"), pytest.param(1, 4, 1, 256, id="step256"),
         pytest.param(120, 2, 2, 64, id="chunk64"), pytest.param(130, 4, 2, 128, id="chunk128")]


class Case:
    """Requests over a shuffled pool, values of any kind set by the test."""

    def __init__(self, lens, news, block, Hq, Hkv, D, fmt, seed, width=None):
        g, rng = torch.Generator().manual_seed(seed), random.Random(seed)
        need = [-(-n // block) for n in lens]
        P, ids = sum(need) + 2, list(range(sum(need) + 2))
        rng.shuffle(ids)
        self.table = [[ids.pop() for _ in range(n)] + [-1] * (max(need) - n) for n in need]
        if width is not None:
            self.table = [row[:width] for row in self.table]
        self.lens, self.fmt, self.block = lens, fmt, block
        self.cu = [0]
        for n in news:
            self.cu.append(self.cu[-1] + n)
        self.q = torch.randn(self.cu[-1], Hq, D, generator=g).bfloat16()
        self.limit = int(ref.LIMIT[fmt])
        x = torch.randn(2, P, Hkv, block, D, generator=g) * self.limit / 5
        x = x.clamp(-self.limit, self.limit)
        self.codes = [c.round().to(torch.int8) if fmt == "int8" else c.to(torch.float8_e4m3fn) for c in x]
        self.scales = [torch.full((P, Hkv), 0.02 * 127 / self.limit) for _ in range(2)]

    def bits(self, side):
        return self.codes[side].view(torch.uint8)

    def run(self, status=0, **kw):
        cache = i8.QuantKVCache(*(c.view(torch.uint8).cuda().view(c.dtype) for c in self.codes),
                                *(s.cuda() for s in self.scales))
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        r = i8.paged_attention(self.q.cuda(), cache, i32(self.table), i32(self.lens), i32(self.cu), want_lse=True, **kw)
        if status:
            with pytest.raises(i8.I8Error) as e:
                i8.sync_check()
            assert e.value.status == status
        else:
            i8.sync_check()
        return r

    def want(self, scale=None):
        D = self.q.shape[2]
        k, v = (c.view(torch.uint8).cuda().view(c.dtype).float().double() for c in self.codes)
        return ref.attention_definition(self.q.cuda(), k, v, self.scales[0].cuda(), self.scales[1].cuda(), self.table,
                                        self.lens, self.cu, D ** -0.5 if scale is None else scale, float(self.limit))

    def check(self, status=0, **kw):
        ref.check_attention(*self.run(status), self.want(**kw))


# ------------------------------------------------------------------ lengths past the table
@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
def test_sequence_longer_than_its_table(new, Hq, Hkv, D):
    """The tokens past the table are absent, the others stay where they are: the
    rows' positions are the sequence's, and sync_check says that it was cut."""
    lens = [400, 333, 500]
    c = Case(lens, [min(new, 100)] * 3, 16, Hq, Hkv, D, "int8", 1, width=21)   # 336 tokens of 400 and 500
    c.check(status=7)


def test_table_that_ran_out_of_width():
    """What build_block_tables gives where the width runs out: the rows whose
    own tokens have a block see exactly what they would in a wide table."""
    c = Case([200], [150], 16, 4, 2, 128, "int8", 2)
    want, _, bound, _ = c.want()
    c.table = [c.table[0][:8]]                           # 128 tokens: the rows of positions 50..127
    cut, _ = c.run(status=7)
    assert ((cut.double() - want).abs() <= bound)[:78].all()


# ------------------------------------------------------------------ V's scales far apart
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("far", [1e-18, 1e-30, 3e-36, 1e-37, 1e-41])
@pytest.mark.parametrize("order", ["small_first", "large_first", "between"])
@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
def test_values_far_apart(new, Hq, Hkv, D, order, far, fmt):
    """Blocks whose values differ by up to 10^41: the sum of exponentials counts
    all of them."""
    c = Case([400, 40 + new], [new, new], 16, Hq, Hkv, D, fmt, 3)
    for row in c.table:
        ids = [b for b in row if b >= 0]
        small = {"small_first": ids[: len(ids) // 2], "large_first": ids[len(ids) // 2:], "between": ids[1::2]}[order]
        for b in small:
            c.scales[1][b] *= far
    c.check()


@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
@pytest.mark.parametrize("exponent", [20, 39, 40, 41, 80])
def test_values_on_both_sides_of_the_first_block(new, Hq, Hkv, D, exponent):
    """The first block's values between those of the others, around the distance
    (2^40) at which the sum changes its form."""
    c = Case([400, 40 + new], [new, new], 16, Hq, Hkv, D, "int8", 15)
    for row in c.table:
        for i, b in enumerate(b for b in row if b >= 0):
            c.scales[1][b] *= (1.0, 2.0 ** exponent, 2.0 ** -exponent, 1.0)[i % 4]
    c.check()


@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
@pytest.mark.parametrize("loud", [0, 1])
def test_the_attended_block_is_the_quiet_one(new, Hq, Hkv, D, loud):
    """All of a row's weight lies on tokens whose values are 10^36 times smaller
    than the others': the row's result is those values."""
    c = Case([160 + new], [new], 16, Hq, Hkv, D, "int8", 4)
    ids = [b for b in c.table[0] if b >= 0][: 10]
    c.q = c.q.abs()
    for i, b in enumerate(ids):
        quiet = (i >= 5) == bool(loud)
        c.codes[0][b] = 120 if quiet else -120
        if quiet:
            c.scales[1][b] *= 1e-36
    for b in c.table[0][10:]:
        c.codes[0][b] = -120
    c.scales[0][:] = 0.5
    c.check()


@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
def test_blocks_of_zeros_everywhere(new, Hq, Hkv, D):
    """Values that are all zero, in some blocks and in every block of a
    request: 0, and the sum of exponentials of all tokens."""
    c = Case([150 + new, 90 + new], [new, new], 16, Hq, Hkv, D, "int8", 5)
    for i, b in enumerate(c.table[0]):
        if i % 3 != 1:
            c.scales[1][b] = 0.0
            c.codes[1][b] = 0
    for b in c.table[1]:
        if b >= 0:
            c.scales[1][b] = 0.0
            c.codes[1][b] = 0
    c.check()


# ------------------------------------------------------------------ NaN
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
def test_nan_in_a_row_of_q(new, Hq, Hkv, D, fmt):
    """The row's result is NaN; no other row's is; a row that sees nothing gives
    0 and -inf all the same."""
    c = Case([300, 64, 2], [new, new, new], 16, Hq, Hkv, D, fmt, 6)
    for t in (0, new, 2 * new + new // 2):
        c.q[t, Hq - 1, D // 2] = float("nan")
    c.q[2 * new, 0, 3] = float("nan")
    c.check()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
def test_nan_scales(new, Hq, Hkv, D, side, fmt):
    """A block with a NaN scale spoils the rows that see one of its tokens."""
    c = Case([300, 80 + new, 16 * 7], [new, new, min(new, 112)], 16, Hq, Hkv, D, fmt, 7)
    c.scales[side][c.table[0][3], Hkv - 1] = float("nan")
    c.scales[side][c.table[1][(80 + new - 1) // 16], 0] = float("nan")     # the last block
    c.check()


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
def test_nan_codes(new, Hq, Hkv, D, side):
    """NaN codes of E4M3 in tokens: rows that see the token are NaN (a value's
    in its head dimension), the rows before it are not; places past the end and
    of blocks that are missing may hold anything."""
    c = Case([300, 80 + new, 250 + new], [new, new, new], 16, Hq, Hkv, D, "e4m3", 8)
    bits = c.bits(side)
    bits[c.table[0][2], Hkv - 1, 5, 7] = 0x7F                              # an old token
    last = 80 + new - 1
    bits[c.table[1][last // 16], 0, last % 16, D - 1] = 0xFF               # the newest token
    if new > 2:
        t = 250 + new // 2                                                 # a new token in the middle
        bits[c.table[2][t // 16], 0, t % 16, 1] = 0x7F
        bits[c.table[2][(t + 3) // 16], Hkv - 1, (t + 3) % 16, D // 2] = 0x7F
    for r, n in enumerate(c.lens):                                         # no token's places
        if n % 16:
            c.codes[0].view(torch.uint8)[c.table[r][n // 16], :, n % 16:] = 0x7F
            c.codes[1].view(torch.uint8)[c.table[r][n // 16], :, n % 16:] = 0xFF
    c.check()


@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
def test_nan_codes_and_missing_blocks(new, Hq, Hkv, D):
    c = Case([300, 260], [new, new], 16, Hq, Hkv, D, "e4m3", 9)
    c.bits(1)[c.table[0][1], 0, 3, 2] = 0x7F
    c.bits(0)[c.table[1][0], 0, 3, 2] = 0x7F
    c.table[0][4], c.table[0][5], c.table[1][9] = -1, 10 ** 6, -5
    c.check(status=7)


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
def test_infinite_scales_do_not_vanish(new, Hq, Hkv, D, side):
    """A block with an infinite scale: rows that see it are not finite, the
    others' are those of the definition."""
    c = Case([300, 80 + new], [new, new], 16, Hq, Hkv, D, "int8", 10)
    c.scales[side][c.table[0][3], Hkv - 1] = float("inf")
    out, lse = c.run()
    group = Hq // Hkv
    assert not torch.isfinite(out[:new, (Hkv - 1) * group:].float()).any()
    c.scales[side][c.table[0][3], Hkv - 1] = 1.0
    o, l, bound, lse_bound = c.want()
    rest = torch.ones(out.shape[:2], dtype=torch.bool, device="cuda")
    rest[:new, (Hkv - 1) * group:] = False
    assert ((out.double() - o).abs() <= bound)[rest].all()
    assert ((lse.double() - l).abs() <= lse_bound)[rest].all()


# ------------------------------------------------------------------ many requests, and what is left out
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("R", [129, 300, 1000])
def test_many_requests(R, D):
    """Ragged batches of more requests than a CTA has threads for, some empty:
    every thread walks over several of them."""
    rng = random.Random(R)
    lens = [rng.choice([0, 1, 5, 16, 17, 40]) for _ in range(R)]
    news = [min(n, rng.choice([0, 1, 1, 1, 2])) for n in lens]
    Case(lens, news, 16, 4, 2, D, "int8", 11).check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("R", [129, 300, 1000])
def test_many_requests_a_few_with_many_rows(R, D):
    rng = random.Random(R + 1)
    lens = [rng.choice([0, 1, 16, 17, 30]) for _ in range(R)]
    news = [min(n, rng.choice([0, 1, 1])) for n in lens]
    for at in (0, R // 3, R // 2, R - 1):
        lens[at], news[at] = 70 + at % 50, 60 + at % 7
    Case(lens, news, 16, 4, 2, D, "int8", 12).check()


@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
def test_left_out_requests_are_not_written(new, Hq, Hkv, D):
    """Offsets past q or before it: that request's rows keep what was there, its
    neighbour's are right."""
    c = Case([150, 140], [new, new], 16, Hq, Hkv, D, "int8", 13)
    want = c.want()
    for cu, kept in (([0, new, 2 * new + 1], 0), ([-1, new, 2 * new], 1)):
        good = Case([150, 140], [new, new], 16, Hq, Hkv, D, "int8", 13)
        good.cu = cu
        out = torch.full((2 * new, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
        good.run(status=7, out=out, max_new=new)
        rows = [slice(0, new), slice(new, 2 * new)]
        for r in range(2):
            if r == kept:
                err = (out[rows[r]].double() - want[0][rows[r]]).abs()
                assert (err <= want[2][rows[r]]).all()
            else:
                assert (out[rows[r]] == 7).all()


@pytest.mark.parametrize("new,Hq,Hkv,D", FORMS)
def test_offsets_that_go_back_are_reported(new, Hq, Hkv, D):
    c = Case([150, 140], [new, new], 16, Hq, Hkv, D, "int8", 13)
    c.cu = [2 * new, 0, new]                             # the first request has a negative count
    out = torch.full((2 * new, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    c.lens = [150, 0]                                    # and the second sees nothing
    c.run(status=7, out=out, max_new=new)
    assert (out[:new] == 0).all() and (out[new:] == 7).all()


def test_workspace_of_another_type_is_refused():
    c = Case([40], [1], 16, 2, 1, 64, "int8", 16)
    for bad, error in ((1 << 20, TypeError), (torch.empty(1 << 20, dtype=torch.uint8), ValueError),
                       (torch.empty(1 << 20, 2, dtype=torch.uint8, device="cuda")[:, 0], ValueError)):
        with pytest.raises(error):
            c.run(workspace=bad)


def test_repeats_itself_exactly():
    for new, Hq, Hkv, D in ((1, 8, 2, 128), (4, 8, 2, 128), (130, 4, 2, 128)):
        c = Case([3000, 700, 150], [new] * 3, 16, Hq, Hkv, D, "int8", 14)
        a, la = c.run()
        for _ in range(4):
            b, lb = c.run()
            assert torch.equal(a, b) and torch.equal(la, lb)
