"""The 4-bit formats by their definition, in 64 bits, and their layout: what the
tests of the 4-bit route compare with.  Tensors may be on any device."""
import torch

BLOCK = {"nvfp4": 16, "mxfp4": 32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def unpack(codes):
    """uint8 [rows, K / 2] -> the codes' values, fp64 [rows, K]."""
    nibbles = torch.stack((codes & 15, codes >> 4), 2).flatten(1).long()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    return table[nibbles]


def untile(block_scales, rows, K, fmt):
    """The block scales' bytes, uint8 [rows, ceil(K / 256) * 256 / block]."""
    per = 256 // BLOCK[fmt]
    tiles, deep, size = block_scales.shape
    assert size == 128 * per
    flat = block_scales.view(tiles, deep, per // 4, 32, 4, 4).permute(0, 4, 3, 1, 2, 5)
    return flat.reshape(tiles * 128, deep * per)[:rows]


def tile(scales, fmt):
    """uint8 [rows, K / block] -> the library's tiles."""
    per = 256 // BLOCK[fmt]
    rows, groups = scales.shape
    tiles, deep = -(-rows // 128), -(-groups // per)
    full = torch.zeros(tiles * 128, deep * per, dtype=torch.uint8, device=scales.device)
    full[:rows, :groups] = scales
    return full.view(tiles, 4, 32, deep, per // 4, 4).permute(0, 3, 4, 2, 1, 5).reshape(tiles, deep, 128 * per).contiguous()


def scale_values(scales, fmt):
    if fmt == "nvfp4":
        return scales.view(torch.float8_e4m3fn).double()
    return torch.where(scales == 255, torch.nan, torch.exp2(scales.double() - 127))


def values(rows, row_scales=True):
    """FP4Rows -> fp64 [rows, K]."""
    n, K = rows.shape
    fmt = rows.fmt
    s = scale_values(untile(rows.block_scales, n, K, fmt)[:, : K // BLOCK[fmt]].contiguous(), fmt)
    v = unpack(rows.codes) * s.repeat_interleave(BLOCK[fmt], 1)
    if row_scales and rows.row_scales is not None:
        v = v * rows.row_scales.double()[:, None]
    return v


def _e2m1(x):
    """Nibbles of the nearest values, ties to the even code."""
    middle = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=x.device)
    a = x.abs()
    low = torch.bucketize(a, middle)                    # how many midpoints lie below
    high = torch.bucketize(a, middle, right=True)       # below or at it
    code = torch.where((low != high) & (low % 2 == 1), high, low)
    return (code + 8 * torch.signbit(x).long()).to(torch.uint8)


def _e4m3(x):
    """Codes of the nearest E4M3 values to x >= 0 (fp64), ties to the even code."""
    table = torch.arange(127, dtype=torch.uint8, device=x.device).view(torch.float8_e4m3fn).double()
    middle = (table[1:] + table[:-1]) / 2
    low, high = torch.bucketize(x, middle), torch.bucketize(x, middle, right=True)
    return torch.where((low != high) & (low % 2 == 1), high, low).to(torch.uint8)


def _power_above(x):
    """The exponent of the smallest power of two that is at least x (log2 alone may
    be off in its last digit)."""
    k = torch.floor(torch.log2(x)) - 1
    for _ in range(3):
        k = torch.where(torch.exp2(k) < x, k + 1, k)
    return k


def quantize(t, fmt):
    """fp64 rows -> (codes uint8 [rows, K / 2], block scales uint8 [rows, K / block],
    row scales fp64 [rows]); every step from its definition, finite rows."""
    rows, K = t.shape
    blocks = t.reshape(rows, -1, BLOCK[fmt])
    most = blocks.abs().amax(2)
    if fmt == "nvfp4":
        row = most.amax(1)
        s = torch.where(row > 0, torch.exp2(_power_above(row / 2688).clamp(min=-126)), 0.0)
        over = torch.where(s > 0, s, 1.0)[:, None]
        scales = _e4m3(most / over / 6)
        S = scale_values(scales, fmt) * over
    else:
        s = torch.ones_like(most[:, 0])
        E = _power_above(most / 6).clamp(min=-127)
        scales = (E + 127).to(torch.uint8)
        S = torch.exp2(E)
    q = torch.where(S[:, :, None] > 0, blocks / torch.where(S > 0, S, 1.0)[:, :, None], 0.0)
    nibbles = _e2m1(q)
    if fmt == "nvfp4":
        nibbles = torch.where(S[:, :, None] > 0, nibbles, torch.zeros_like(nibbles))
    nibbles = nibbles.reshape(rows, K)
    return nibbles[:, 0::2] | (nibbles[:, 1::2] << 4), scales, s
