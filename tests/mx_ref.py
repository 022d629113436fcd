"""Float64 definitions of the microscaled formats: codes, scales, their layout, and
the bounds the tests hold the kernels to.  Plain torch on whatever device the tensors
are on."""
from __future__ import annotations

import torch

F8, F4 = 0, 1
LEAD = {F8: 8, F4: 2}             # exponent of the format's largest power of two
MAX = {F8: 448.0, F4: 6.0}
MANT = {F8: 3, F4: 1}             # mantissa bits
LOW = {F8: -6, F4: 0}             # exponent of the smallest normal number


def up(v, m):
    return -(-v // m) * m


def pow2(e):
    """2^e in float64, exactly (torch.pow is off by an ulp on some devices)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def log2_floor(v):
    """floor(log2 v) of float64 v > 0, exactly."""
    return torch.frexp(v)[1].long() - 1


def values(fmt, device="cpu"):
    """The 256 or 16 values of the format by code (e4m3's NaNs as nan)."""
    bits = torch.arange(256 if fmt == F8 else 16, dtype=torch.float64, device=device)
    m = 2 ** MANT[fmt]
    half = len(bits) // 2
    mag = bits % half
    e, f = (mag // m), mag % m
    v = torch.where(e == 0, f / m * 2.0 ** LOW[fmt],
                    (1 + f / m) * pow2(e - 1 + LOW[fmt]))
    if fmt == F8:
        v = torch.where(mag == 127, float("nan"), v)
    return torch.where(bits >= half, -v, v)


def round_code(v, fmt):
    """Nearest value of the format, ties to even, ends at the largest; float64."""
    a = v.abs()
    step = pow2(log2_floor(a.clamp(min=2.0 ** LOW[fmt])) - MANT[fmt])
    q = torch.round(a / step) * step      # torch.round: half to even
    return torch.copysign(q.clamp(max=MAX[fmt]), v)


def quantize(x, fmt):
    """(values over their scales [rows][padded], scale bytes [rows][blocks]) of x."""
    rows, cols = x.shape
    v = torch.zeros((rows, up(cols, 128)), dtype=torch.float64, device=x.device)
    v[:, :cols] = x.double()
    v = v.view(rows, -1, 32)
    top = v.abs().amax(2)
    bad = ~torch.isfinite(v).all(2)
    e = log2_floor(torch.where(bad | (top == 0), 2.0 ** -127, top))
    byte = (e - LEAD[fmt] + 127).clamp(min=0)
    q = round_code(torch.where(bad.unsqueeze(2), 0.0, v) * pow2(127 - byte).unsqueeze(2), fmt)
    return q.view(rows, -1), torch.where(bad, 255, byte)


def to_tiles(byte, fill=0):
    rows, blocks = byte.shape
    p = torch.full((up(rows, 128), up(blocks, 4)), fill, dtype=torch.uint8, device=byte.device)
    p[:rows, :blocks] = byte.to(torch.uint8)
    return p.view(-1, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def from_tiles(scales, rows, cols):
    t = scales.view(up(rows, 128) // 128, up(cols, 128) // 128, 32, 4, 4)
    return t.permute(0, 3, 2, 1, 4).reshape(up(rows, 128), -1)[:rows].long()


def unpack(codes, rows, cols, fmt):
    """Code numbers [rows][padded]."""
    c = codes.view(rows, -1).long()
    if fmt == F8:
        return c
    return torch.stack((c & 15, c >> 4), 2).view(rows, -1)


def scale_of(byte):
    return torch.where(byte == 255, float("nan"), pow2(byte - 127))


def dequantize(codes, scales, rows, cols, fmt):
    q = values(fmt, codes.device)[unpack(codes, rows, cols, fmt)].view(rows, -1, 32)
    return (q * scale_of(from_tiles(scales, rows, cols)).unsqueeze(2)).view(rows, -1)[:, :cols]


def pack(q, fmt):
    """Values of the format -> codes (zero as +0)."""
    table = values(fmt, q.device)
    half = len(table) // 2
    mag = table[:half].nan_to_num(nan=1e9).contiguous()
    c = torch.searchsorted(mag, q.abs().contiguous()) + half * (q < 0)
    if fmt == F8:
        return c.to(torch.uint8)
    return (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8)


def random_mx(rows, cols, fmt, gen, device="cuda", std=1.0):
    """A microscaled matrix of normal values: (codes, scales, float64 values)."""
    x = torch.randn((rows, cols), device=device, generator=gen) * std
    q, byte = quantize(x, fmt)
    codes, scales = pack(q, fmt), to_tiles(byte, fill=255)
    return codes, scales, dequantize(codes.view(-1), scales, rows, cols, fmt)


def check_quantized(codes, scales, rows, cols, fmt, want, err, what):
    """A quantised matrix against float64 values known to within err: scales that one
    value within err of the block's largest magnitude has, codes within half a step
    (of the scale taken) of one value within err."""
    byte = from_tiles(scales, rows, cols)
    tiles = up(cols, 128)
    v = torch.zeros((rows, tiles), dtype=torch.float64, device=want.device)
    e = torch.zeros_like(v)
    v[:, :cols], e[:, :cols] = want, err
    v, e = v.view(rows, -1, 32), e.view(rows, -1, 32)

    def byte_of(m):
        return (log2_floor(m.clamp(min=2.0 ** -140)) - LEAD[fmt] + 127).clamp(min=0)

    lo, hi = byte_of((v.abs() - e).amax(2)), byte_of((v.abs() + e).amax(2))
    assert ((byte >= lo) & (byte <= hi)).all(), f"{what}: scale of no value near the largest"
    got = (values(fmt, codes.device)[unpack(codes, rows, cols, fmt)].view(rows, -1, 32)
           * scale_of(byte).unsqueeze(2))
    s = scale_of(byte).unsqueeze(2)
    a = (v.abs() + e) / s
    step = pow2(log2_floor(a.clamp(min=2.0 ** LOW[fmt])) - MANT[fmt])
    bound = torch.where(a > MAX[fmt], a - MAX[fmt], step / 2).maximum(step / 2) * s + e
    worst = ((got - v).abs() - bound).max().item()
    assert worst <= 0, f"{what}: {worst:.3e} over the bound"
    pad = unpack(codes, rows, cols, fmt)[:, cols:]
    assert (pad == 0).all(), f"{what}: padding"
