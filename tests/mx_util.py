"""A plain 64-bit implementation of the microscaled matrices (format in
include/ciera.h), on the CPU, and the inputs of their tests."""
import math

import torch

BLOCK = 32
TOP = {8: 448.0, 4: 6.0}
E4M3 = [(m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)]
E4M3[127] = math.nan
E4M3 += [-v for v in E4M3]
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E2M1 += [-v for v in E2M1]


def pitch(cols):
    return -(-cols // 128) * 128


def sections(bits, rows, cols):
    line = pitch(cols) * bits // 8
    at = -(-rows * line // 128) * 128
    return line, at, at + rows * pitch(cols) // BLOCK


def _nearest_code(bits, t):
    """Code of the value of the element type nearest to |t| (float64), ties to the even code; the sign on top."""
    grid = torch.tensor(E4M3[:127] if bits == 8 else E2M1[:8], dtype=torch.float64)
    a = t.abs()
    hi = torch.searchsorted(grid, a).clamp(max=grid.numel() - 1)
    lo = (hi - 1).clamp(min=0)
    dh, dl = grid[hi] - a, a - grid[lo]
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = torch.where(up, hi, lo)
    return code + (128 if bits == 8 else 8) * torch.signbit(t).long()


def encode(bits, x):
    """The encoded bytes of the BF16 matrix x (a CPU tensor)."""
    rows, cols = x.shape
    kp = pitch(cols)
    v = torch.zeros(rows, kp, dtype=torch.float64)
    v[:, :cols] = x.double()
    v = v.view(rows, kp // BLOCK, BLOCK)
    amax = v.abs().amax(2)
    bad = ~torch.isfinite(amax)
    m, p = torch.frexp(torch.where(bad, torch.zeros_like(amax), amax))
    mt, pt = math.frexp(TOP[bits])
    e = torch.where(amax > 0, p - pt + (m > mt), torch.full_like(p, -126)).clamp(min=-126)
    v = torch.where(bad[:, :, None], torch.zeros_like(v), v)
    code = _nearest_code(bits, v / torch.ldexp(torch.ones_like(amax), e)[:, :, None]).view(rows, kp)
    if bits == 4:
        code = code[:, 0::2] | (code[:, 1::2] << 4)
    line, at, size = sections(bits, rows, cols)
    out = torch.zeros(size, dtype=torch.uint8)
    out[:rows * line] = code.to(torch.uint8).reshape(-1)
    out[at:] = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8).reshape(-1)
    return out


def decode(bits, buf, rows, cols):
    """What the encoded bytes stand for, in float64."""
    line, at, size = sections(bits, rows, cols)
    q = buf[:rows * line].view(rows, line).long()
    if bits == 4:
        q = torch.stack((q & 15, q >> 4), 2).view(rows, -1)
    v = torch.tensor(E4M3 if bits == 8 else E2M1, dtype=torch.float64)[q].view(rows, -1, BLOCK)
    b = buf[at:size].view(rows, -1).long()
    s = torch.ldexp(torch.ones(b.shape, dtype=torch.float64), b - 127)
    s[b == 255] = math.nan
    return (v * s[:, :, None]).view(rows, -1)[:, :cols]


def activations(gen, rows, cols, std=1.0):
    x = torch.randn(rows, cols, generator=gen) * std
    x[:, torch.rand(cols, generator=gen) < 0.02] *= 16
    return x.to(torch.bfloat16)


def split(gen, tokens, groups, empty=0.3, lead=0, tail=0):
    """offsets of `groups` groups over tokens rows, about a share `empty` of them without rows."""
    live = (torch.rand(groups, generator=gen) >= empty).double()
    if not live.any():
        live[-1] = 1.0
    rows = tokens - lead - tail
    cuts = torch.cumsum(live * torch.rand(groups, generator=gen, dtype=torch.float64), 0)
    cuts = (cuts / cuts[-1] * rows).round().long() if cuts[-1] > 0 else cuts.long()
    return torch.cat((torch.zeros(1, dtype=torch.int64), cuts)) + lead


def bounds(offsets, tokens):
    return [(0, tokens)] if offsets is None else list(zip(offsets.tolist()[:-1], offsets.tolist()[1:]))
