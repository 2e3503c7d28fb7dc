"""Plain forms of 4-bit rows and of rotation, for the tests of paged caches: the byte order of the pages, the values that codes
and scales stand for, and the intervals in which codes and scales may lie when the value they come from is off by a
given amount (both are monotone in it, so no tolerance on codes is needed)."""
from __future__ import annotations

import torch

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# every positive E4M3 value, ascending: byte i + 1 holds SCALES[i]
SCALES = torch.tensor([((1 + (i & 7) / 8) * 2.0 ** ((i >> 3) - 7)) if i >> 3 else (i & 7) * 2.0 ** -9 for i in range(1, 0x7F)],
                      dtype=torch.float64)


def order(dim, keys):
    """place[b]: where byte b of a row (dims 2 b, 2 b + 1) is stored."""
    n = dim // 16
    place = [0] * (8 * n)
    for s in range(n):
        for t in range(4):
            for i in range(2):
                place[8 * s + 2 * t + i] = 2 * n * t + 2 * s + i
    return torch.tensor(place if keys else [n * (b % 8) + b // 8 for b in range(8 * n)])


def unpack(pool, scales, keys):
    """Values [...][dim] in 64 bits of bytes [...][dim / 2] and scale bytes [...][dim / 16]."""
    b = pool[..., order(2 * pool.shape[-1], keys).to(pool.device)].long()
    c = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    x = LEVELS.to(pool.device)[c & 7] * (1 - 2 * (c >> 3)).double()
    s = scales.view(torch.float8_e4m3fn).double() if scales.dtype is torch.uint8 else scales.double()
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def codes(pool, keys):
    """Signed level numbers [...][dim] of bytes [...][dim / 2]; no byte holds -0."""
    b = pool[..., order(2 * pool.shape[-1], keys).to(pool.device)].long()
    c = torch.stack((b & 15, b >> 4), -1).flatten(-2)
    assert not (c == 8).any(), "-0 is stored as 0"
    return (c & 7) * (1 - 2 * (c >> 3))


def code_of(y):
    """Signed level number of the E2M1 value nearest to y (ties to the even one, saturating)."""
    a, n = y.abs(), torch.zeros(y.shape, dtype=torch.long, device=y.device)
    levels = LEVELS.to(y.device)
    for i in range(7):
        mid = (levels[i] + levels[i + 1]) / 2
        n += (a > mid) | ((a == mid) & (i % 2 == 1))
    return torch.where(y < 0, -n, n)


def scale_of(amax):
    """Byte of the smallest positive E4M3 value s with 6 s >= amax, or of 448."""
    s = (6 * SCALES).to(amax.device)
    return torch.searchsorted(s, amax.contiguous()).clamp(max=len(SCALES) - 1) + 1


def check_group(pool, scales, y, off, keys):
    """Rows of bytes and scale bytes hold the values y [...][dim] (64 bits), each off by at most `off`."""
    amax = y.unflatten(-1, (-1, 16)).abs().amax(-1)
    most = off.unflatten(-1, (-1, 16)).amax(-1)
    got = scales.long()
    lo, hi = scale_of((amax - most).clamp(min=0)), scale_of(amax + most)
    assert ((lo <= got) & (got <= hi)).all(), "a scale is not the smallest that holds its group"
    s = SCALES.to(y.device)[got - 1].repeat_interleave(16, -1)
    c = codes(pool, keys)
    assert ((code_of((y - off) / s) <= c) & (c <= code_of((y + off) / s))).all(), "a code is not the nearest"


def pack(x, keys):
    """Values [...][dim] -> (bytes [...][dim / 2], scale bytes [...][dim / 16])."""
    y = x.double()
    byte = scale_of(y.unflatten(-1, (-1, 16)).abs().amax(-1))
    c = code_of(y / SCALES.to(y.device)[byte - 1].repeat_interleave(16, -1))
    n = torch.where(c < 0, 8 - c, c)
    b = (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)
    out = torch.empty_like(b)
    out[..., order(x.shape[-1], keys).to(x.device)] = b
    return out, byte.to(torch.uint8)


def rotate(x, pos, inv_freq, at, halves):
    """x [n][heads][dim] in 64 bits, pos [n], inv_freq [R / 2] -> rotated, and |x| + |y| of each element's pair (0: not turned)."""
    x, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    r = 2 * inv_freq.shape[0]
    angle = (pos.double()[:, None] * inv_freq.double())[:, None]
    c, s = torch.cos(angle), torch.sin(angle)
    i = (slice(at, at + r // 2), slice(at + r // 2, at + r)) if halves else (slice(at, at + r, 2), slice(at + 1, at + r, 2))
    a, b = x[..., i[0]].clone(), x[..., i[1]].clone()
    x[..., i[0]], x[..., i[1]] = a * c - b * s, a * s + b * c
    size[..., i[0]] = size[..., i[1]] = a.abs() + b.abs()
    return x, size
