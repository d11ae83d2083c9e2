"""Plain 64-bit forms of the checkpoints in 8 bits and of the gated feed-forward block, and the error
bounds of their tests. No library code.

fp32's exp and division as the kernels use them: the relative error of __expf(z) is at most
(2 + 1.173 |z|) units of 2^-23, that of __fdividef two of them (the CUDA programming guide's table of
intrinsic functions). z itself is computed with at most 8 roundings of 2^-24, so it is off by at
most 4 |z| 2^-23, which exp turns into a relative error."""
from __future__ import annotations

import math

import torch

GROUP = 16
ULP = 2.0 ** -23


def quantised(x: torch.Tensor):
    """x [rows][features] bf16 -> (e4m3 bytes, exponent bytes, the values they stand for in 64 bits), group by
    group by search: the least k with amax <= 448 * 2^k, the nearest of the 127 magnitudes of e4m3
    (to even where two are as near)."""
    rows, features = x.shape
    groups = -(-features // GROUP)
    at = torch.zeros(rows, groups * GROUP, dtype=torch.float64)
    at[:, :features] = x.cpu().double()
    at = at.view(rows, groups, GROUP)
    finite = torch.where(torch.isnan(at), torch.zeros_like(at), at.abs())
    most = finite.amax(2)
    k = torch.full_like(most, -126)
    for e in range(-126, 121):
        k = torch.where((most > 448.0 * 2.0 ** e) & (k == e), torch.full_like(k, e + 1), k)
    k = k.clamp(max=120)                                               # an infinity
    table = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    scaled = at.abs() / torch.exp2(k).unsqueeze(2)
    high = torch.searchsorted(table, scaled.clamp(max=448.0).nan_to_num(0.0)).clamp(max=126)
    low = (high - 1).clamp(min=0)
    up, down = table[high] - scaled, scaled - table[low]
    code = torch.where((down < up) | ((down == up) & (low % 2 == 0)), low, high)
    code = torch.where(torch.isinf(at), torch.full_like(code, 126), code)
    value = table[code] * torch.exp2(k).unsqueeze(2)
    value = torch.where(value >= 2.0 ** 128, torch.full_like(value, math.inf), value)       # 448 * 2^120 and 256 * 2^120
    nan = torch.isnan(at)
    code, value = torch.where(nan, torch.full_like(code, 127), code), torch.where(nan, at, value)
    sign = torch.signbit(at)
    code, value = code + 128 * (sign & ~nan), torch.where(sign, -value, value)
    return (code.flatten(1).to(torch.uint8), (k + 127).to(torch.uint8), value.flatten(1)[:, :features])


def stands_for(values: torch.Tensor, scales: torch.Tensor, features: int) -> torch.Tensor:
    """The values of one part of a checkpoint, in 64 bits."""
    v = values.view(torch.float8_e4m3fn).double().unflatten(1, (-1, GROUP))
    return (v * torch.exp2(scales.double() - 127).unsqueeze(2)).flatten(1)[:, :features]


def act(g: torch.Tensor, kind: str):
    """act(g), act'(g), and bounds of what fp32 does to both, in 64 bits."""
    if kind == "silu":
        z, dz = g, torch.ones_like(g)
    else:
        c = 2 * math.sqrt(2 / math.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g * g)
    s = torch.sigmoid(z)
    off = ((2 + 6 * z.abs()) * torch.sigmoid(-z) + 4) * ULP               # of s, relatively
    value, slope = g * s, s + g * s * torch.sigmoid(-z) * dz
    # slope: s and 1 - s are off by off * s; five more roundings of each term
    slope_off = s * (off + 3 * ULP) + g.abs() * dz * s * (torch.sigmoid(-z) * (off + 4 * ULP) + off * s + ULP)
    # and below 2^-126, where fp32 has no more normal numbers (and __fdividef by more than 2^126 gives 0), s
    # may be 0
    tiny = 2.0 ** -125
    return value, slope, value.abs() * (off + ULP) + g.abs() * tiny, slope_off + (1 + g.abs() * dz) * tiny
