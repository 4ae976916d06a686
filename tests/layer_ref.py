"""The layer operators in 64 bits, from their definitions, on the CPU (torch
float64 and integer bits only; none of the package's code)."""
from __future__ import annotations

import torch

F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
U24 = 2.0 ** -24  # half a step of float32, relative


def half_step(dtype):
    return {torch.bfloat16: 2.0 ** -8, torch.float32: U24}[dtype]


def f64(t):
    return t.detach().cpu().double()


def byte(t):
    return t.detach().cpu().view(torch.uint8).long()


# ------------------------------------------------------------------- mx8

E4M3 = torch.tensor([float("nan") if c & 127 == 127 else
                     (-1.0) ** (c >> 7) * ((c & 7) * 2.0 ** -9 if not c >> 3 & 15 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3 & 15) - 7))
                     for c in range(256)], dtype=torch.float64)


def group_amax(v):
    """Largest finite magnitude of each group of 32, [T, ceil(K / 32)]."""
    T, K = v.shape
    p = torch.zeros(T, (K + 31) // 32 * 32, dtype=torch.float64)
    p[:, :K] = torch.where(torch.isfinite(v), v.abs(), 0.0)
    return p.view(T, -1, 32).amax(-1) if K else p.view(T, 0)


def mx8_exponent(a):
    """Smallest s >= -117 with a <= 448 * 2^s."""
    s = torch.full_like(a, -117)
    while True:
        more = a > 448 * torch.exp2(s)
        if not more.any():
            return s
        s = torch.where(more, s + 1, s)


def mx8_codes(v):
    """float64 rows -> (code bytes, scale bytes); ties to even, not finite -> NaN."""
    s = mx8_exponent(group_amax(v))
    q = v / torch.exp2(s).repeat_interleave(32, 1)[:, :v.shape[1]]
    a = q.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    r = torch.round(a / step) * step
    grid = E4M3[:127]
    code = torch.searchsorted(grid, torch.where(torch.isfinite(r), r, 0.0)).long()
    code = torch.where(torch.isfinite(v), code | (torch.signbit(v).long() << 7), 127)
    return code, (s + 127).long()


def mx8_values(codes, scales):
    """Code and scale bytes -> float64."""
    K = codes.shape[1]
    return E4M3[codes] * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)[:, :K]


def assert_mx8(codes, scales, v, rel, what):
    """codes, scales stand for float64 v, whose float32 form is off by up to
    rel, relative: scales are the exact ones unless the group's maximum is
    that near a border; values are off by half a step (2^-4 of the value, or
    half the smallest step under the scale) and rel."""
    c, s = byte(codes), byte(scales)
    a = group_amax(v)
    lo, hi = mx8_exponent(a * (1 - rel)) + 127, mx8_exponent(a * (1 + rel)) + 127
    assert ((s >= lo) & (s <= hi)).all(), f"{what}: scale bytes"
    got = mx8_values(c, s)
    fine = torch.isfinite(v)
    assert torch.equal(torch.isnan(got), ~fine), f"{what}: NaN codes"
    tiny = torch.exp2(s.double() - 127).repeat_interleave(32, 1)[:, :v.shape[1]] * 2.0 ** -10
    off = (got - v).abs()[fine]
    most = (v.abs() * (2.0 ** -4 + 2 * rel) + tiny)[fine]
    assert (off <= most).all(), f"{what}: values off by {(off / most).max()} of what they may be"


# ---------------------------------------------------------- 4-bit weights

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def weight_values(packed, scale, blocks, amax=None, bound=448.0):
    """float64 [E, N, K]; blocks "1x16", "16x16" or "16x16t"; amax [E] or [E * N]."""
    p, b = packed.detach().cpu().long(), byte(scale)
    v = E2M1[torch.stack((p & 15, p >> 4), -1)].flatten(-2)
    s = E4M3[b]
    if blocks == "16x16t":
        s = s.transpose(-1, -2)
    if blocks != "1x16":
        s = s.repeat_interleave(16, -2)
    v = v * s.repeat_interleave(16, -1)
    if amax is not None:
        v = v * (f64(amax) / (6 * bound)).view(v.shape[0], -1, 1)
    return v


def cuts(ends, T):
    """Row ranges of the experts, clamped and never decreasing."""
    got, at = [0], 0
    for e in ends.detach().cpu().tolist():
        at = max(at, min(max(e, 0), T))
        got.append(at)
    return got


def assert_near(got, want, most, what):
    g = f64(got)
    same = (g == want) | (torch.isnan(g) & torch.isnan(want))
    off = torch.where(same, 0.0, (g - want).abs())
    bad = ~(off <= most) & ~same
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / most)[bad].max())} of what they may be"


def product_bound(x, w, out_dtype, y):
    """One rounding to the output's type, and fp32 sums of K exact products in
    any order: K - 1 additions (and the second-level scale's division and
    product), each off by up to one unit 2^-23 of the sum of magnitudes (a
    matrix core may cut instead of rounding)."""
    K = x.shape[1]
    return y.abs() * half_step(out_dtype) + (K + 8) * 2.0 ** -23 * (x.abs() @ w.abs().transpose(-1, -2))


# ------------------------------------------------------------- gradients

def norm_gradient(dy, hidden, w, rstd, dhidden):
    """(dx, dweight) in float64."""
    n, d = hidden * rstd[:, None], dy * w
    dx = rstd[:, None] * (d - n * (d * n).mean(1, keepdim=True))
    return dx if dhidden is None else dx + dhidden, (dy * n).sum(0)


def swiglu_gradient(dout, g, u):
    s = 1 / (1 + torch.exp(-g))
    return dout * u * s * (1 + g * (1 - s)), dout * g * s
