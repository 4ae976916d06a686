"""Attention on an NVFP4 cache in 64 bits, from its definitions, on the CPU (torch
float64 and integer bits; none of the package's code)."""
from __future__ import annotations

import math

import torch

from tests.layer_ref import E2M1, E4M3, byte, f64


def rotate(y, positions, freqs, interleaved, multiplier=1.0, back=False):
    """y [T, H, D] in 64 bits: pairs turned by positions * freqs."""
    y, R = y.clone(), 2 * len(freqs)
    if R == 0:
        return y
    angle = positions.double()[:, None] * freqs
    c, s = multiplier * torch.cos(angle)[:, None], multiplier * torch.sin(angle)[:, None] * (-1 if back else 1)
    at = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = y[..., at[0]].clone(), y[..., at[1]].clone()
    y[..., at[0]], y[..., at[1]] = a * c - b * s, b * c + a * s
    return y


def norm_rope(x, w, positions, freqs, interleaved=False, multiplier=1.0, eps=1e-6):
    y = f64(x)
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * f64(w)
    return rotate(y, positions, freqs, interleaved, multiplier)


def norm_rope_gradient(dz, x, w, positions, freqs, interleaved=False, multiplier=1.0, eps=1e-6):
    """(dx, dw or None, the magnitudes that dx's terms have, those of dw's)."""
    dy, x = rotate(f64(dz), positions, freqs, interleaved, multiplier, back=True), f64(x)
    if w is None:
        return dy, None, dy.abs(), None
    rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n, d = x * rstd, dy * f64(w)
    dx = rstd * (d - n * (d * n).mean(-1, keepdim=True))
    return dx, (dy * n).sum((0, 1)), rstd * (d.abs() + n.abs() * (d * n).abs().mean(-1, keepdim=True)), (dy * n).abs().sum((0, 1))


def cache_values(codes, scales, amax=None):
    """float64 [pages, heads, page, dim] of a cache's codes and scales."""
    p = codes.detach().cpu().long()
    v = E2M1[torch.stack((p & 15, p >> 4), -1)].flatten(-2) * E4M3[byte(scales)].repeat_interleave(16, -1)
    return v if amax is None else v * (f64(amax) / 2688).view(1, -1, 1, 1)


def rows_of(values, table, L):
    """Rows of one sequence [L, heads, dim]: table its row of page numbers."""
    page = values.shape[2]
    j = torch.arange(L)
    return values[table.long()[j // page], :, j % page]


def attention(q, keys, values, table, lens, ends, scale=None, causal=True):
    """(out [T, Hq, D], lse [T, Hq], what out may be off by, what lse may be off by) for bf16 q; keys, values as
    cache_values gives them."""
    q = f64(q)
    T, Hq, D = q.shape
    Hk = keys.shape[1]
    G, scale = Hq // Hk, D ** -0.5 if scale is None else scale
    out, lse = torch.zeros_like(q), torch.full((T, Hq), -math.inf, dtype=torch.float64)
    off, loff = torch.zeros_like(q), torch.zeros(T, Hq, dtype=torch.float64)
    at = 0
    for b, L in enumerate(lens.tolist()):
        end = b + 1 if ends is None else max(at, min(max(int(ends[b]), 0), T))
        n, t = end - at, slice(at, end)
        at = end
        if n == 0 or L <= 0:
            continue
        k = rows_of(keys, table[b], L).repeat_interleave(G, 1)
        v = rows_of(values, table[b], L).repeat_interleave(G, 1)
        s = torch.einsum("thd,lhd->thl", q[t], k) * scale
        if causal:
            hidden = torch.arange(L)[None, :] > torch.arange(n)[:, None] + (L - n)
            s = s.masked_fill(hidden[:, None], -math.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
        total = p.sum(-1, keepdim=True)
        p = torch.where(total > 0, p / total.clamp(min=1e-300), 0.0)
        out[t] = torch.einsum("thl,lhd->thd", p, v)
        lse[t] = (top + torch.log(total)).squeeze(-1)
        # a score: D products summed in fp32 (a matrix core may cut, 2^-23), the power of two's and log2(e)'s products and the
        # difference from the maximum, three roundings of numbers up to the row's largest score's size
        size = torch.einsum("thd,lhd->thl", q[t].abs(), k.abs()) * scale
        size = torch.where(torch.isfinite(s), size, 0.0).amax(-1)
        delta = (D + 16) * 2.0 ** -23 * size + 2.0 ** -20
        # a weight: that, and its rounding to fp16: 2^-11 of it, or half of fp16's smallest step 2^-24 where it is small; weights
        # are 2^11 times exp(s - m) with m at most the row's maximum, so that step is at most 2^-35 of the largest weight; L terms
        # summed in fp32; the result's rounding to bf16
        spread = torch.einsum("thl,lhd->thd", p, v.abs())
        small = L * 2.0 ** -36 * v.abs().amax(0)
        off[t] = out[t].abs() * 2.0 ** -8 + spread * (2.0 ** -11 + 2 * delta + (L + 64) * 2.0 ** -23).unsqueeze(-1) + small
        loff[t] = 2 * delta + (L + 64) * 2.0 ** -23 + torch.where(torch.isfinite(lse[t]), lse[t].abs(), 0.0) * 2.0 ** -22
    return out, lse, off, loff
