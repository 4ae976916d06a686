"""Operators of attention whose keys and values are stored in NVFP4, on torch
tensors.

Queries, keys and values are [T, heads, D], rows of D elements that start at
multiples of 16 bytes; tokens and heads may have any strides, so that parts of one
projection are taken as they are.  The cache is a `PagedCache`; what it holds for
a row is what `quantize` gives for it.  A slot is numbered page * page_size + its
place in the page.

Positions, slots, page tables and lengths are int32 tensors on the device; no
call waits for them.  Every function runs on torch's current stream, on the
current device, allocates its outputs (and workspace, one a call) with torch and
computes in the HIP kernels.  There is no CPU path, and nothing is recorded for
autograd: `norm_rope_backward` is called by name.
"""
from __future__ import annotations

import math

import torch

from .layer import _n


def rotary_frequencies(dim, *, base=10000.0, factor=1.0, scaling="none", original_length=None, device=None):
    """Angle of one step for each of the dim / 2 pairs, and the rotation's
    multiplier -> (float64 [dim / 2], float).  f_i = base^(-2 i / dim), scaled for
    contexts `factor` times as long as those trained on:

    "none"    as it is (factor is not read);
    "linear"  f_i / factor;
    "base"    base * factor^(dim / (dim - 2)): the slowest pair turns factor times
              slower, the fastest as before;
    "parts"   the YaRN method: pairs that turn more than 32 times in original_length
              stay, those that turn less than once are divided by factor, a ramp
              between, from the pair below the one that turns 32 times to the pair
              above the one that turns once; the multiplier is 0.1 ln(factor) + 1.
    """
    if dim < 0 or dim % 2:
        raise ValueError("dim must be even")
    if not (0 < base < math.inf and 1 <= factor < math.inf):
        raise ValueError("base > 0 and factor >= 1, both finite, are required")
    if scaling not in ("none", "linear", "base", "parts"):
        raise ValueError("scaling must be 'none', 'linear', 'base' or 'parts'")
    if scaling == "parts" and not (base > 1 and original_length and 0 < original_length < math.inf):
        raise ValueError("scaling 'parts' needs original_length > 0 and base > 1")
    if scaling == "base" and dim > 2:
        base = base * factor ** (dim / (dim - 2))
    f = [base ** (-2 * i / dim) for i in range(dim // 2)]
    multiplier = 1.0
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "parts":
        # the pair, as a fraction, that turns r times in original_length
        pair = lambda r: dim * math.log(original_length / (r * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), dim - 1)
        ramp = [min(max((i - low) / max(high - low, 0.001), 0.0), 1.0) for i in range(dim // 2)]
        f = [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)]
        multiplier = 0.1 * math.log(factor) + 1.0
    return torch.tensor(f, dtype=torch.float64, device="cuda" if device is None else device), multiplier


class PagedCache:
    """Keys and values in NVFP4: `k`, `v` uint8 [pages, heads, page_size, dim / 2],
    `k_scale`, `v_scale` uint8 [pages, heads, page_size, dim / 16], and a
    second-level scale's amax for each head, `k_amax`, `v_amax` float32 [heads] (or
    None).  page_size is a power of two, 16 to 65536; dim % 16 == 0, up to 512
    (attention: dim % 32 == 0, up to 256)."""

    __slots__ = ("k", "k_scale", "v", "v_scale", "k_amax", "v_amax")

    def __init__(self, k, k_scale, v, v_scale, *, k_amax=None, v_amax=None):
        self.k, self.k_scale, self.v, self.v_scale, self.k_amax, self.v_amax = k, k_scale, v, v_scale, k_amax, v_amax

    @classmethod
    def empty(cls, pages, page_size, heads, dim, *, k_amax=None, v_amax=None, device=None):
        """A cache of zeros."""
        make = lambda n: torch.zeros(pages, heads, page_size, n, dtype=torch.uint8, device="cuda" if device is None else device)
        return cls(make(dim // 2), make(dim // 16), make(dim // 2), make(dim // 16), k_amax=k_amax, v_amax=v_amax)


def norm_rope(q, k, positions, freqs, *, q_weight=None, k_weight=None, interleaved=False, multiplier=1.0, eps=1e-6):
    """Norm of each head's row with the rotation of its position -> (q, k), dense,
    in their type (float32 or bfloat16): y = x (mean(x^2) + eps)^(-1/2) weight (y =
    x without a weight), then the pairs (y_i, y_{i+R/2}), or (y_2i, y_2i+1) where
    interleaved, turned by positions[t] * freqs[i] and taken times multiplier.  freqs
    float64 [R / 2], R % 16 == 0, R <= D: elements from R on are not turned; R = 0
    is the norm alone.  weights float32 [D].  D % 16 == 0, up to 512.  Computed in
    64 bits, rounded to float32 and from there to bfloat16."""
    return _n.norm_rope(q, k, positions, freqs, q_weight, k_weight, interleaved, multiplier, eps)


def norm_rope_backward(dq, dk, q, k, positions, freqs, *, q_weight=None, k_weight=None, interleaved=False, multiplier=1.0,
                       eps=1e-6):
    """Gradient of `norm_rope` from the gradients of its outputs and from its inputs
    -> (dq, dk, dq_weight, dk_weight): the inputs', dense, and the weights', float32
    [D], summed over tokens and heads (None without a weight)."""
    return _n.norm_rope_backward(dq, dk, q, k, positions, freqs, q_weight, k_weight, interleaved, multiplier, eps)


def norm_rope_write(q, k, v, positions, freqs, cache, slots, *, q_weight=None, k_weight=None, interleaved=False,
                    multiplier=1.0, eps=1e-6):
    """`norm_rope` whose keys go straight to the cache, with the values v -> q.  The
    cache then holds what `write_cache` of `norm_rope`'s keys gives."""
    return _n.norm_rope_write(q, k, v, slots, cache.k, cache.k_scale, cache.v, cache.v_scale, cache.k_amax, cache.v_amax,
                              positions, freqs, q_weight, k_weight, interleaved, multiplier, eps)


def write_cache(cache, k, v, slots):
    """Quantizes the rows of token t into slots[t].  Slots that are negative or past
    the cache are skipped; the others differ from each other."""
    return _n.write_cache(k, v, slots, cache.k, cache.k_scale, cache.v, cache.v_scale, cache.k_amax, cache.v_amax)


def read_cache(cache, slots, *, out_dtype=torch.bfloat16):
    """The rows of the slots -> (k, v) [len(slots), heads, dim], as `dequantize`;
    zeros for slots that are negative or past the cache."""
    return _n.read_cache(slots, cache.k, cache.k_scale, cache.v, cache.v_scale, cache.k_amax, cache.v_amax, out_dtype)


def cache_attention(q, cache, table, lens, ends=None, *, scale=None, causal=True):
    """softmax(scale q K^T) V over the cache -> (out bfloat16 [T, heads, D], lse
    float32 [T, heads]), lse the log of the sum of exp(scale q k).

    q bfloat16 [T, heads, D], heads a multiple of the cache's: equal runs of them
    share a head of keys.  Sequence b owns the queries from ends[b - 1] up to
    ends[b] (int32 [B], non-decreasing; None: T == B, query b alone) and lens[b]
    keys; key j lies in page table[b, j // page_size] (int32 [B, pages at most]).
    causal: the sequence's last queries and keys are the same tokens, so query i of
    n sees the keys j <= lens[b] - n + i; otherwise all (an encoder's states).
    Queries without keys and those past the last end get 0 and -inf; NaN those that
    see a key of a page that is not in the cache or with a NaN among its scales or its
    value's, and all of a sequence with more keys than its row of the table names.
    scale > 0, D ** -0.5 by default.  The same call gives the same bits; the last ones
    may change with the other sequences and the table's width."""
    return _n.cache_attention(q, cache.k, cache.k_scale, cache.v, cache.v_scale, cache.k_amax, cache.v_amax, table, lens, ends,
                              scale, causal)
