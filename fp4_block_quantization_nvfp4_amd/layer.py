"""Operators of a layer whose weights are stored in NVFP4, on torch tensors.

8-bit rows ("mx8"): `codes` float8_e4m3fn [T, K] and `scales` float8_e8m0fnu
[T, ceil(K / 32)], one power of two for each 32 consecutive elements of a row
(the last group may be shorter; K % 16 == 0): the smallest one, from 2^-117
up, under which no finite value exceeds 448; what is not finite becomes NaN.
Any scale is read: 255 as NaN, values below 2^-126 possibly as zero, those from
2^128 on as infinite.  uint8 views of either are taken too.

4-bit weights are the outputs of `quantize`, `quantize_4over6`, `quantize_2d`,
`quantize_rowcol` and `quantize_4over6_2d`, for experts stacked along a first
axis.  As in `dequantize`, `tile16`, `global_amax`, `row_scaled` and `bound`
name the producer's scales.

Every function runs on torch's current stream, on the current device, allocates
its outputs with torch and computes in the HIP kernels.  The rows are contiguous
tensors; there is no CPU path.

Nothing is recorded for autograd: inputs that require a gradient are taken as
they are, and the outputs require none.  A training step calls the gradients by
name, as examples/expert_layer.py does: `add_rms_norm_backward`,
`swiglu_backward`, `grouped_matmul` with the transposed weights and
`grouped_wgrad`.
"""
from __future__ import annotations

import torch


class _Native:
    """The compiled binding (bind/layer.cpp), loaded at its first use; it checks
    the arguments, allocates the outputs and calls the C ABI."""

    def __getattr__(self, name):
        try:
            from . import _layer
        except ImportError as e:
            raise ImportError(f"{e}: build it with `python -m fp4_block_quantization_nvfp4_amd.build`") from e
        f = getattr(_layer, name)
        setattr(self, name, f)
        return f


_n = _Native()


def add_rms_norm(x, weight, residual=None, *, eps=1e-6):
    """Norm of h = x + residual, y = h * rstd * weight with rstd = (mean(h^2) +
    eps)^(-1/2) -> (codes, scales, hidden, rstd): y as mx8, h in x's type (x
    itself without a residual) and rstd float32 [T].  x float32 or bfloat16
    [T, H], H % 16 == 0; weight float32 [H]."""
    return _n.add_rms_norm(x, weight, residual, eps)


def add_rms_norm_backward(dy, hidden, weight, rstd, dhidden=None):
    """Gradient of `add_rms_norm` -> (dx, dweight).  dy is the gradient of y,
    dhidden the one that reaches the sum h from elsewhere (the residual path);
    dx, in dy's type, is the gradient of x and of residual alike; dweight is
    float32 [H]."""
    return _n.add_rms_norm_backward(dy, hidden, weight, rstd, dhidden)


def swiglu_checkpoint(gate_up, *, keep=True):
    """y = g * sigmoid(g) * u of rows [g | u] [T, 2F] -> (codes, scales, kept,
    kept_scales): y as mx8 [T, F], and with keep the mx8 checkpoint of g and u
    that `swiglu_backward` reads (else None, None).  F % 16 == 0."""
    return _n.swiglu_checkpoint(gate_up, keep)


def swiglu_backward(dout, kept, kept_scales):
    """Gradient of the gated activation at the checkpoint's values ->
    dgate_up [T, 2F] in dout's type."""
    return _n.swiglu_backward(dout, kept, kept_scales)


def matvec(x, packed, scale, *, x_scale=None, tile16=False, global_amax=None, row_scaled=False, bound=448.0,
           out_dtype=torch.bfloat16):
    """x W^T for a 4-bit weight W [N, K] and a few rows x [T, K], bfloat16 or
    mx8 (with x_scale) -> [T, N].  Up to 16 rows cost one read of the
    weights."""
    return _n.matvec(x, packed, scale, x_scale, tile16, global_amax, row_scaled, bound, out_dtype)


def grouped_matmul(x, ends, packed, scale, *, x_scale=None, tile16=False, transposed_tiles=False, global_amax=None,
                   row_scaled=False, bound=448.0, out_dtype=torch.bfloat16):
    """Rows grouped by expert times the experts' 4-bit weights W_e [N, K] ->
    [T, N].  ends: int32 [E] on the device, the non-decreasing cumulative row
    counts: expert e owns rows ends[e - 1] up to ends[e]; rows past the last
    end belong to no expert and give zeros.  For the gradient of the forward
    product's input pass the gradient of its output and the transposed
    weights: a quantization of their own (`quantize_rowcol`), or the columnwise
    codes of `quantize_2d` / `quantize_4over6_2d` with the tile scales as they
    are, [K / 16, N / 16] seen from here (transposed_tiles)."""
    return _n.grouped_matmul(x, ends, packed, scale, x_scale, tile16, transposed_tiles, global_amax, row_scaled, bound,
                             out_dtype)


def grouped_wgrad(dy, x, ends, *, x_scale=None, out_dtype=torch.float32):
    """Weight gradient of `grouped_matmul`: for each expert the sum over its
    rows of dy[t]^T x[t] -> [E, N, K].  dy bfloat16 [T, N], N % 16 == 0; x
    bfloat16 or mx8 (with x_scale).  An expert without rows gets zeros."""
    return _n.grouped_wgrad(dy, x, ends, x_scale, out_dtype)
