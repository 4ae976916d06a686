"""Operators of a layer whose weights are stored in NVFP4, on torch tensors.

8-bit rows ("mx8"): `codes` float8_e4m3fn [T, K] and `scales` float8_e8m0fnu
[T, ceil(K / 32)], one power of two for each 32 consecutive elements of a row
(the last group may be shorter; K % 16 == 0): the smallest one, from 2^-117
up, under which no finite value exceeds 448; what is not finite becomes NaN.
uint8 views of either are taken too.

4-bit weights are the outputs of `quantize`, `quantize_4over6`, `quantize_2d`,
`quantize_rowcol` and `quantize_4over6_2d`, for experts stacked along a first
axis.  As in `dequantize`, `tile16`, `global_amax`, `row_scaled` and `bound`
name the producer's scales.

Every function runs on torch's current stream, allocates its outputs with
torch and computes in the HIP kernels.  The rows are contiguous tensors; there
is no CPU path.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .api import _DT, _check_input, _ptr, _stream

_F8, _E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _groups(K):
    return (K + 31) // 32


def _same(t, like, what):
    """t has like's shape, type and device, and is contiguous."""
    if not isinstance(t, torch.Tensor) or t.shape != like.shape or t.dtype != like.dtype or t.device != like.device \
            or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {str(like.dtype)[6:]} {list(like.shape)} tensor on the same device")
    return t


def _array(t, dtype, n, device, what):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {str(dtype)[6:]} tensor of {n} elements on the same device")
    return t


def _mx8_empty(T, K, device, halves=1):
    return (torch.empty((T, halves * K), dtype=_F8, device=device),
            torch.empty((T, halves * _groups(K)), dtype=_E8, device=device))


def _codes(t, what):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what}: a device tensor is required (no CPU path)")
    if t.dim() != 2 or t.dtype not in (_F8, torch.uint8) or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous 2-D float8_e4m3fn (or uint8) tensor")
    return t


def _scale_bytes(t, rows, n, device, what):
    if not isinstance(t, torch.Tensor) or t.dtype not in (_E8, torch.uint8) or tuple(t.shape) != (rows, n) \
            or t.device != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous float8_e8m0fnu (or uint8) [{rows}, {n}] tensor on the same device")
    return t


def add_rms_norm(x, weight, residual=None, *, eps=1e-6):
    """Norm of h = x + residual, y = h * rstd * weight with rstd = (mean(h^2) +
    eps)^(-1/2) -> (codes, scales, hidden, rstd): y as mx8, h in x's type (x
    itself without a residual) and rstd float32 [T].  x float32 or bfloat16
    [T, H], H % 16 == 0; weight float32 [H]."""
    T, H = _check_input(x, "add_rms_norm")
    _array(weight, torch.float32, H, x.device, "weight")
    if residual is not None:
        _same(residual, x, "residual")
    codes, scales = _mx8_empty(T, H, x.device)
    hidden = None if residual is None else torch.empty_like(x)
    rstd = torch.empty(T, dtype=torch.float32, device=x.device)
    L.check(L.lib().nvfp4_add_rms_norm(_ptr(x), _ptr(residual), _DT[x.dtype], _ptr(weight), T, H, float(eps),
                                       _ptr(codes), _ptr(scales), _ptr(hidden), _ptr(rstd), _stream()),
            "nvfp4_add_rms_norm")
    return codes, scales, x if hidden is None else hidden, rstd


def add_rms_norm_backward(dy, hidden, weight, rstd, dhidden=None):
    """Gradient of `add_rms_norm` -> (dx, dweight).  dy is the gradient of y,
    dhidden the one that reaches the sum h from elsewhere (the residual path);
    dx, in dy's type, is the gradient of x and of residual alike; dweight is
    float32 [H]."""
    T, H = _check_input(dy, "add_rms_norm_backward")
    _same(hidden, dy, "hidden")
    if dhidden is not None:
        _same(dhidden, dy, "dhidden")
    _array(weight, torch.float32, H, dy.device, "weight")
    _array(rstd, torch.float32, T, dy.device, "rstd")
    dx = torch.empty_like(dy)
    dweight = torch.empty(H, dtype=torch.float32, device=dy.device)
    nws = L.lib().nvfp4_add_rms_norm_backward_workspace_bytes(T, H)
    ws = torch.empty(max(nws, 4), dtype=torch.uint8, device=dy.device)
    L.check(L.lib().nvfp4_add_rms_norm_backward(_ptr(dy), _ptr(hidden), _ptr(dhidden), _DT[dy.dtype], _ptr(weight),
                                                _ptr(rstd), T, H, _ptr(dx), _ptr(dweight), _ptr(ws), ws.numel(),
                                                _stream()), "nvfp4_add_rms_norm_backward")
    return dx, dweight


def swiglu_checkpoint(gate_up, *, keep=True):
    """y = g * sigmoid(g) * u of rows [g | u] [T, 2F] -> (codes, scales, kept,
    kept_scales): y as mx8 [T, F], and with keep the mx8 checkpoint of g and u
    that `swiglu_backward` reads (else None, None).  F % 16 == 0."""
    T, F2 = _check_input(gate_up, "swiglu_checkpoint")
    if F2 % 32:
        raise ValueError("swiglu_checkpoint: gate_up must be [T, 2F] with F % 16 == 0")
    F = F2 // 2
    codes, scales = _mx8_empty(T, F, gate_up.device)
    kept, kept_scales = _mx8_empty(T, F, gate_up.device, 2) if keep else (None, None)
    L.check(L.lib().nvfp4_swiglu(_ptr(gate_up), _DT[gate_up.dtype], T, F, _ptr(codes), _ptr(scales), _ptr(kept),
                                 _ptr(kept_scales), _stream()), "nvfp4_swiglu")
    return codes, scales, kept, kept_scales


def swiglu_backward(dout, kept, kept_scales):
    """Gradient of the gated activation at the checkpoint's values ->
    dgate_up [T, 2F] in dout's type."""
    T, F = _check_input(dout, "swiglu_backward")
    _codes(kept, "kept")
    if tuple(kept.shape) != (T, 2 * F) or kept.device != dout.device:
        raise ValueError("kept must be [T, 2F] on dout's device")
    _scale_bytes(kept_scales, T, 2 * _groups(F), dout.device, "kept_scales")
    dgate_up = torch.empty((T, 2 * F), dtype=dout.dtype, device=dout.device)
    L.check(L.lib().nvfp4_swiglu_backward(_ptr(dout), _DT[dout.dtype], T, F, _ptr(kept), _ptr(kept_scales),
                                          _ptr(dgate_up), _stream()), "nvfp4_swiglu_backward")
    return dgate_up


def _rows(x, x_scale, what):
    """Checks rows that are bf16, or mx8 with x_scale; returns T, K."""
    if x_scale is None:
        T, K = _check_input(x, what)
        if x.dtype != torch.bfloat16:
            raise ValueError(f"{what}: x must be bfloat16, or float8_e4m3fn with x_scale")
    else:
        _codes(x, f"{what}: x")
        T, K = x.shape
        _scale_bytes(x_scale, T, _groups(K), x.device, "x_scale")
    return T, K


def _weights(x, packed, scale, lead, K, blocks, global_amax, row_scaled, out_dtype):
    """Checks 4-bit weights [*lead, N, K / 2]; returns N, the second-level
    scale's mode and its amax."""
    for t, name in ((packed, "packed"), (scale, "scale")):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.uint8 or t.device != x.device:
            raise ValueError(f"{name} must be a uint8 tensor on x's device")
    d = len(lead)
    if packed.dim() != d + 2 or tuple(packed.shape[:d]) != lead or packed.shape[-1] * 2 != K:
        raise ValueError(f"packed must be {[*lead, 'N', K // 2]}")
    N = packed.shape[-2]
    want = {L.BLOCK_1X16: (N, K // 16), L.BLOCK_16X16: (N // 16, K // 16), L.BLOCK_16X16_T: (K // 16, N // 16)}[blocks]
    if tuple(scale.shape) != lead + want:
        raise ValueError(f"scale must be {list(lead + want)}")
    if out_dtype not in _DT:
        raise ValueError("out_dtype must be float32 or bfloat16")
    if global_amax is None:
        if row_scaled:
            raise ValueError("row_scaled needs a global_amax for each row")
        return N, L.SCALE_NONE, None
    experts = lead[0] if lead else 1
    if not isinstance(global_amax, torch.Tensor):
        global_amax = torch.full((experts,), float(global_amax), dtype=torch.float32, device=x.device)
    n = experts * N if row_scaled else experts
    _array(global_amax, torch.float32, n, x.device, "global_amax")
    return N, L.SCALE_ROW if row_scaled else L.SCALE_TENSOR, global_amax


def matvec(x, packed, scale, *, x_scale=None, tile16=False, global_amax=None, row_scaled=False, bound=448.0,
           out_dtype=torch.bfloat16):
    """x W^T for a 4-bit weight W [N, K] and a few rows x [T, K], bfloat16 or
    mx8 (with x_scale) -> [T, N].  Up to 16 rows cost one read of the
    weights."""
    T, K = _rows(x, x_scale, "matvec")
    blocks = L.BLOCK_16X16 if tile16 else L.BLOCK_1X16
    N, mode, amax = _weights(x, packed, scale, (), K, blocks, global_amax, row_scaled, out_dtype)
    packed, scale = packed.contiguous(), scale.contiguous()
    out = torch.empty((T, N), dtype=out_dtype, device=x.device)
    L.check(L.lib().nvfp4_matvec(_ptr(x), _ptr(x_scale), T, N, K, _ptr(packed), _ptr(scale), blocks, _ptr(amax), mode,
                                 float(bound), _ptr(out), _DT[out_dtype], _stream()), "nvfp4_matvec")
    return out


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
    T, K = _rows(x, x_scale, "grouped_matmul")
    if transposed_tiles and not tile16:
        raise ValueError("transposed_tiles goes with tile16")
    blocks = L.BLOCK_16X16_T if transposed_tiles else L.BLOCK_16X16 if tile16 else L.BLOCK_1X16
    E = packed.shape[0] if isinstance(packed, torch.Tensor) and packed.dim() == 3 else 0
    if E < 1:
        raise ValueError("packed must be [E, N, K / 2] with at least one expert")
    N, mode, amax = _weights(x, packed, scale, (E,), K, blocks, global_amax, row_scaled, out_dtype)
    _array(ends, torch.int32, E, x.device, "ends")
    packed, scale = packed.contiguous(), scale.contiguous()
    out = torch.empty((T, N), dtype=out_dtype, device=x.device)
    L.check(L.lib().nvfp4_grouped_matmul(_ptr(x), _ptr(x_scale), T, E, N, K, _ptr(ends), _ptr(packed), _ptr(scale),
                                         blocks, _ptr(amax), mode, float(bound), _ptr(out), _DT[out_dtype],
                                         _stream()), "nvfp4_grouped_matmul")
    return out


def grouped_wgrad(dy, x, ends, *, x_scale=None, out_dtype=torch.float32):
    """Weight gradient of `grouped_matmul`: for each expert the sum over its
    rows of dy[t]^T x[t] -> [E, N, K].  dy bfloat16 [T, N], N % 16 == 0; x
    bfloat16 or mx8 (with x_scale).  An expert without rows gets zeros."""
    T, N = _check_input(dy, "grouped_wgrad")
    if dy.dtype != torch.bfloat16:
        raise ValueError("grouped_wgrad: dy must be bfloat16")
    Tx, K = _rows(x, x_scale, "grouped_wgrad")
    if Tx != T or x.device != dy.device:
        raise ValueError("dy and x must have the same rows, on one device")
    if out_dtype not in _DT:
        raise ValueError("out_dtype must be float32 or bfloat16")
    E = ends.numel() if isinstance(ends, torch.Tensor) else 0
    if E < 1:
        raise ValueError("ends must hold at least one expert")
    _array(ends, torch.int32, E, dy.device, "ends")
    dw = torch.empty((E, N, K), dtype=out_dtype, device=dy.device)
    L.check(L.lib().nvfp4_grouped_wgrad(_ptr(dy), _ptr(x), _ptr(x_scale), T, E, N, K, _ptr(ends), _ptr(dw),
                                        _DT[out_dtype], _stream()), "nvfp4_grouped_wgrad")
    return dw
