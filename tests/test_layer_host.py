"""The layer operators' entry points without a GPU: bad arguments are refused
on the host with the documented status before anything is launched (fake,
never-dereferenced device addresses), CPU tensors are refused by the binding,
and the 64-bit definitions that the GPU tests use hold against values worked
out by hand and, for the gradients, against differences."""
import math

import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
from fp4_block_quantization_nvfp4_amd import _lib as L
from tests import layer_ref as R

A = 1 << 20  # a fake, 256-byte-aligned device address (never dereferenced)
INF = float("inf")


def norm(*, x=A, res=A, dt=L.BF16, w=A, T=4, H=64, eps=1e-6, codes=A, scales=A, hidden=A, rstd=A):
    return L.lib().nvfp4_add_rms_norm(x, res, dt, w, T, H, eps, codes, scales, hidden, rstd, None)


@pytest.mark.parametrize("kw,status", [
    (dict(H=24), L.E_SHAPE), (dict(T=-1), L.E_SHAPE), (dict(H=-16), L.E_SHAPE), (dict(H=32784), L.E_RANGE),
    (dict(T=1 << 31, H=16), L.E_RANGE), (dict(T=1 << 20, H=16384), L.E_RANGE),
    (dict(dt=3), L.E_DTYPE), (dict(eps=-1.0), L.E_ARG), (dict(eps=float("nan")), L.E_ARG),
    (dict(res=None), L.E_NULL), (dict(hidden=None), L.E_NULL), (dict(x=None), L.E_NULL), (dict(w=None), L.E_NULL),
    (dict(codes=None), L.E_NULL), (dict(scales=None), L.E_NULL), (dict(rstd=None), L.E_NULL),
    (dict(x=A + 8), L.E_ALIGN), (dict(res=A + 2), L.E_ALIGN), (dict(w=A + 4), L.E_ALIGN), (dict(codes=A + 8), L.E_ALIGN),
    (dict(hidden=A + 8), L.E_ALIGN), (dict(rstd=A + 2), L.E_ALIGN),
    (dict(T=0, x=None, w=None, codes=None, scales=None, rstd=None), L.OK),
    (dict(H=0, x=None, w=None, codes=None, scales=None, rstd=None), L.OK),
])
def test_norm_rejects(kw, status):
    assert norm(**kw) == status


def norm_bwd(*, dy=A, hidden=A, dh=A, dt=L.BF16, w=A, rstd=A, T=4, H=64, dx=A, dw=A, ws=A, n=None):
    lib = L.lib()
    n = lib.nvfp4_add_rms_norm_backward_workspace_bytes(T, H) if n is None else n
    return lib.nvfp4_add_rms_norm_backward(dy, hidden, dh, dt, w, rstd, T, H, dx, dw, ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(H=40), L.E_SHAPE), (dict(T=-4), L.E_SHAPE), (dict(H=65536), L.E_RANGE), (dict(dt=2), L.E_DTYPE),
    (dict(n=4 * 64 * 4 - 1), L.E_ARG), (dict(dy=None), L.E_NULL), (dict(hidden=None), L.E_NULL),
    (dict(w=None), L.E_NULL), (dict(rstd=None), L.E_NULL), (dict(dx=None), L.E_NULL), (dict(dw=None), L.E_NULL),
    (dict(ws=None), L.E_NULL), (dict(dy=A + 8), L.E_ALIGN), (dict(dh=A + 8), L.E_ALIGN), (dict(dx=A + 4), L.E_ALIGN),
    (dict(dw=A + 4), L.E_ALIGN), (dict(ws=A + 8), L.E_ALIGN), (dict(T=0, dw=None), L.E_NULL), (dict(H=0, dw=None), L.OK),
])
def test_norm_backward_rejects(kw, status):
    assert norm_bwd(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(F=8), L.E_SHAPE), (dict(T=-1), L.E_SHAPE), (dict(dt=9), L.E_DTYPE), (dict(T=1 << 20, F=8192), L.E_RANGE),
    (dict(kept=None), L.E_NULL), (dict(ks=None), L.E_NULL), (dict(x=None), L.E_NULL), (dict(codes=None), L.E_NULL),
    (dict(x=A + 8), L.E_ALIGN), (dict(codes=A + 8), L.E_ALIGN), (dict(kept=A + 8), L.E_ALIGN),
    (dict(T=0, x=None, codes=None), L.OK), (dict(F=0, x=None), L.OK),
])
def test_swiglu_rejects(kw, status):
    a = dict(x=A, dt=L.BF16, T=4, F=32, codes=A, scales=A, kept=A, ks=A) | kw
    assert L.lib().nvfp4_swiglu(a["x"], a["dt"], a["T"], a["F"], a["codes"], a["scales"], a["kept"], a["ks"], None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(F=8), L.E_SHAPE), (dict(dt=9), L.E_DTYPE), (dict(kept=None), L.E_NULL), (dict(ks=None), L.E_NULL),
    (dict(d=None), L.E_NULL), (dict(out=None), L.E_NULL), (dict(d=A + 8), L.E_ALIGN), (dict(out=A + 8), L.E_ALIGN),
    (dict(T=0, d=None), L.OK),
])
def test_swiglu_backward_rejects(kw, status):
    a = dict(d=A, dt=L.BF16, T=4, F=32, kept=A, ks=A, out=A) | kw
    assert L.lib().nvfp4_swiglu_backward(a["d"], a["dt"], a["T"], a["F"], a["kept"], a["ks"], a["out"], None) == status


PRODUCT = [
    (dict(K=24), L.E_SHAPE), (dict(T=-1), L.E_SHAPE), (dict(N=-1), L.E_SHAPE), (dict(N=40, blocks=1), L.E_SHAPE),
    (dict(N=40, blocks=2), L.E_SHAPE), (dict(blocks=3), L.E_ARG), (dict(out_dt=7), L.E_DTYPE), (dict(mode=4), L.E_ARG),
    (dict(blocks=1, mode=L.SCALE_ROW), L.E_ARG), (dict(bound=300.0), L.E_ARG), (dict(K=(1 << 20) + 16), L.E_RANGE),
    (dict(N=(1 << 20) + 1), L.E_RANGE), (dict(T=1 << 31), L.E_RANGE), (dict(T=1 << 28), L.E_RANGE),
    (dict(N=1 << 20, K=1 << 14), L.E_RANGE), (dict(x=None), L.E_NULL), (dict(packed=None), L.E_NULL),
    (dict(scales=None), L.E_NULL), (dict(amax=None), L.E_NULL), (dict(out=None), L.E_NULL), (dict(x=A + 8), L.E_ALIGN),
    (dict(packed=A + 4), L.E_ALIGN), (dict(amax=A + 1), L.E_ALIGN), (dict(out=A + 8), L.E_ALIGN),
    (dict(T=0, x=None, out=None), L.OK), (dict(N=0, packed=None, out=None), L.OK),
]


@pytest.mark.parametrize("kw,status", PRODUCT)
def test_matvec_rejects(kw, status):
    a = dict(x=A, T=4, N=64, K=64, packed=A, scales=A, blocks=0, amax=A, mode=1, bound=448.0, out=A, out_dt=L.BF16) | kw
    assert L.lib().nvfp4_matvec(a["x"], None, a["T"], a["N"], a["K"], a["packed"], a["scales"], a["blocks"], a["amax"],
                                a["mode"], a["bound"], a["out"], a["out_dt"], None) == status


@pytest.mark.parametrize("kw,status", PRODUCT + [
    (dict(E=0), L.E_SHAPE), (dict(E=65535), L.E_RANGE), (dict(E=1 << 13, N=1 << 10, K=1 << 11), L.E_RANGE),
    (dict(ends=None), L.E_NULL), (dict(ends=A + 2), L.E_ALIGN)])
def test_grouped_matmul_rejects(kw, status):
    a = dict(x=A, T=4, E=2, N=64, K=64, ends=A, packed=A, scales=A, blocks=0, amax=A, mode=1, bound=448.0, out=A,
             out_dt=L.BF16) | kw
    assert L.lib().nvfp4_grouped_matmul(a["x"], None, a["T"], a["E"], a["N"], a["K"], a["ends"], a["packed"], a["scales"],
                                        a["blocks"], a["amax"], a["mode"], a["bound"], a["out"], a["out_dt"],
                                        None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(K=24), L.E_SHAPE), (dict(N=40), L.E_SHAPE), (dict(E=0), L.E_SHAPE), (dict(out_dt=5), L.E_DTYPE),
    (dict(ends=None), L.E_NULL), (dict(dw=None), L.E_NULL), (dict(dy=None), L.E_NULL), (dict(x=None), L.E_NULL),
    (dict(T=0, dy=None, x=None, dw=None), L.E_NULL), (dict(dy=A + 8), L.E_ALIGN), (dict(x=A + 4), L.E_ALIGN),
    (dict(dw=A + 8), L.E_ALIGN), (dict(K=0, dw=None), L.OK),
])
def test_grouped_wgrad_rejects(kw, status):
    a = dict(dy=A, x=A, T=4, E=2, N=64, K=64, ends=A, dw=A, out_dt=L.F32) | kw
    assert L.lib().nvfp4_grouped_wgrad(a["dy"], a["x"], None, a["T"], a["E"], a["N"], a["K"], a["ends"], a["dw"],
                                       a["out_dt"], None) == status


def test_cpu_tensors_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    p, s = torch.zeros(2, 32, 32, dtype=torch.uint8), torch.zeros(2, 32, 4, dtype=torch.uint8)
    ends = torch.tensor([2, 4], dtype=torch.int32)
    for call in (lambda: nv.add_rms_norm(x, torch.ones(64)), lambda: nv.swiglu_checkpoint(x),
                 lambda: nv.add_rms_norm_backward(x, x, torch.ones(64), torch.ones(4)),
                 lambda: nv.swiglu_backward(x, torch.zeros(4, 128, dtype=R.F8), torch.zeros(4, 4, dtype=torch.uint8)),
                 lambda: nv.matvec(x, p[0], s[0]), lambda: nv.grouped_matmul(x, ends, p, s),
                 lambda: nv.matvec(x.to(R.F8), p[0], s[0], x_scale=torch.ones(4, 2, dtype=torch.uint8)),
                 lambda: nv.grouped_wgrad(x, x, ends)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


# ------------------------------------------------- the 64-bit definitions

def test_mx8_definition():
    v = torch.zeros(6, 48, dtype=torch.float64)
    v[0, 0], v[0, 1], v[0, 2] = 448.0, -1.0625, 2.0 ** -10   # scale 2^0; a tie to even; half the smallest step
    v[1, 3] = 448.0 * (1 + 2.0 ** -23)                       # just over: scale 2^1
    v[2, 40], v[2, 41] = INF, 3.0                            # the infinity does not count; short last group
    v[3, 5] = float("nan")
    v[4, 0] = 1e-40
    v[5, 0] = 3.4e38
    c, s = R.mx8_codes(v)
    assert s[0].tolist() == [127, 10] and s[1, 0] == 128 and s[4, 0] == 10
    assert c[0, :3].tolist() == [0x7E, 0x80 | 0x38, 0]       # 1.0625 lies halfway between 1 and 1.125
    assert c[1, 3] == 0x76                                   # 224
    assert c[2, 40] == 127 and R.mx8_values(c, s)[2, 41] == 3.0
    assert c[3, 5] == 127 and s[3, 0] == 10
    assert 448 * 2.0 ** (int(s[5, 0]) - 127) >= 3.4e38 > 448 * 2.0 ** (int(s[5, 0]) - 128)


def test_gradients_against_differences():
    """The gradient formulas that the kernels are tested against."""
    g = torch.Generator().manual_seed(5)
    x, r, w, dy = (torch.randn(*s, dtype=torch.float64, generator=g) for s in ((3, 32), (3, 32), (32,), (3, 32)))

    def y(x):
        h = x + r
        return (h * (h * h).mean(1, keepdim=True).add(1e-6).rsqrt() * w * dy).sum()

    h = x + r
    rstd = (h * h).mean(1).add(1e-6).rsqrt()
    got = R.norm_gradient(dy, h, w, rstd, None)[0]
    for _ in range(4):
        d = torch.randn(3, 32, dtype=torch.float64, generator=g)
        e = 1e-5
        assert math.isclose(((y(x + e * d) - y(x - e * d)) / (2 * e)).item(), (got * d).sum().item(), rel_tol=1e-7, abs_tol=1e-8)
    gate, up, do = (torch.randn(3, 16, dtype=torch.float64, generator=g) * 2 for _ in range(3))
    dg, du = R.swiglu_gradient(do, gate, up)
    f = lambda a, b: (a / (1 + torch.exp(-a)) * b * do).sum()
    for _ in range(4):
        a, b = (torch.randn(3, 16, dtype=torch.float64, generator=g) for _ in range(2))
        e = 1e-5
        slope = (f(gate + e * a, up + e * b) - f(gate - e * a, up - e * b)) / (2 * e)
        assert math.isclose(slope.item(), ((dg * a) + (du * b)).sum().item(), rel_tol=1e-7, abs_tol=1e-8)


def test_row_ranges_definition():
    assert R.cuts(torch.tensor([3, 1, 9, -4]), 7) == [0, 3, 3, 7, 7]
