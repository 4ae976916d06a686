"""The split weight gradient's entry point and the compiled binding without a
GPU: statuses for bad arguments (fake, never-dereferenced addresses), the
workspace query, and what the binding refuses before it touches a device."""
import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
from fp4_block_quantization_nvfp4_amd import _lib as L

A = 1 << 20
BIG = dict(T=16384, E=1, N=1024, K=512)


def query(T, E, N, K):
    return L.lib().nvfp4_grouped_wgrad_workspace_bytes(T, E, N, K)


def test_workspace_query():
    n = query(**BIG)
    block = 1024 * 512 * 4  # one block's sums
    assert n % block == 0 and 4 <= n // block <= 64
    assert query(16, 1, 1024, 512) == 0            # few rows
    assert query(16384, 16, 4096, 2048) == 0       # enough tiles
    assert query(0, 1, 16, 16) == 0 and query(16384, 1, 0, 512) == 0 and query(16384, 1, 1024, 0) == 0
    for bad in ((-1, 1, 16, 16), (4096, 0, 16, 16), (4096, 1, 16, 8), (4096, 1, -16, 16), (1 << 31, 1, 16, 16)):
        assert query(*bad) == 0
    for T in (2048, 5000, 1 << 20, 1 << 26):       # the sums stay below a bound whatever the rows
        for N, K in ((16, 16), (64, 128), (2048, 1024)):
            if T * max(N, K) <= 1 << 33:
                assert query(T, 1, N, K) <= (1 << 28) + 2 * N * K * 4


@pytest.mark.parametrize("kw,status", [
    (dict(K=24), L.E_SHAPE), (dict(N=40), L.E_SHAPE), (dict(E=0), L.E_SHAPE), (dict(out_dt=5), L.E_DTYPE),
    (dict(ends=None), L.E_NULL), (dict(dw=None), L.E_NULL), (dict(dy=None), L.E_NULL), (dict(x=None), L.E_NULL),
    (dict(ws=None), L.E_NULL), (dict(less=1), L.E_ARG), (dict(ws=A + 8), L.E_ALIGN), (dict(dy=A + 8), L.E_ALIGN),
    (dict(x=A + 4), L.E_ALIGN), (dict(dw=A + 8), L.E_ALIGN), (dict(ends=A + 2), L.E_ALIGN), (dict(K=0, dw=None, ws=None), L.OK),
])
def test_split_wgrad_rejects(kw, status):
    a = dict(dy=A, x=A, ends=A, dw=A, out_dt=L.F32, ws=A, less=0, **BIG) | kw
    n = query(a["T"], a["E"], a["N"], a["K"]) - a["less"]
    assert L.lib().nvfp4_grouped_wgrad_split(a["dy"], a["x"], None, a["T"], a["E"], a["N"], a["K"], a["ends"], a["dw"],
                                             a["out_dt"], a["ws"], max(n, 0), None) == status


def test_what_is_no_tensor_is_refused():
    x, w = torch.zeros(4, 64), torch.ones(64)
    for call in (lambda: nv.add_rms_norm(None, w), lambda: nv.add_rms_norm([[1.0]], w), lambda: nv.swiglu_checkpoint(3),
                 lambda: nv.swiglu_backward("x", x, x), lambda: nv.matvec(None, x, x), lambda: nv.matvec(None, x, x, x_scale=x),
                 lambda: nv.grouped_matmul(None, x, x, x), lambda: nv.grouped_wgrad(None, x, x),
                 lambda: nv.add_rms_norm_backward(None, x, w, w)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


def test_the_binding_counts_its_arguments():
    from fp4_block_quantization_nvfp4_amd import _layer

    for name in ("add_rms_norm", "add_rms_norm_backward", "swiglu_checkpoint", "swiglu_backward", "matvec", "grouped_matmul",
                 "grouped_wgrad"):
        with pytest.raises(TypeError, match="arguments expected"):
            getattr(_layer, name)()
        with pytest.raises(TypeError):
            getattr(_layer, name)(x=1)
