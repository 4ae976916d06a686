"""The layer operators where their definitions are easy to miss: products without
a k, scale bytes at the ends of the format, rows far from 1, experts that have
nearly all rows.  Definitions are those of tests/layer_ref.py."""
import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
from fp4_block_quantization_nvfp4_amd import _lib as L
from tests import layer_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_layer import BF, F32

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("T,N", [(1, 1), (3, 7), (300, 33), (70001, 129)])
@pytest.mark.parametrize("dt", [L.BF16, L.F32])
@pytest.mark.parametrize("experts", [False, True])
def test_products_without_a_k(T, N, dt, experts):
    """K == 0 writes zeros over all of the output and nothing behind it."""
    size = T * N * (2 if dt == L.BF16 else 4)
    out = torch.full((size + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    p = out.data_ptr()
    assert p % 16 == 0
    if experts:
        ends = torch.tensor([T // 2, T // 2], dtype=torch.int32, device="cuda")
        st = L.lib().nvfp4_grouped_matmul(None, None, T, 2, N, 0, ends.data_ptr(), None, None, 0, None, 0, 448.0, p, dt, stream())
    else:
        st = L.lib().nvfp4_matvec(None, None, T, N, 0, None, None, 0, None, 0, 448.0, p, dt, stream())
    assert st == L.OK
    assert not out[:size].any() and bool((out[size:] == 0x5A).all())
