"""Every form of the products' kernels (tile sizes, fragments, rows at a time,
scale layouts, row types) at a size that launches it, against the definitions of
tests/layer_ref.py.  The forms that large layers run come first: wide tiles of
128 rows, the weight gradient's wide tile, four fragments.  The launch plan has
to name the form, so that a change of the rules shows here."""
import ctypes

import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
from fp4_block_quantization_nvfp4_amd import _lib as L
from tests import layer_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_layer import BF, F32, check_grouped, check_wgrad, rows, split, weights

pytestmark = pytest.mark.gpu

MATVEC, GROUPED, WGRAD = 4, 5, 6
MX8 = pytest.mark.parametrize("mx8", [False, True], ids=["bf16", "mx8"])
BLOCKS = pytest.mark.parametrize("blocks", ["1x16", "16x16", "16x16t"])


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def plan(entry, T, E, N, K, mx8):
    out = (ctypes.c_int64 * 10)()
    assert L.lib().nvfp4_selftest_layer_plan(entry, T, E, N, K, int(mx8), out) == L.OK
    return list(out[:5])


def ceil(a, b):
    return -(-a // b)


def tile_of(T, E, N, K, mx8):
    """(rows, n's) of k_grouped's tile."""
    kernel, grid, _, _, r = plan(4, T, E, N, K, mx8)
    assert kernel == GROUPED
    widths = [w for w in (128, 256) if grid == 8 * ceil(min(ceil(T, r) + E, T) * ceil(N, w), 8) + (192 if r == 128 else 0)]
    assert len(widths) == 1
    return r, widths[0]


def weight(seed, E, N, K, blocks):
    if blocks != "16x16t":
        return weights(seed, E, N, K, blocks)
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = []
    for _ in range(E):
        w = (torch.randn(K, N, device="cuda", generator=g) * 0.02).to(BF)
        a = nv.amax(w)
        q.append(nv.quantize_2d(w, a) + (a,))
    _, col, tiles, amax = (torch.stack(t) for t in zip(*q))
    return col, tiles, amax.view(-1)


@MX8
@BLOCKS
@pytest.mark.parametrize("T,E,N,K,tile", [
    (2500, 3, 3600, 272, (128, 256)), (2304, 1, 4112, 528, (128, 256)),
    (2048, 32, 1552, 144, (64, 256)), (1100, 16, 2576, 336, (64, 256)),
    (700, 16, 2320, 272, (32, 256)), (900, 40, 1552, 128, (32, 256)),
    (700, 3, 400, 272, (128, 128)), (200, 3, 2576, 400, (64, 128)), (150, 3, 3200, 208, (32, 128))])
def test_grouped_tiles(T, E, N, K, tile, blocks, mx8):
    assert tile_of(T, E, N, K, mx8) == tile
    x, xs, xv = rows(T + K, T, K, mx8)
    p, s, a = weight(N, E, N, K, blocks)
    check_grouped(x, xs, xv, split(T, T, E, empty=(E // 2,) if E > 2 else ()), p, s, a, blocks, BF)


@MX8
@pytest.mark.parametrize("out", [BF, F32], ids=["out16", "out32"])
@pytest.mark.parametrize("T,E,N,K", [(700, 4, 2064, 1936), (300, 2, 4112, 2064)])
def test_wgrad_wide_tile(T, E, N, K, out, mx8):
    kernel, grid, _, _, block = plan(6, T, E, N, K, mx8)
    assert kernel == WGRAD and block == 0 and grid == E * 8 * ceil(ceil(N, 256) * ceil(K, 128), 8)
    check_wgrad(T, E, N, K, mx8, out, split(T, T, E))


def matvec_form(T, E, N, K, mx8):
    kernel, grid, _, _, at_a_time = plan(4 if E else 3, T, max(E, 1), N, K, mx8)
    assert kernel == MATVEC
    frags = [f for f in (1, 2, 4) if grid == ceil(N, 16 * f)]
    assert len(frags) == 1
    return frags[0], at_a_time


# K % 64 == 0: a lane's four scales are a word
@MX8
@BLOCKS
@pytest.mark.parametrize("K", [144, 320])
@pytest.mark.parametrize("T,E,N,form", [(100, 32, 2064, (4, 16)), (128, 8, 2064, (2, 16)), (136, 8, 2048, (2, 32)), (9, 4, 400, (1, 16)),
                                        (150, 4, 400, (1, 32))])
def test_matvec_of_experts(T, E, N, K, form, blocks, mx8):
    assert matvec_form(T, E, N, K, mx8) == form
    x, xs, xv = rows(T + K, T, K, mx8)
    p, s, a = weight(N, E, N, K, blocks)
    check_grouped(x, xs, xv, split(T, T, E), p, s, a, blocks, F32)


@MX8
@pytest.mark.parametrize("blocks", ["1x16", "16x16"])
@pytest.mark.parametrize("K", [80, 192])
@pytest.mark.parametrize("T,N,form", [(1, 65552, (4, 16)), (4, 65552, (4, 16)), (10, 16400, (2, 16)), (20, 16400, (2, 32)), (3, 336, (1, 16)),
                                      (40, 336, (1, 32))])
def test_matvec_alone(T, N, K, form, blocks, mx8):
    assert matvec_form(T, 0, N, K, mx8) == form
    x, xs, xv = rows(T + K, T, K, mx8)
    p, s, a = weight(N, 1, N, K, blocks)
    got = nv.matvec(x, p[0], s[0], x_scale=xs, tile16=blocks != "1x16", global_amax=a, out_dtype=F32)
    w = R.weight_values(p, s, blocks, a)[0]
    y = xv @ w.t()
    R.assert_near(got, y, R.product_bound(xv, w, F32, y), "matvec")
