"""The layer operators at the sizes where their launch plans change: weight
gradients whose rows are split among workgroups, row counts around the switch
from 16 to 32 rows at a time and from there to row tiles, tiles of either
width, weights a few words wide, long rows of which a workgroup of the norm's
gradient takes several; and the codes of 32-bit rows.  Definitions and tolerances
are those of tests/layer_ref.py and tests/test_gpu_layer.py."""
import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
from fp4_block_quantization_nvfp4_amd import _lib as L
from tests import layer_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_layer import (BF, F32, INF, NAN, check_grouped, check_norm, check_wgrad, gen, randn, rows, split,
                                  weights)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def is_split(T, E, N, K):
    return L.lib().nvfp4_grouped_wgrad_workspace_bytes(T, E, N, K) > 0


@pytest.mark.parametrize("mx8", [False, True], ids=["bf16", "mx8"])
@pytest.mark.parametrize("T,E,N,K", [(4096, 1, 256, 128), (6001, 1, 272, 144), (9000, 3, 64, 272), (5000, 5, 16, 16),
                                     (12345, 2, 528, 48)])
@pytest.mark.parametrize("out", [BF, F32], ids=["out16", "out32"])
def test_wgrad_of_many_rows(T, E, N, K, mx8, out):
    assert is_split(T, E, N, K)
    check_wgrad(T, E, N, K, mx8, out, split(T, T, E, empty=(E // 2,) if E > 2 else ()))


@pytest.mark.parametrize("ends", [[0, 0, 0], [9000, 9000, 9000], [0, 9000, 9000], [10, 20, 9000], [300, 8000, 8001],
                                  [9000, 100, 5], [-4, 70, 90]])
def test_wgrad_of_many_rows_in_any_ranges(ends):
    """Experts without rows, of one block, of many, and rows of none."""
    assert is_split(9000, 3, 80, 96)
    check_wgrad(9000, 3, 80, 96, True, F32, torch.tensor(ends, dtype=torch.int32))


def test_wgrad_of_many_experts_and_rows():
    T, E = 100000, 70
    assert is_split(T, E, 16, 16)
    ends = torch.cat((torch.arange(1, 66), torch.tensor([15000, 15000, 15001, 99999, 100000]))).int()
    check_wgrad(T, E, 16, 16, False, F32, ends)


def test_split_wgrad_repeats_and_stays_in_its_experts():
    """Bit for bit the same on each call; an infinity or NaN spoils its column of
    its own expert alone, whichever block it falls into."""
    T, E, N, K = 9000, 3, 80, 96
    ends = torch.tensor([3000, 3100, 9000], dtype=torch.int32).cuda()
    x, dy = randn(gen(1), T, K).cuda(), randn(gen(2), T, N).cuda()
    want = nv.grouped_wgrad(dy, x, ends)
    assert torch.equal(want, nv.grouped_wgrad(dy, x, ends))
    bad = x.clone()
    bad[2999, 5], bad[8999, K - 1] = NAN, INF
    got = nv.grouped_wgrad(dy, bad, ends)
    assert torch.isnan(got[0, :, 5]).all() and not torch.isfinite(got[2, :, K - 1]).any()
    got[0, :, 5], got[2, :, K - 1] = want[0, :, 5], want[2, :, K - 1]
    assert torch.equal(got, want)


def test_split_wgrad_in_a_graph():
    """The workspace is part of the capture: replays with new inputs, eager work
    between them, equal eager calls."""
    T, E, N, K = 9000, 2, 80, 96
    ends = torch.tensor([7000, 9000], dtype=torch.int32).cuda()
    x, dy = randn(gen(1), T, K).cuda(), randn(gen(2), T, N).cuda()
    nv.grouped_wgrad(dy, x, ends)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = nv.grouped_wgrad(dy, x, ends)
    for i in range(4):
        x.copy_(randn(gen(10 + i), T, K)), dy.copy_(randn(gen(20 + i), T, N))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, nv.grouped_wgrad(dy, x, ends)), i


def test_split_wgrad_workspace_is_checked():
    T, E, N, K = 9000, 2, 80, 96
    lib, need = L.lib(), L.lib().nvfp4_grouped_wgrad_workspace_bytes(T, E, N, K)
    a = 1 << 20  # never dereferenced
    call = lambda ws, n: lib.nvfp4_grouped_wgrad_split(a, a, None, T, E, N, K, a, a, L.F32, ws, n, None)
    assert call(None, need) == L.E_NULL and call(a, need - 1) == L.E_ARG and call(a + 8, need) == L.E_ALIGN


@pytest.mark.parametrize("mx8", [False, True], ids=["bf16", "mx8"])
@pytest.mark.parametrize("blocks", ["1x16", "16x16"])
@pytest.mark.parametrize("T,E,N,K", [(17, 1, 48, 144), (32, 1, 1040, 272), (33, 1, 64, 2064), (95, 1, 272, 528), (96, 1, 16, 16),
                                     (97, 1, 144, 80), (100, 3, 80, 304), (250, 3, 2048, 64), (800, 8, 400, 48)])
def test_rows_around_the_switches(T, E, N, K, mx8, blocks):
    x, xs, xv = rows(T + K, T, K, mx8)
    p, s, a = weights(N, E, N, K, blocks)
    check_grouped(x, xs, xv, split(T, T, E), p, s, a, blocks, F32)


@pytest.mark.parametrize("T", [20, 40, 400])
@pytest.mark.parametrize("N", [16, 32, 48, 80, 272])
@pytest.mark.parametrize("K", [16, 48, 64, 80, 128, 144])
def test_transposed_tiles_of_narrow_weights(T, N, K):
    """Four tiles along n are read as a word: fewer than four, and words that end
    past the last tile."""
    E = 2
    g = torch.Generator(device="cuda").manual_seed(N + K)
    q = []
    for _ in range(E):
        w = (torch.randn(K, N, device="cuda", generator=g) * 0.02).to(BF)
        a = nv.amax(w)
        q.append(nv.quantize_2d(w, a) + (a,))
    _, col, tiles, amax = (torch.stack(t) for t in zip(*q))
    x, xs, xv = rows(T, T, K, False)
    check_grouped(x, xs, xv, split(T, T, E), col, tiles, amax.view(-1), "16x16t", F32)


@pytest.mark.parametrize("T,E,N,K", [(700, 2, 64, 144), (2000, 2, 1040, 80), (9000, 1, 1040, 48), (200, 2, 400, 208)])
def test_row_sums_do_not_depend_on_the_tile(T, E, N, K):
    """The same rows give the same bits in a longer call, whose tiles are wider
    and higher or split."""
    x, _, _ = rows(1, T, K, False)
    p, s, a = weights(2, E, N, K)
    ends = torch.tensor([T // 3, T], dtype=torch.int32).cuda()[-E:]
    ends[-1] = T
    long = torch.cat((x, x, x, x, x, x))
    lends = torch.cat((ends[:-1], ends.new_tensor([6 * T])))
    y, z = nv.grouped_matmul(x, ends, p, s, global_amax=a), nv.grouped_matmul(long, lends, p, s, global_amax=a)
    assert torch.equal(y, z[:T])


# y of 32-bit rows is in 64 bits up to its codes, off by 2^-40 of its value.
# With 8 borders of codes in an octave, about 2^-36 of all values are that near
# to one: of 3 million, 4e-5 may differ.


@pytest.mark.parametrize("H", [2064, 16400])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_codes_of_32_bit_rows_are_exact(H, residual):
    g = gen(H)
    x, r, w = randn(g, 180, H, dtype=F32), randn(g, 180, H, dtype=F32), randn(g, H, dtype=F32)
    codes, scales, hidden, rstd = nv.add_rms_norm(x.cuda(), w.cuda(), r.cuda() if residual else None, eps=2.0 ** -20)
    h = R.f64(x) + R.f64(r) if residual else R.f64(x)
    root = (h.square().mean(1, keepdim=True) + 2.0 ** -20).rsqrt()
    c, s = R.mx8_codes(h * root * R.f64(w))
    assert torch.equal(R.byte(codes), c) and torch.equal(R.byte(scales), s)
    assert torch.equal(hidden.cpu(), h.float())
    assert ((R.f64(rstd) - root[:, 0]).abs() <= root[:, 0] * R.U24).all()


@pytest.mark.parametrize("keep", [False, True])
def test_swiglu_codes_of_32_bit_rows_are_exact(keep):
    x = randn(gen(5), 1500, 4096, dtype=F32, by=3.0)
    codes, scales, _, _ = nv.swiglu_checkpoint(x.cuda(), keep=keep)
    g, u = R.f64(x)[:, :2048], R.f64(x)[:, 2048:]
    c, s = R.mx8_codes(g / (1 + torch.exp(-g)) * u)
    assert torch.equal(R.byte(codes), c) and torch.equal(R.byte(scales), s)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(530, 16400), (300, 32752), (1100, 16384)])
@pytest.mark.parametrize("res", [True, False], ids=["residual", "plain"])
def test_norm_of_many_long_rows(T, H, dtype, res):
    """More rows than workgroups: each sums its share of the weight's gradient."""
    g = gen(T + H)
    x, r = randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype, by=3.0)
    w = 1 + 0.2 * torch.randn(H, generator=g)
    dy, dh = randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype)
    check_norm(x, r if res else None, w, upstream=(dy, dh if res else None))
