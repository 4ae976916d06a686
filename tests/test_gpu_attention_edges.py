"""Attention on an NVFP4 cache on the GPU, where a result could pass for another one:
sequences longer than their row of the table."""
import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
from tests.gpu_util import need_gpu
from tests.test_gpu_attention import filled, gen, randn, tables

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------- longer than the table's row


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hk,D,n,L", [(4, 2, 64, 60, 60), (2, 2, 128, 100, 100), (4, 2, 64, 100, 100), (8, 2, 128, 70, 5000), (16, 2, 256, 90, 90),
                                         (4, 2, 96, 200, 17), (4, 2, 64, 40, 33)])
def test_longer_than_the_row(Hq, Hk, D, n, L, causal):
    """A row of one page for more keys than it holds: every query of that sequence gets NaN, those too that the keys in the
    page would leave without any (60 queries of 4 heads on 2 go to the split kernel, 100 to the tiled one); the sequences
    beside it are as without it."""
    g = gen(n + D)
    c = filled(g, 5, 16, Hk, D)
    table = torch.tensor([[2], [0], [4]], dtype=torch.int32).cuda()
    ends, T = ints(9, 9 + n, 9 + n + 12), n + 21
    q = randn(g, T, Hq, D).cuda()
    out, lse = nv.cache_attention(q, c, table, ints(16, L, 11), ends, causal=causal)
    mine = slice(9, 9 + n)
    if L > 16:
        assert torch.isnan(out[mine]).all() and torch.isnan(lse[mine]).all()
    want, wl = nv.cache_attention(q, c, table, ints(16, 16, 11), ends, causal=causal)
    for at in (slice(0, 9), slice(9 + n, T)):
        assert torch.isfinite(out[at]).all() and torch.equal(out[at], want[at]) and torch.equal(lse[at], wl[at])


def test_longer_than_the_row_among_many():
    """Rows of several pages, in parts that are joined."""
    g = gen(40)
    table, pages = tables(g, [640, 640], 64)
    c = filled(g, pages, 64, 2, 128)
    n = 700
    q = randn(g, 2 * n, 4, 128).cuda()
    out, lse = nv.cache_attention(q, c, table.cuda(), ints(640, 641), ints(n, 2 * n))
    assert torch.isnan(out[n:]).all() and torch.isnan(lse[n:]).all()
    assert (out[:60] == 0).all() and (lse[:60] == -INF).all() and torch.isfinite(out[60:n]).all() and torch.isfinite(lse[60:n]).all()
