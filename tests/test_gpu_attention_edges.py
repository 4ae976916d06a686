"""Attention on an NVFP4 cache on the GPU, where a result could pass for another one:
sequences longer than their row of the table, scores that are not finite or very large, many
sequences at a time, one in as many pieces as there may be, no pages and the largest."""
import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
from tests import attention_ref as A
from tests import layer_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_attention import check_attention, filled, gen, randn, tables

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


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


# ------------------------------------------------- scores that are not finite


def one_sign(page, pages, Hk, D):
    """Keys that are all positive."""
    g = gen(41)
    c = filled(g, pages, page, Hk, D)
    c.k.copy_(torch.tensor([0x12, 0x34, 0x56, 0x71], dtype=torch.uint8)[torch.randint(0, 4, c.k.shape, generator=g)])
    return c


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n,L", [(1, 1), (3, 40), (20, 300), (5, 3000), (80, 80), (80, 30), (300, 900), (130, 5000)])
def test_scores_that_are_all_minus_infinity(D, n, L):
    """-inf for every key that a query sees: exp(-inf + inf) is NaN, and 0 is only for queries that see none."""
    c = one_sign(64, -(-L // 64) + 1, 2, D)
    table = torch.arange(-(-L // 64), dtype=torch.int32).view(1, -1).cuda()
    q = randn(gen(n), n, 4, D)
    want, wl = nv.cache_attention(q.cuda(), c, table, ints(L), ints(n))
    first = max(n - L, 0)  # the queries before see no key
    row = (first + n) // 2
    q[row, 1, 3] = -INF
    out, lse = nv.cache_attention(q.cuda(), c, table, ints(L), ints(n))
    assert torch.isnan(out[row, 1]).all() and torch.isnan(lse[row, 1])
    assert (out[:first] == 0).all() and (lse[:first] == -INF).all()
    keep = torch.ones(n, 4, dtype=torch.bool)
    keep[row, 1] = False
    assert torch.equal(out[keep.cuda()], want[keep.cuda()]) and torch.equal(lse[keep.cuda()], wl[keep.cuda()])
    if first:
        q[0, 2, 5] = -INF  # sees no key
        out, lse = nv.cache_attention(q.cuda(), c, table, ints(L), ints(n))
        assert (out[:first] == 0).all() and (lse[:first] == -INF).all()


@pytest.mark.parametrize("what", ["k_amax", "v_amax"])
@pytest.mark.parametrize("n,L,D", [(20, 7, 64), (40, 33, 128), (90, 50, 128), (200, 180, 256), (700, 600, 64)])
def test_amax_that_is_nan(n, L, D, what):
    """A NaN second-level scale reaches the queries of its head that see a key, and no other."""
    g = gen(42)
    c = filled(g, -(-L // 64), 64, 2, D)
    table = torch.arange(-(-L // 64), dtype=torch.int32).view(1, -1).cuda()
    q = randn(g, n, 4, D).cuda()
    want, wl = nv.cache_attention(q, c, table, ints(L), ints(n))
    getattr(c, what)[1] = NAN
    out, lse = nv.cache_attention(q, c, table, ints(L), ints(n))
    first = n - L
    assert torch.equal(out[:, :2], want[:, :2]) and torch.equal(lse[:, :2], wl[:, :2])
    assert (out[:first] == 0).all() and (lse[:first] == -INF).all()
    assert torch.isnan(out[first:, 2:]).all() and (what == "v_amax" or torch.isnan(lse[first:, 2:]).all())


@pytest.mark.parametrize("by", [1e4, 1e6, 1e8, 1e12, 1e20, 1e30])
@pytest.mark.parametrize("n,L,D", [(1, 2000, 64), (3, 500, 128), (70, 2000, 128), (150, 700, 64), (90, 300, 256), (16, 40000, 128)])
def test_very_large_scores(n, L, D, by):
    """Scores far past 2^24, finite: all the weight is on the largest one (or on those within the rounding of a score)."""
    g = gen(43)
    table, pages = tables(g, [L], 64)
    c = filled(g, pages, 64, 1, D, amax=False)
    check_attention(randn(g, n, 4, D, by=by).cuda(), c, table, [L], [n], True, what=f"by {by}")
    # keys of twos, but one of threes: far ahead of the others
    c.k.fill_(0x44), c.k_scale.fill_(0x38)
    q = torch.full((n, 4, D), by).bfloat16()
    j = L // 3
    c.k[table[0, j // 64], 0, j % 64] = 0x55
    out, lse = nv.cache_attention(q.cuda(), c, table.cuda(), ints(L), ints(n), causal=False)
    value = A.cache_values(c.v, c.v_scale)[table[0, j // 64].item(), 0, j % 64]
    score = R.f64(q)[0, 0, 0] * 3 * D * D ** -0.5
    # the weight of all the others is 0; the result's rounding, and the weight's own: 2^-11
    R.assert_near(out, value.expand(n, 4, D), value.abs().expand(n, 4, D) * (2.0 ** -8 + 2.0 ** -11) + 1e-30, "the largest")
    R.assert_near(lse, score.expand(n, 4), score.expand(n, 4) * 2.0 ** -20, "its score")


# ------------------------------------------------- many sequences, many pieces


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128])
def test_many_sequences_of_many_rows(D, causal):
    """More sequences than are scanned at a time (256), some of more rows than the split kernel takes on both sides of that
    border and at it, a few of them long enough for their keys to be shared by workgroups; some without queries or keys."""
    g = gen(44)
    B = 310
    n = torch.randint(0, 4, (B,), generator=g)
    lens = torch.randint(0, 90, (B,), generator=g)
    for b in (0, 3, 100, 254, 255, 256, 257, 300, 309):
        n[b] = 66 + b % 7
        lens[b] = 1900 if b in (3, 255, 256, 309) else 75 + b % 50
    n[20:30], lens[40:45] = 0, 0
    table, pages = tables(g, lens.tolist(), 32)
    c = filled(g, pages, 32, 1, D)
    ends = torch.cumsum(n, 0)
    check_attention(randn(g, int(ends[-1]) + 5, 2, D).cuda(), c, table, lens.tolist(), ends.tolist(), causal)


@pytest.mark.parametrize("lens", [[70000], [70000, 3], [1, 0, 40000, 129, 33000]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_unit_in_as_many_pieces_as_there_may_be(lens, D):
    """One head of keys, so long that pieces of an even cut would be more than the 512 that a unit may lie in."""
    g = gen(45)
    table, pages = tables(g, lens, 256)
    c = filled(g, pages, 256, 1, D)
    check_attention(randn(g, len(lens), 4, D).cuda(), c, table, lens, None, True)


# ------------------------------------------------- the smallest and the largest


def test_a_cache_without_pages():
    """Nothing is written, zeros are read, and sequences have no keys, or NaN for keys of pages that are not there."""
    c = nv.PagedCache.empty(0, 16, 2, 64)
    x = torch.ones(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    nv.write_cache(c, x, x, ints(0, 1, -1, 1 << 20))
    for t in nv.read_cache(c, ints(0, 5, -1)):
        assert t.shape == (3, 2, 64) and (t == 0).all()
    table = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    out, lse = nv.cache_attention(x, c, table, ints(0, 3, 0, 32))
    assert (out[::2] == 0).all() and (lse[::2] == -INF).all() and torch.isnan(out[1::2]).all() and torch.isnan(lse[1::2]).all()
    many = torch.ones(90, 4, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = nv.cache_attention(many, c, table[:2], ints(0, 30), ints(40, 90), causal=False)
    assert (out[:40] == 0).all() and (lse[:40] == -INF).all() and torch.isnan(out[40:]).all() and torch.isnan(lse[40:]).all()


@pytest.mark.parametrize("n", [1, 70])
def test_the_largest_pages(n):
    """65536 slots a page, a sequence that goes on in a second one."""
    g = gen(46)
    lens = [65536 + 200, 65535]
    table, pages = tables(g, lens, 65536)
    c = filled(g, pages, 65536, 2, 32)
    ends = None if n == 1 else [n, 2 * n]
    check_attention(randn(g, 2 * n, 4, 32).cuda(), c, table, lens, ends, True)


def test_many_heads_of_keys():
    g = gen(47)
    lens = [5, 0, 33, 70]
    table, pages = tables(g, lens, 16)
    c = filled(g, pages, 16, 1000, 32)
    check_attention(randn(g, 4, 1000, 32).cuda(), c, table, lens, None, True)
    check_attention(randn(g, 140, 1000, 32).cuda(), c, table, lens, [1, 60, 100, 139], True)
