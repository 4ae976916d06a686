"""Launch geometry of the layer operators, without a GPU: every launch of every
accepted shape stays inside the dispatch limits, covers its rows and columns, and
the grids of the grouped kernels hold every unit of work for any row ranges."""
import ctypes
import random

import pytest

from fp4_block_quantization_nvfp4_amd import _lib as L

NORM, NORM_BWD, SUM_ROWS, SWIGLU, MATVEC, GROUPED, WGRAD, JOIN, ZERO = range(9)
MOST = 1 << 33
SLOTS = 512


def plan(entry, T, E=1, N=16, K=16, mx8=0):
    out = (ctypes.c_int64 * 10)()
    st = L.lib().nvfp4_selftest_layer_plan(entry, T, E, N, K, mx8, out)
    return st, list(out[:5]), list(out[5:])


def check_limits(launch, what):
    _, x, y, lanes, _ = launch
    assert x >= 1 and y >= 1 and 64 <= lanes <= 1024 and lanes % 64 == 0, (what, launch)
    assert x < 1 << 31 and x * lanes < 1 << 32 and y <= 65535, (what, launch)


def ceil(a, b):
    return -(-a // b)


@pytest.mark.parametrize("entry", [0, 1])
def test_norm_launches(entry):
    for H in (16, 32, 1024, 1040, 7168, 16384, 16400, 32768):
        for T in (1, 2, 255, 513, 1 << 20, MOST // H):
            if T >= 1 << 31 or T * H > MOST:
                continue
            st, a, b = plan(entry, T, K=H)
            assert st == L.OK and a[0] == (NORM_BWD if entry else NORM)
            check_limits(a, (T, H))
            assert a[3] * (16 if H <= 16384 else 32) >= H and a[1] <= T
            if entry:
                check_limits(b, (T, H))
                assert b[0] == SUM_ROWS and b[1] * 16 == H
                assert L.lib().nvfp4_add_rms_norm_backward_workspace_bytes(T, H) == a[1] * H * 4


def test_swiglu_launches():
    for F in (16, 32, 48, 8192, 1 << 20, 1 << 32):
        for T in (1, 3, 1 << 20, MOST // (2 * F)):
            if T * 2 * F > MOST:
                continue
            st, a, _ = plan(2, T, K=F)
            assert st == L.OK and a[0] == SWIGLU
            check_limits(a, (T, F))
            assert a[1] * a[3] >= T * ceil(F, 32) * 2 and T * ceil(F, 32) * 2 + a[3] < 1 << 32


def products():
    """Accepted (T, E, N, K), the extremes of each among them."""
    top = (1 << 31) - 1
    got = [(top, 1, 1, 0), (top, 1, 4, 0), (top, 2, 4, 0), (1 << 30, 65534, 8, 0), (1 << 29, 1, 16, 16), (1 << 29, 65534, 16, 16),
           (1, 65534, 1 << 13, 16), (1 << 20, 65534, 1 << 13, 16), (1 << 13, 1, 1 << 20, 16), (1 << 13, 8, 1 << 20, 1 << 10),
           (1 << 13, 1, 16, 1 << 20), (1 << 13, 512, 16, 1 << 20), (1 << 20, 1, 1 << 13, 1 << 13)]
    r = random.Random(3)
    while len(got) < 400:
        T, E, N = (int(2 ** r.uniform(0, top)) for top in (30, 16, 20))
        K = 16 * int(2 ** r.uniform(0, 16))
        if E <= 65534 and T * N <= MOST and T * K <= MOST and E * N * K <= MOST:
            got.append((T, E, N, K))
    return got


@pytest.mark.parametrize("entry", [3, 4])
@pytest.mark.parametrize("mx8", [0, 1])
def test_product_launches(entry, mx8):
    for T, E, N, K in products():
        st, a, _ = plan(entry, T, E, N, K, mx8)
        assert st == L.OK, (T, E, N, K)
        check_limits(a, (T, E, N, K))
        if K == 0:
            assert a[0] == ZERO
            continue
        # 32-bit row numbers, a tile added: no overflow
        assert T + max(a[4], 128) < 1 << 31
        if a[0] == MATVEC:
            assert any(a[1] == ceil(N, 16 * f) for f in (1, 2, 4))
        else:
            assert a[0] == GROUPED and a[4] in (32, 64, 128)


def blocks_of(units, split):
    """Workgroups up to the last that has work (unit_of_block in nvfp4_experts.hpp)."""
    over = units % SLOTS if split else 0
    parts = 4 if over * 8 <= SLOTS else 2 if over * 4 <= SLOTS else 1
    whole = units - (over if parts > 1 else 0)
    n = 8 * ceil(whole, 8)
    if split and parts > 1 and over:
        n += 8 * ceil(over * parts, 8)
    return n


def ranges(rng, T, E):
    """Row counts of E experts and of none, as full of short tiles as they come."""
    kind = rng.randrange(4)
    if kind == 0:
        cuts = sorted(rng.randint(0, T) for _ in range(E))
    elif kind == 1:  # a row each, the rest in one
        cuts = [min(T, i + 1) for i in range(E)]
    elif kind == 2:
        tile = rng.choice((32, 64, 128))
        cuts = [min(T, i * tile + i + 1) for i in range(E)]
    else:
        cuts = [T if i >= E // 2 else 0 for i in range(E)]
    ends = [0] + cuts + [T]
    return [b - a for a, b in zip(ends, ends[1:])]


def test_grouped_grids_hold_every_unit():
    rng = random.Random(5)
    seen = set()
    for _ in range(4000):
        E = rng.choice((0, 1, 2, 3, 8, 63, 64, 130))
        T, N = int(2 ** rng.uniform(0, 16)), int(2 ** rng.uniform(0, 13))
        st, a, _ = plan(4 if E else 3, T, max(E, 1), N, 64)
        if a[0] != GROUPED:
            continue
        tiles = sum(ceil(n, a[4]) for n in (ranges(rng, T, E) if E else [T]))
        # the launcher's width is not reported: the narrow one is the larger grid, and the grid tells which
        for width in (128, 256):
            need = blocks_of(tiles * ceil(N, width), a[4] == 128)
            bound = 8 * ceil(min(ceil(T, a[4]) + E, T) * ceil(N, width), 8) + (SLOTS * 3 // 8 if a[4] == 128 else 0)
            if a[1] == bound:
                seen.add((a[4], width))
                assert need <= a[1], (T, E, N, a, need)
    assert len(seen) == 6


def test_matvec_workgroups_have_few_tiles_each():
    """Whatever the experts' rows, tiles of 16 rows are at most two a workgroup,
    of 32 rows four."""
    rng = random.Random(9)
    seen = set()
    for _ in range(2000):
        E, N = rng.choice((1, 2, 8, 63, 64, 130, 1000)), int(2 ** rng.uniform(0, 13))
        T = int(2 ** rng.uniform(0, 16))
        st, a, _ = plan(4, T, E, N, 64)
        if a[0] != MATVEC:
            continue
        seen.add(a[4])
        tiles = sum(ceil(n, a[4]) for n in ranges(rng, T, E))
        assert ceil(tiles, a[2]) <= (2 if a[4] == 16 else 4), (T, E, N, a, tiles)
    assert seen == {16, 32}


def test_wgrad_launches_and_workspace():
    rng = random.Random(6)
    splits = 0
    for T, E, N, K in products() + [(int(2 ** rng.uniform(10, 17)), rng.choice((1, 2, 5, 70)), 16 * rng.randint(1, 64), 16 * rng.randint(1, 32))
                                    for _ in range(300)]:
        N = N // 16 * 16
        if N == 0 or K == 0:
            continue
        st, a, _ = plan(5, T, E, N, K)
        assert st == L.OK and a[0] == WGRAD
        check_limits(a, (T, E, N, K))
        assert a[1] % (8 * E) == 0 and any(a[1] // E == 8 * ceil(ceil(N, w) * ceil(K, 128), 8) for w in (128, 256))
        st, a, b = plan(6, T, E, N, K)
        check_limits(a, (T, E, N, K))
        ws = L.lib().nvfp4_grouped_wgrad_workspace_bytes(T, E, N, K)
        assert (ws > 0) == (b[1] > 0)
        if not ws:
            continue
        splits += 1
        check_limits(b, (T, E, N, K))
        assert b[0] == JOIN and b[2] == E
        tiles, block = ceil(N, 256) * ceil(K, 128), a[4]
        for _ in range(5):
            blocks = [ceil(n, block) for n in ranges(rng, T, E)]
            assert blocks_of(sum(blocks) * tiles, False) <= a[1]
            assert sum(blocks[:-1]) * N * K * 4 <= ws  # the blocks of experts are the workspace's
    assert splits > 50


def test_plan_refusals():
    assert plan(7, 16)[0] == L.E_ARG and plan(-1, 16)[0] == L.E_ARG
    assert plan(0, 16, K=24)[0] == L.E_SHAPE and plan(0, 16, K=32784)[0] == L.E_RANGE
    assert plan(4, 16, 0)[0] == L.E_SHAPE and plan(5, 16, 1, 24, 16)[0] == L.E_SHAPE
    assert plan(3, 1 << 31)[0] == L.E_RANGE and plan(2, 1 << 20, K=8192)[0] == L.E_RANGE
    assert L.lib().nvfp4_selftest_layer_plan(0, 16, 1, 16, 16, 0, None) == L.E_NULL


# (E, N, rows in all) and the kernel that was the faster one there, by 5% or more
# on rows that differ from expert to expert; with k from 512 to 8192
MEASURED = [(8, 2048, 128, MATVEC), (8, 2048, 160, MATVEC), (8, 2048, 256, GROUPED), (8, 2048, 384, GROUPED), (6, 1024, 192, MATVEC),
            (6, 1024, 576, GROUPED), (4, 1040, 256, MATVEC), (4, 1040, 384, MATVEC), (16, 1024, 320, MATVEC), (32, 512, 544, MATVEC),
            (32, 512, 1024, GROUPED), (32, 512, 2048, GROUPED), (64, 2048, 1088, GROUPED), (64, 2048, 2048, GROUPED), (1, 4096, 96, MATVEC),
            (1, 16384, 32, MATVEC), (1, 1024, 96, MATVEC), (32, 4096, 64, MATVEC), (16, 4096, 192, MATVEC), (8, 4096, 96, MATVEC)]


@pytest.mark.parametrize("E,N,T,kernel", MEASURED)
def test_products_take_the_kernel_that_was_faster(E, N, T, kernel):
    assert plan(4, T, E, N, 2048)[1][0] == kernel
