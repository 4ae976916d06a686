"""The layer operators on the GPU against their definitions in 64 bits
(tests/layer_ref.py): both directions, types, odd and empty sizes, rows and
scales that are not finite, row ranges of any kind, other streams, replays of
a captured step.  Tolerances count the roundings that the definitions allow;
each is derived where it is used."""
import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
from tests import layer_ref as R
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=BF, by=1.0):
    return (torch.randn(*shape, generator=g) * by).to(dtype)


# ------------------------------------------------------------------ norm

# sum of H squares in fp32: 32 in a lane's chain, 6 + 16 joins, the mean, eps,
# the root and the reciprocal: below 64 roundings of positive terms
NORM_REL = 64 * R.U24


def check_norm(x, r, w, eps=1e-6, upstream=None):
    cuda = lambda t: None if t is None else t.cuda()
    codes, scales, hidden, rstd = nv.add_rms_norm(x.cuda(), w.cuda(), cuda(r), eps=eps)
    T, H = x.shape
    assert codes.dtype == R.F8 and codes.shape == (T, H) and scales.dtype == R.E8 and scales.shape == (T, (H + 31) // 32)
    assert hidden.dtype == x.dtype and rstd.dtype == F32
    h = R.f64(x) if r is None else R.f64(x) + R.f64(r)
    want = 1 / torch.sqrt((h * h).sum(1) / H + eps)
    R.assert_near(rstd, want, want * NORM_REL, "rstd")
    R.assert_near(hidden, h, h.abs() * (R.half_step(x.dtype) + 2 * R.U24), "hidden")
    R.assert_mx8(codes, scales, h * want[:, None] * R.f64(w), NORM_REL + 4 * R.U24, "norm")
    if upstream is None:
        return
    dy, dh = upstream
    dx, dw = nv.add_rms_norm_backward(dy.cuda(), hidden, w.cuda(), rstd, cuda(dh))
    hid, s = R.f64(hidden), R.f64(rstd)
    gx, gw = R.norm_gradient(R.f64(dy), hid, R.f64(w), s, None if dh is None else R.f64(dh))
    n, d = hid * s[:, None], R.f64(dy) * R.f64(w)
    # the row's mean of d n is off by at most 64 roundings of the mean magnitude,
    # the rest of the formula by fewer than 16 of each term's
    size = s[:, None] * (d.abs() + n.abs() * (d * n).abs().mean(1, keepdim=True))
    extra = 0 if dh is None else R.f64(dh).abs()
    R.assert_near(dx, gx, gx.abs() * R.half_step(dy.dtype) + 80 * R.U24 * (size + extra), "dx")
    # T terms, each of two roundings, summed in some order
    R.assert_near(dw, gw, (T + 8) * R.U24 * (R.f64(dy) * n).abs().sum(0) + 1e-37, "dweight")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 16), (1, 7168), (3, 48), (5, 1040), (17, 4096), (2, 16384), (2, 16400), (3, 32768),
                                 (1500, 64), (130, 2064)])
@pytest.mark.parametrize("res", [True, False], ids=["residual", "plain"])
def test_norm(T, H, dtype, res):
    g = gen(T * H)
    x, r = randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype, by=3.0)
    w = 1 + 0.2 * torch.randn(H, generator=g)
    dy, dh = randn(g, T, H, dtype=dtype), randn(g, T, H, dtype=dtype)
    check_norm(x, r if res else None, w, upstream=(dy, dh if res else None))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_norm_wide_range_and_zero_rows(dtype):
    g = gen(3)
    x = randn(g, 12, 272, dtype=F32) * torch.exp2(torch.randint(-30, 30, (12, 272), generator=g).float())
    x[4] = 0.0  # a row of zeros: rstd = eps^(-1/2), codes 0 under the smallest scale
    x[5, 32:64] = 0.0
    x[6] *= 2.0 ** -60
    w = torch.randn(272, generator=g) * torch.exp2(torch.randint(-20, 20, (272,), generator=g).float())
    check_norm(x.to(dtype), torch.zeros(12, 272, dtype=dtype), w, upstream=(randn(g, 12, 272, dtype=dtype), None))


def test_norm_rows_that_are_not_finite():
    """An infinity or a NaN stays in its own row: rstd is 0 or NaN there, as 1
    over the root of infinity or NaN, and the other rows are as without it."""
    g = gen(4)
    x, w = randn(g, 6, 96), torch.ones(96)
    x[1, 5], x[3, 90], x[4, 0] = INF, NAN, -INF
    codes, scales, _, rstd = nv.add_rms_norm(x.cuda(), w.cuda())
    keep = [0, 2, 5]
    clean = nv.add_rms_norm(x[keep].cuda(), w.cuda())
    assert torch.equal(R.byte(codes)[keep], R.byte(clean[0])) and torch.equal(R.byte(scales)[keep], R.byte(clean[1]))
    assert rstd[1] == 0 and rstd[4] == 0 and torch.isnan(rstd[3])
    v = R.mx8_values(R.byte(codes), R.byte(scales))
    assert torch.isnan(v[1, 5]) and torch.isnan(v[4, 0]) and torch.isnan(v[3]).all()
    assert (v[1, :5] == 0).all() and (v[1, 6:] == 0).all()


def test_norm_gradient_against_differences():
    g = gen(8)
    T, H = 4, 512
    x, r, dy = (randn(g, T, H, dtype=F32) for _ in range(3))
    w = 1 + 0.1 * torch.randn(H, generator=g)
    _, _, hidden, rstd = nv.add_rms_norm(x.cuda(), w.cuda(), r.cuda())
    dx, dw = nv.add_rms_norm_backward(dy.cuda(), hidden, w.cuda(), rstd)

    def loss(x, w):
        h = x + R.f64(r)
        return ((h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6)) * w * R.f64(dy)).sum()

    for _ in range(3):
        a, b = torch.randn(T, H, dtype=torch.float64, generator=g), torch.randn(H, dtype=torch.float64, generator=g)
        e = 1e-5
        slope = (loss(R.f64(x) + e * a, R.f64(w) + e * b) - loss(R.f64(x) - e * a, R.f64(w) - e * b)) / (2 * e)
        got = (R.f64(dx) * a).sum() + (R.f64(dw) * b).sum()
        # fp32 gradients: 100 roundings of the terms' magnitudes; differences: e^2
        size = (R.f64(dx).abs() * a.abs()).sum() + (R.f64(dw).abs() * b.abs()).sum()
        assert abs(got - slope) <= 100 * R.U24 * size + 1e-6


# ---------------------------------------------------------------- swiglu

SIG_REL = 16 * R.U24  # exponent's product with its correction, 2^x, the sum, the reciprocal: a few units each


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,F", [(1, 16), (1, 8192), (3, 48), (7, 1040), (16, 2048), (300, 176)])
def test_swiglu(T, F, dtype):
    g = gen(T + F)
    x, d = randn(g, T, 2 * F, dtype=dtype, by=2.0), randn(g, T, F, dtype=dtype)
    check_swiglu(x, d)


def check_swiglu(x, d):
    T, F = d.shape
    codes, scales, kept, ks = nv.swiglu_checkpoint(x.cuda())
    plain = nv.swiglu_checkpoint(x.cuda(), keep=False)
    assert plain[2] is None and plain[3] is None
    assert torch.equal(R.byte(codes), R.byte(plain[0])) and torch.equal(R.byte(scales), R.byte(plain[1]))
    gate, up = R.f64(x)[:, :F], R.f64(x)[:, F:]
    y = gate / (1 + torch.exp(-gate)) * up
    R.assert_mx8(codes, scales, y, SIG_REL + 4 * R.U24, "swiglu")
    for part, name in ((0, gate), (1, up)):  # the checkpoint is an exact function of the inputs
        wc, wsc = R.mx8_codes(name)
        G = (F + 31) // 32
        gc, gs = R.byte(kept)[:, part * F:part * F + F], R.byte(ks)[:, part * G:part * G + G]
        assert torch.equal(gs, wsc)
        v, u = R.mx8_values(gc, gs), R.mx8_values(wc, wsc)
        assert torch.equal(v.nan_to_num(1e300), u.nan_to_num(1e300))
    got = nv.swiglu_backward(d.cuda(), kept, ks)
    assert got.dtype == d.dtype
    v = R.mx8_values(R.byte(kept)[:, :F], R.byte(ks)[:, :(F + 31) // 32])
    u = R.mx8_values(R.byte(kept)[:, F:], R.byte(ks)[:, (F + 31) // 32:])
    dg, du = R.swiglu_gradient(R.f64(d), v, u)
    s = 1 / (1 + torch.exp(-v))
    # 1 + g (1 - s) can cancel: its terms' magnitudes count; 1 - s is off by a unit of 1
    size = R.f64(d).abs() * u.abs() * s * (1 + v.abs() * (1 - s) + v.abs() * 4 * R.U24)
    most = dg.abs() * R.half_step(d.dtype) + (SIG_REL + 8 * R.U24) * size
    R.assert_near(got[:, :F], dg, most + v.abs() * 16 * R.U24 * R.f64(d).abs() * u.abs() * s + 1e-37, "dgate")
    R.assert_near(got[:, F:], du, du.abs() * (R.half_step(d.dtype) + SIG_REL + 8 * R.U24) + 1e-37, "dup")


def test_swiglu_wide_range():
    g = gen(11)
    x = randn(g, 9, 160, dtype=F32) * torch.exp2(torch.randint(-40, 6, (9, 160), generator=g).float())
    x[0, :80] = torch.linspace(-85.0, 85.0, 80)
    x[1, 80:] = 0.0
    check_swiglu(x, randn(g, 9, 80, dtype=F32))


def test_swiglu_values_that_are_not_finite():
    x = torch.ones(3, 64)
    x[0, 3], x[1, 40], x[2, 0] = NAN, INF, -INF  # -inf * sigmoid(-inf) = -inf * 0
    codes, scales, kept, ks = nv.swiglu_checkpoint(x.cuda())
    v = R.mx8_values(R.byte(codes), R.byte(scales))
    assert torch.isnan(v[0, 3]) and torch.isnan(v[1, 8]) and torch.isnan(v[2, 0]) and int(torch.isnan(v).sum()) == 3
    k = R.mx8_values(torch.cat((R.byte(kept)[:, :32], R.byte(kept)[:, 32:]), 1), R.byte(ks))
    assert int(torch.isnan(k).sum()) == 3 and (k[~torch.isnan(k)] == 1).all()
    big = torch.full((1, 32), 3.0, dtype=F32)
    big[0, :16] = torch.tensor([-3e38, -200.0, -104.0, -90.0, 90.0, 200.0, 3e30, 0.0] * 2)
    c, s, _, _ = nv.swiglu_checkpoint(big.cuda())
    got = R.mx8_values(R.byte(c), R.byte(s))
    assert torch.isfinite(got).all() and got[0, 0] == 0 and got[0, 7] == 0


# -------------------------------------------------------------- products

def weights(seed, E, N, K, blocks="1x16", amax="tensor", scale=0.02):
    """4-bit weights as the library's own producers write them, on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    packed, scales, amaxes = [], [], []
    for _ in range(E):
        w = (torch.randn(N, K, device="cuda", generator=g) * scale).to(BF)
        if amax == "row":
            p, s, a = nv.quantize_4over6(w, None, e4m3_scale_bound=448, row_scaled=True)
        elif blocks == "1x16":
            a = nv.amax(w) if amax == "tensor" else None
            p, s = nv.quantize(w * (1 if a is not None else 20), global_amax=a)
        else:
            a = nv.amax(w) if amax == "tensor" else None
            p, _, s = nv.quantize_2d(w * (1 if a is not None else 20), a, columnwise=False)
        packed.append(p), scales.append(s), amaxes.append(a)
    am = None if amax == "none" else torch.cat(amaxes)
    return torch.stack(packed), torch.stack(scales), am


def rows(seed, T, K, mx8):
    g = gen(seed)
    x = torch.randn(T, K, generator=g) * (0.5 + 1.5 * torch.rand(T, 1, generator=g))
    if not mx8:
        x = x.to(BF)
        return x.cuda(), None, R.f64(x)
    c, s = R.mx8_codes(x.double())
    codes, scales = c.to(torch.uint8).view(R.F8), s.to(torch.uint8).view(R.E8)
    return codes.cuda(), scales.cuda(), R.mx8_values(c, s)


@pytest.mark.parametrize("mx8", [False, True], ids=["bf16", "mx8"])
@pytest.mark.parametrize("T,N,K", [(1, 16, 16), (1, 1, 32), (2, 100, 48), (5, 1001, 2064), (16, 256, 4096), (16, 37, 7168),
                                   (1, 4096, 272), (17, 33, 144), (40, 515, 400), (130, 300, 1040)])
@pytest.mark.parametrize("amax", ["none", "tensor", "row"])
@pytest.mark.parametrize("out", [BF, F32], ids=["out16", "out32"])
def test_matvec(T, N, K, mx8, amax, out):
    x, xs, xv = rows(N + K, T, K, mx8)
    p, s, a = weights(T + K, 1, N, K, "1x16", amax)
    got = nv.matvec(x, p[0], s[0], x_scale=xs, global_amax=a, row_scaled=amax == "row", out_dtype=out)
    w = R.weight_values(p, s, "1x16", a)[0]
    y = xv @ w.t()
    assert got.dtype == out
    R.assert_near(got, y, R.product_bound(xv, w, out, y), "matvec")


@pytest.mark.parametrize("mx8", [False, True], ids=["bf16", "mx8"])
@pytest.mark.parametrize("T,N,K", [(1, 16, 16), (16, 4112, 528), (3, 18432, 80), (100, 272, 656)])
@pytest.mark.parametrize("amax", ["none", "tensor"])
def test_matvec_tiles(T, N, K, mx8, amax):
    x, xs, xv = rows(N + K, T, K, mx8)
    p, s, a = weights(T, 1, N, K, "16x16", amax)
    got = nv.matvec(x, p[0], s[0], x_scale=xs, tile16=True, global_amax=a, out_dtype=F32)
    w = R.weight_values(p, s, "16x16", a)[0]
    y = xv @ w.t()
    R.assert_near(got, y, R.product_bound(xv, w, F32, y), "matvec")


def check_grouped(x, xs, xv, ends, p, s, a, blocks, out, row_scaled=False, what="grouped"):
    T, E = xv.shape[0], p.shape[0]
    got = nv.grouped_matmul(x, ends.cuda(), p, s, x_scale=xs, tile16=blocks != "1x16", transposed_tiles=blocks == "16x16t",
                            global_amax=a, row_scaled=row_scaled, out_dtype=out)
    w = R.weight_values(p, s, blocks, a)
    c = R.cuts(ends, T)
    y, most = torch.zeros(T, w.shape[1], dtype=torch.float64), torch.zeros(T, w.shape[1], dtype=torch.float64)
    for e in range(E):
        r = slice(c[e], c[e + 1])
        y[r] = xv[r] @ w[e].t()
        most[r] = R.product_bound(xv[r], w[e], out, y[r])
    R.assert_near(got, y, most, what)  # rows of no expert: exactly zero
    return got


def split(seed, T, E, empty=()):
    g = gen(seed)
    share = torch.rand(E, generator=g) ** 2 + 0.05
    share[list(empty)] = 0
    cut = (torch.cumsum(share, 0) / share.sum() * T).round().to(torch.int32)
    cut[-1] = T
    return cut


SIZES = [(1, 1, 16, 16), (3, 2, 16, 16), (64, 32, 272, 144), (40, 3, 96, 272), (200, 2, 272, 400), (777, 5, 1040, 528),
         (300, 1, 512, 2064), (1500, 3, 256, 128), (513, 9, 640, 112)]


@pytest.mark.parametrize("mx8", [False, True], ids=["bf16", "mx8"])
@pytest.mark.parametrize("T,E,N,K", SIZES)
@pytest.mark.parametrize("blocks,out", [("1x16", BF), ("1x16", F32), ("16x16", BF)])
def test_grouped_matmul(T, E, N, K, mx8, blocks, out):
    x, xs, xv = rows(T + K, T, K, mx8)
    p, s, a = weights(N, E, N, K, blocks)
    check_grouped(x, xs, xv, split(T, T, E, empty=(E // 2,) if E > 2 else ()), p, s, a, blocks, out)


@pytest.mark.parametrize("T,N", [(30, 1001), (700, 333)])
@pytest.mark.parametrize("amax", ["none", "row"])
def test_grouped_matmul_odd_width_and_other_scales(T, N, amax):
    x, xs, xv = rows(T, T, 304, False)
    p, s, a = weights(N, 3, N, 304, "1x16", amax)
    check_grouped(x, xs, xv, split(T, T, 3), p, s, a, "1x16", F32, row_scaled=amax == "row")


@pytest.mark.parametrize("T", [20, 400])
@pytest.mark.parametrize("mx8", [False, True], ids=["bf16", "mx8"])
def test_grouped_matmul_transposed_tiles(T, mx8):
    """The columnwise codes of the 16x16 quantization with its tile scales as
    they are: the operand of the input's gradient."""
    E, N, K = 3, 304, 272
    g = torch.Generator(device="cuda").manual_seed(2)
    q = []
    for _ in range(E):
        w = (torch.randn(N, K, device="cuda", generator=g) * 0.02).to(BF)
        a = nv.amax(w)
        q.append(nv.quantize_2d(w, a) + (a,))
    row, col, tiles, amax = (torch.stack(t) for t in zip(*q))
    amax = amax.view(-1)
    assert torch.equal(R.weight_values(col, tiles, "16x16t", amax), R.weight_values(row, tiles, "16x16", amax).transpose(1, 2))
    x, xs, xv = rows(T, T, N, mx8)
    check_grouped(x, xs, xv, split(T, T, E), col, tiles, amax, "16x16t", BF)


ENDS = {"falling": [300, 100, 250, 400], "negative": [-5, -1, 200, 200], "past the end": [100, 9000, 9000, 2 ** 31 - 1],
        "none owned": [0, 0, 0, 0], "rows left over": [10, 20, 150, 151], "all in the last": [0, 0, 0, 400]}


@pytest.mark.parametrize("kind", list(ENDS))
@pytest.mark.parametrize("T", [60, 400])
def test_row_ranges_of_any_kind(kind, T):
    ends = torch.tensor(ENDS[kind], dtype=torch.int32)
    x, xs, xv = rows(T, T, 176, False)
    p, s, a = weights(1, 4, 272, 176)
    check_grouped(x, xs, xv, ends, p, s, a, "1x16", F32, what=kind)
    check_wgrad(T, 4, 272, 176, False, F32, ends)


@pytest.mark.parametrize("T,E", [(100, 200), (5000, 130), (9, 64), (70, 65)])
def test_many_experts(T, E):
    """More experts than a wave has lanes, most of them with few or no rows."""
    ends = split(E, T, E, empty=range(0, E, 3))
    x, xs, xv = rows(T, T, 48, True)
    p, s, a = weights(1, E, 32, 48)
    check_grouped(x, xs, xv, ends, p, s, a, "1x16", F32)
    check_wgrad(T, E, 32, 48, True, F32, ends)


def check_wgrad(T, E, N, K, mx8, out, ends):
    x, xs, xv = rows(T + N, T, K, mx8)
    dy = randn(gen(T), T, N, by=0.5)
    got = nv.grouped_wgrad(dy.cuda(), x, ends.cuda(), x_scale=xs, out_dtype=out)
    assert got.shape == (E, N, K) and got.dtype == out
    c = R.cuts(ends, T)
    for e in range(E):
        d, v = R.f64(dy)[c[e]:c[e + 1]], xv[c[e]:c[e + 1]]
        y = d.t() @ v
        # as product_bound, the sum running over the expert's rows
        most = y.abs() * R.half_step(out) + (d.shape[0] + 8) * 2.0 ** -23 * (d.abs().t() @ v.abs())
        R.assert_near(got[e], y, most, f"dw of expert {e}")


@pytest.mark.parametrize("mx8", [False, True], ids=["bf16", "mx8"])
@pytest.mark.parametrize("T,E,N,K", SIZES)
@pytest.mark.parametrize("out", [BF, F32], ids=["out16", "out32"])
def test_grouped_wgrad(T, E, N, K, mx8, out):
    check_wgrad(T, E, N, K, mx8, out, split(T, T, E, empty=(E // 2,) if E > 2 else ()))


def test_empty_calls():
    p, s, a = weights(1, 3, 32, 48)
    ends = torch.zeros(3, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 48, dtype=BF, device="cuda")
    assert nv.grouped_matmul(x, ends, p, s, global_amax=a).shape == (0, 32)
    assert nv.matvec(x, p[0], s[0], global_amax=a[:1]).shape == (0, 32)
    dw = nv.grouped_wgrad(torch.empty(0, 32, dtype=BF, device="cuda"), x, ends)
    assert dw.shape == (3, 32, 48) and not dw.any()
    assert not nv.matvec(torch.empty(4, 0, dtype=BF, device="cuda"), p[0][:, :0], s[0][:, :0], global_amax=a[:1]).any()
    c, sc, h, r = nv.add_rms_norm(x, torch.ones(48, device="cuda"))
    assert c.shape == (0, 48) and sc.shape == (0, 2) and r.shape == (0,)
    dx, dw = nv.add_rms_norm_backward(x, x, torch.ones(48, device="cuda"), r)
    assert dx.shape == (0, 48) and not dw.any()
    assert [tuple(t.shape) for t in nv.swiglu_checkpoint(torch.empty(0, 96, dtype=BF, device="cuda"))] == [
        (0, 48), (0, 2), (0, 96), (0, 4)]


@pytest.mark.parametrize("T", [6, 300])
def test_values_that_are_not_finite_stay_in_their_rows(T):
    """An infinity or NaN in a row of x changes that row of the product alone,
    and that expert's gradient alone; so does one in the last k's, next to the
    columns that a tile reads past the end.  A NaN scale spoils its own column."""
    E, N, K = 3, 272, 176
    ends = torch.tensor([T // 3, 2 * T // 3, T], dtype=torch.int32)
    x, _, xv = rows(1, T, K, False)
    p, s, a = weights(2, E, N, K)
    clean = nv.grouped_matmul(x, ends.cuda(), p, s, global_amax=a)
    bad = x.clone()
    at = T // 3  # first row of the second expert
    bad[at, K - 1], bad[T - 1, 0] = INF, NAN
    got = nv.grouped_matmul(bad, ends.cuda(), p, s, global_amax=a)
    keep = torch.ones(T, dtype=torch.bool)
    keep[[at, T - 1]] = False
    assert torch.equal(got.cpu()[keep], clean.cpu()[keep])
    assert not torch.isfinite(got[at]).any() and torch.isnan(got[T - 1]).all()
    dy = randn(gen(9), T, N).cuda()
    d0, d1 = nv.grouped_wgrad(dy, x, ends.cuda()), nv.grouped_wgrad(dy, bad, ends.cuda())
    assert torch.equal(d0[0], d1[0])
    assert torch.equal(d0[1, :, :K - 1], d1[1, :, :K - 1]) and not torch.isfinite(d1[1, :, K - 1]).any()
    assert torch.equal(d0[2, :, 1:], d1[2, :, 1:]) and torch.isnan(d1[2, :, 0]).all()
    dyb = dy.clone()
    dyb[at - 1, 3] = NAN  # last row of the first expert
    d2 = nv.grouped_wgrad(dyb, x, ends.cuda())
    assert torch.isnan(d2[0, 3]).all() and torch.equal(d2[1:], d0[1:]) and torch.equal(d2[0, 4:], d0[0, 4:])
    s2 = s.clone()
    s2[1, 7, K // 16 - 1] = 0x7F
    got = nv.grouped_matmul(x, ends.cuda(), p, s2, global_amax=a)
    mid = slice(T // 3, 2 * T // 3)
    assert torch.isnan(got[mid, 7]).all()
    got[mid, 7] = clean[mid, 7]
    assert torch.equal(got, clean)


def test_negative_and_extreme_scales():
    """Scale bytes are read as e4m3 numbers, with their sign, and mx8 scales over
    their whole written range."""
    g = gen(21)
    N, K, T = 48, 96, 9
    p = torch.randint(0, 256, (1, N, K // 2), dtype=torch.uint8, generator=g).cuda()
    s = torch.randint(0, 256, (1, N, K // 16), dtype=torch.uint8, generator=g)
    s[(s & 127) == 127] = 0x7E
    c = torch.randint(0, 256, (T, K), dtype=torch.uint8, generator=g)
    c[(c & 127) == 127] = 0x01
    xs = torch.randint(10, 200, (T, 1), dtype=torch.uint8, generator=g).expand(T, 3).contiguous()
    xv = R.mx8_values(c.long(), xs.long())
    w = R.weight_values(p, s, "1x16")[0]
    y = xv @ w.t()
    got = nv.matvec(c.cuda(), p[0], s[0].cuda(), x_scale=xs.cuda(), out_dtype=F32)
    R.assert_near(got, y, R.product_bound(xv, w, F32, y) + 1e-37, "matvec")


def test_offsets_past_32_bits():
    """Rows whose byte offset passes 2^32: products and weight gradient of the
    last rows equal those of a short call on the same rows."""
    T, K, N = 270_000, 8192, 64
    x = torch.empty(T, K, dtype=BF, device="cuda")
    x[:1000].normal_(), x[-1000:].normal_()
    x[1000:-1000] = 0
    p, s, a = weights(3, 2, N, K)
    ends = torch.tensor([T - 700, T], dtype=torch.int32, device="cuda")
    y = nv.grouped_matmul(x, ends, p, s, global_amax=a)
    last = nv.grouped_matmul(x[-700:].contiguous(), ends.new_tensor([0, 700]), p, s, global_amax=a, out_dtype=BF)
    w = R.weight_values(p, s, "1x16", a)[1]
    xv = R.f64(x[-700:])
    want = xv @ w.t()
    R.assert_near(y[-700:], want, R.product_bound(xv, w, BF, want), "last rows")
    assert torch.equal(y[-700:], last) and not y[1000:T - 1000].any()
    dy = torch.zeros(T, N, dtype=BF, device="cuda")
    dy[-700:].normal_()
    dw = nv.grouped_wgrad(dy, x, ends)
    ref = nv.grouped_wgrad(dy[-700:].contiguous(), x[-700:].contiguous(), ends.new_tensor([0, 700]))
    assert torch.equal(dw, ref)


def test_refusals_on_the_device():
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn(8, 96, device="cuda", generator=g).to(BF)
    p, s, a = weights(1, 2, 32, 96)
    ends = torch.tensor([3, 8], dtype=torch.int32, device="cuda")
    w = torch.ones(96, device="cuda")
    ok = dict(global_amax=a)
    for call in (lambda: nv.add_rms_norm(x.t(), w), lambda: nv.add_rms_norm(x, w[:80]), lambda: nv.add_rms_norm(x, w.to(BF)),
                 lambda: nv.add_rms_norm(x, w, x.float()), lambda: nv.add_rms_norm(x, w, x[:4]),
                 lambda: nv.swiglu_checkpoint(x[:, :80].contiguous()), lambda: nv.swiglu_backward(x, x, x),
                 lambda: nv.matvec(x.float(), p[0], s[0]), lambda: nv.matvec(x, p[0], s[0][:, :5]),
                 lambda: nv.matvec(x, p[0][:, :40], s[0]), lambda: nv.matvec(x, p[0], s[0], row_scaled=True),
                 lambda: nv.matvec(x, p[0], s[0], global_amax=a), lambda: nv.matvec(x, p[0], s[0], out_dtype=torch.float16),
                 lambda: nv.matvec(x, p[0], s[0], tile16=True),
                 lambda: nv.grouped_matmul(x, ends.long(), p, s, **ok), lambda: nv.grouped_matmul(x, ends[:1], p, s, **ok),
                 lambda: nv.grouped_matmul(x, ends.cpu(), p, s, **ok), lambda: nv.grouped_matmul(x, ends, p[0], s[0], **ok),
                 lambda: nv.grouped_matmul(x, ends, p, s, transposed_tiles=True, **ok),
                 lambda: nv.grouped_matmul(x.view(torch.uint8).view(R.F8)[:, :96].contiguous(), ends, p, s, **ok),
                 lambda: nv.grouped_wgrad(x.float(), x, ends), lambda: nv.grouped_wgrad(x[:4], x, ends)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(nv.NVFP4Error):
        nv.matvec(x, p[0], s[0], global_amax=a[:1], bound=300.0)
    with pytest.raises(nv.NVFP4Error):
        nv.grouped_wgrad(x[:, :40].contiguous(), x, ends)


def layer_step(s):
    """A training step of the two products around a gated activation."""
    codes, scales, hidden, rstd = nv.add_rms_norm(s["x"], s["w"], s["r"])
    gate_up = nv.grouped_matmul(codes, s["ends"], s["p1"], s["s1"], x_scale=scales, tile16=True, global_amax=s["a1"])
    y, ys, kept, ks = nv.swiglu_checkpoint(gate_up)
    dmid = nv.grouped_matmul(s["dy"], s["ends"], s["c2"], s["s2"], tile16=True, transposed_tiles=True, global_amax=s["a2"])
    dgu = nv.swiglu_backward(dmid, kept, ks)
    dw1 = nv.grouped_wgrad(dgu, codes, s["ends"], x_scale=scales)
    dn = nv.grouped_matmul(dgu, s["ends"], s["c1"], s["s1"], tile16=True, transposed_tiles=True, global_amax=s["a1"])
    dx, dw = nv.add_rms_norm_backward(dn, hidden, s["w"], rstd, s["dy"])
    out = nv.grouped_matmul(y, s["ends"], s["p2"], s["s2"], x_scale=ys, tile16=True, global_amax=s["a2"])
    dw2 = nv.grouped_wgrad(s["dy"], y, s["ends"], x_scale=ys)
    few = nv.matvec(hidden[:2].contiguous(), s["p1"][0], s["s1"][0], tile16=True, global_amax=s["a1"][:1])
    return [out, dx, dw, dw1, dw2, few, hidden, rstd, gate_up, dgu]


def layer_state(seed, T=200, H=272, F=144, E=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *shape: torch.randn(*shape, device="cuda", generator=g)
    s = dict(x=r(T, H).to(BF), r=r(T, H).to(BF), w=1 + 0.1 * r(H), dy=r(T, H).to(BF),
             ends=split(seed, T, E).cuda())
    for i, (N, K) in ((1, (2 * F, H)), (2, (H, F))):
        q = []
        for _ in range(E):
            w = (r(N, K) * 0.05).to(BF)
            a = nv.amax(w)
            q.append(nv.quantize_2d(w, a) + (a,))
        s[f"p{i}"], s[f"c{i}"], s[f"s{i}"], a = (torch.stack(t) for t in zip(*q))
        s[f"a{i}"] = a.view(-1)
    return s


def test_step_repeats_bit_for_bit_on_any_stream():
    s = layer_state(1)
    want = layer_step(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer_step(s)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_captured_step_replays():
    """Each replay, on new inputs and with eager work in between, equals the
    eager step bit for bit."""
    s = layer_state(2)
    layer_step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer_step(s)
    for i in range(4):
        new = layer_state(10 + i)
        for k, v in s.items():
            v.copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = layer_step(new)
        for a, b in zip(want, got):
            assert torch.equal(a, b), i


def test_example_runs():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")
    spec = importlib.util.spec_from_file_location("expert_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    grads, out, one = mod.main(tokens=512, experts=8, hidden=256, inner=128)
    assert [tuple(t.shape) for t in grads] == [(512, 256), (256,), (8, 256, 256), (8, 256, 128)]
    assert all(torch.isfinite(t).all() for t in (*grads, out, one)) and out.shape == (4, 256) and one.shape == (1, 256)
    assert not grads[2][1].any() and not grads[3][1].any() and grads[2][0].any()
