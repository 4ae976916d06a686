"""The layer operators where their definitions are easy to miss: products without
a k, scale bytes at the ends of the format, rows far from 1, experts that have
nearly all rows.  Definitions are those of tests/layer_ref.py."""
import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
from fp4_block_quantization_nvfp4_amd import _lib as L
from tests import layer_ref as R
from tests.gpu_util import need_gpu
from tests.test_gpu_layer import BF, F32, check_grouped, check_norm, gen, randn, rows, weights

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


def row_values(c, s):
    """mx8 rows as the format defines them: byte 255 is NaN, and what passes the
    range of fp32 (2^128, from bytes 247 up) is infinite."""
    v = R.mx8_values(c, s)
    v = torch.where(v.abs() >= 2.0 ** 128, torch.copysign(torch.tensor(float("inf"), dtype=v.dtype), v), v)
    return torch.where((s == 255).repeat_interleave(32, 1)[:, :c.shape[1]], float("nan"), v)


LOW, HIGH = [0, 1, 2, 5, 9, 10], [200, 246, 247, 248, 250, 253, 254]


@pytest.mark.parametrize("scales", [LOW, HIGH, [255]], ids=["low", "high", "nan"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_swiglu_backward_reads_any_scale(scales, dtype):
    """Each scale byte with every code, or every one below 1 (below 2^-126 a value
    may count as zero), beside groups under scale 1."""
    T, F, G = len(scales), 64, 2
    c = torch.arange(T * 2 * F).view(T, 2 * F) * 37 % (0x7F if scales is LOW else 0x38)
    s = torch.full((T, 2 * G), 127)
    s[:, 0] = torch.tensor(scales)  # the first group of g; below that of u, so that products of both stay in range
    s[:, 2] = torch.tensor([255 if b == 255 else 230 if b < 127 else 254 - b for b in scales])
    d = torch.full((T, F), 0.5, dtype=dtype)
    if scales is LOW:
        d *= 2.0 ** 10
    got = R.f64(nv.swiglu_backward(d.cuda(), c.to(torch.uint8).cuda(), s.to(torch.uint8).cuda()))
    g, u = row_values(c[:, :F], s[:, :G]), row_values(c[:, F:], s[:, G:])
    if scales == [255]:
        assert torch.isnan(got[:, :32]).all() and torch.isnan(got[:, F:F + 32]).all()
        assert torch.isfinite(got[:, 32:F]).all() and torch.isfinite(got[:, F + 32:]).all()
        return
    dg, du = R.swiglu_gradient(R.f64(d), g, u)
    # as check_swiglu: roundings of sigma and of the products; d u and d g may each be off
    # by d times what counts as zero, 2^-126, and dgate by that times u
    sig = 1 / (1 + torch.exp(-g))
    lost = 2.0 ** -125 * R.f64(d).abs()
    most = dg.abs() * R.half_step(dtype) + 64 * R.U24 * R.f64(d).abs() * u.abs() * sig * (1 + g.abs()) + lost * (1 + u.abs())
    R.assert_near(got[:, :F], dg, most, "dgate")
    R.assert_near(got[:, F:], du, du.abs() * (R.half_step(dtype) + 64 * R.U24) + lost, "dup")


def one_a_row(T, K, scales):
    """mx8 rows with one code in each, the groups' scales `scales` in turn."""
    c = torch.zeros(T, K, dtype=torch.long)
    at = torch.arange(T) * 5 % K
    c[torch.arange(T), at] = 0x7E - torch.arange(T) * 3 % 0x7E if scales is LOW else 1 + torch.arange(T) % 0x37
    s = torch.tensor([scales[(t + j) % len(scales)] for t in range(T) for j in range((K + 31) // 32)]).view(T, -1)
    return c, s


@pytest.mark.parametrize("T", [4, 16, 60, 400])
@pytest.mark.parametrize("scales", [LOW, HIGH], ids=["low", "high"])
def test_products_read_any_scale(T, scales):
    N, K = 48, 160
    g = torch.Generator().manual_seed(T)
    c, xs = one_a_row(T, K, scales)
    p = torch.randint(0, 256, (1, N, K // 2), dtype=torch.uint8, generator=g)
    s = torch.randint(1, 9, (1, N, K // 16), dtype=torch.uint8, generator=g) + (0x70 if scales is LOW else 0)
    xv, w = row_values(c, xs), R.weight_values(p, s, "1x16")[0]
    y = xv @ w.t()
    most = R.product_bound(xv, w, F32, y) + 2.0 ** -126 * (w.abs().sum(1) + 1)
    ends = torch.tensor([T], dtype=torch.int32, device="cuda")
    x, xsd = c.to(torch.uint8).cuda(), xs.to(torch.uint8).cuda()
    R.assert_near(nv.grouped_matmul(x, ends, p.cuda(), s.cuda(), x_scale=xsd, out_dtype=F32), y, most, "grouped")
    R.assert_near(nv.matvec(x, p[0].cuda(), s[0].cuda(), x_scale=xsd, out_dtype=F32), y, most, "matvec")
    dy = (torch.randint(-8, 9, (T, N), generator=g) / 16).to(BF)
    dw = R.f64(dy).t() @ xv
    most = (T + 8) * 2.0 ** -23 * (R.f64(dy).abs().t() @ xv.abs()) + 2.0 ** -126 * (T + 1)
    R.assert_near(nv.grouped_wgrad(dy.cuda(), x, ends, x_scale=xsd)[0], dw, most, "dw")


@pytest.mark.parametrize("T", [4, 60, 400])
def test_products_of_a_nan_scale(T):
    """Byte 255 makes its 32 elements NaN, codes of zero among them: the row of a
    product, and in the weight gradient those columns of its own expert."""
    N, K = 48, 160
    g = torch.Generator().manual_seed(T)
    c = torch.randint(0, 0x38, (T, K), generator=g)
    xs = torch.full((T, K // 32), 127)
    c[1, 32:64], xs[1, 1] = 0, 255
    p = torch.randint(0, 256, (2, N, K // 2), dtype=torch.uint8, generator=g).cuda()
    s = torch.randint(0x30, 0x40, (2, N, K // 16), dtype=torch.uint8, generator=g).cuda()
    ends = torch.tensor([2, T], dtype=torch.int32, device="cuda")
    x, xsd = c.to(torch.uint8).cuda(), xs.to(torch.uint8).cuda()
    keep = torch.arange(T) != 1
    for y in (nv.grouped_matmul(x, ends, p, s, x_scale=xsd, out_dtype=F32), nv.matvec(x, p[0], s[0], x_scale=xsd, out_dtype=F32)):
        assert torch.isnan(y[1]).all() and torch.isfinite(y.cpu()[keep]).all()
    dw = nv.grouped_wgrad(torch.ones(T, N, dtype=BF, device="cuda"), x, ends, x_scale=xsd)
    assert torch.isnan(dw[0, :, 32:64]).all() and int(torch.isnan(dw).sum()) == 32 * N


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [96, 2064, 16400])
@pytest.mark.parametrize("res", [True, False], ids=["residual", "plain"])
def test_norm_of_rows_far_from_one(H, dtype, res):
    """Rows whose squares pass the range of fp32 at either end, eps = 0, between
    ordinary ones: y and rstd are as for any other row."""
    by = torch.tensor([1.0, 1e20, 2.0 ** 80, 1.0, 1e-24, 2.0 ** -120, 3e37, 1e-20])[:, None]
    g = gen(H)
    x, r = randn(g, 8, H, dtype=F32) * by, randn(g, 8, H, dtype=F32) * by
    w = 1 + 0.2 * torch.randn(H, generator=g)
    dy, dh = randn(g, 8, H, dtype=dtype), randn(g, 8, H, dtype=dtype)
    check_norm(x.to(dtype), r.to(dtype) if res else None, w, eps=0.0, upstream=(dy, dh))


def test_norm_of_rows_of_subnormals():
    """1 over the root passes fp32 (rstd infinite); y does not."""
    x = torch.full((3, 96), 2.0 ** -132).to(BF)
    x[1], x[2, 5:] = 1.0, 0.0
    codes, scales, _, rstd = nv.add_rms_norm(x.cuda(), torch.ones(96, device="cuda"), eps=0.0)
    h = R.f64(x)
    R.assert_mx8(codes, scales, h / h.square().mean(1, keepdim=True).sqrt(), 2.0 ** -20, "norm")
    assert torch.isinf(rstd[0]) and rstd[1] == 1


@pytest.mark.parametrize("H", [16, 2064])
@pytest.mark.parametrize("big", [0, 1, 31, 63])
def test_norm_weight_gradient_keeps_small_terms(H, big):
    """One large term and 63 that are below half its last place each but not
    together: 64 rows are a partial sum each, and these are joined in pairs, so a
    result is off by at most the six roundings of its way there (and four of the
    terms), not by one a row."""
    T = 64
    dy = torch.full((T, H), 1.9 * 2.0 ** -25)
    dy[big] = 1.0
    one = torch.ones(T, H)
    _, dw = nv.add_rms_norm_backward(dy.cuda(), one.cuda(), torch.ones(H, device="cuda"), torch.ones(T, device="cuda"))
    want = R.f64(dy).sum(0)
    R.assert_near(dw, want, 10 * R.U24 * want, "dweight")


HOT = [(512, 32, 80, 272, 7), (300, 20, 48, 144, 0), (2000, 130, 64, 80, 100), (700, 8, 176, 80, 7), (90, 1, 64, 272, 0),
       (400, 70, 32, 64, 69)]


@pytest.mark.parametrize("T,E,N,K,e", HOT)
@pytest.mark.parametrize("kind", ["all", "most", "none"])
@pytest.mark.parametrize("mx8", [False, True], ids=["bf16", "mx8"])
def test_one_expert_has_nearly_all_rows(T, E, N, K, e, kind, mx8):
    """Rows of one expert that many workgroups share, with others' and none's."""
    counts = torch.zeros(E, dtype=torch.int32)
    if kind == "most":
        counts += 1
    counts[e] += {"all": T, "most": T - E - 3, "none": 5}[kind]
    ends = torch.cumsum(counts, 0).int()
    x, xs, xv = rows(T + e, T, K, mx8)
    p, s, a = weights(E, E, N, K)
    y = check_grouped(x, xs, xv, ends, p, s, a, "1x16", F32, what=kind)
    assert torch.equal(y, nv.grouped_matmul(x, ends.cuda(), p, s, x_scale=xs, global_amax=a, out_dtype=F32))


def test_one_hot_expert_takes_no_longer_than_even_ones():
    """Its rows are shared by the workgroups of all experts: the time stays near
    that of an even split, which reads 32 times the weights (of one workgroup's
    making, it was 3.7 times that)."""
    T, E, N, K = 512, 32, 4096, 2048
    p = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((E, N, K // 16), 0x38, dtype=torch.uint8, device="cuda")
    x = torch.randn(T, K, device="cuda").to(BF)

    def time(counts):
        ends = torch.cumsum(torch.tensor(counts), 0).int().cuda()
        for _ in range(20):
            nv.grouped_matmul(x, ends, p, s)
        got = []
        for _ in range(9):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(20):
                nv.grouped_matmul(x, ends, p, s)
            b.record()
            b.synchronize()
            got.append(a.elapsed_time(b))
        return sorted(got)[4]

    even, hot = time([T // E] * E), time([0] * 5 + [T] + [0] * (E - 6))
    assert hot < 1.5 * even, (hot, even)


def test_nothing_is_recorded_for_autograd():
    """As layer.py says: inputs that require a gradient are taken, outputs require none."""
    x = torch.randn(8, 64, device="cuda").to(BF).requires_grad_()
    w = torch.ones(64, device="cuda", requires_grad=True)
    p, s, a = weights(1, 1, 32, 64)
    codes, scales, hidden, rstd = nv.add_rms_norm(x, w, x)
    assert not any(t.requires_grad for t in (codes, scales, hidden, rstd, nv.matvec(x, p[0], s[0], global_amax=a)))
    same = nv.add_rms_norm(x.detach(), w.detach(), x.detach())
    assert all(torch.equal(t.view(torch.uint8), u.view(torch.uint8)) for t, u in zip((codes, scales, hidden, rstd), same))


ELSEWHERE = """
import torch
torch.zeros(1, device="cuda")
here = torch._C._cuda_getDevice
torch._C._cuda_getDevice = lambda: here() + 1  # as if another device were the current one
import fp4_block_quantization_nvfp4_amd as nv
x, w = torch.ones(4, 64, device="cuda", dtype=torch.bfloat16), torch.ones(64, device="cuda")
p, s = torch.zeros(1, 32, 32, dtype=torch.uint8, device="cuda"), torch.zeros(1, 32, 4, dtype=torch.uint8, device="cuda")
ends, one = torch.tensor([4], dtype=torch.int32, device="cuda"), torch.ones(4, device="cuda")
kept = torch.zeros(4, 128, dtype=torch.uint8, device="cuda"), torch.zeros(4, 4, dtype=torch.uint8, device="cuda")
for call in (lambda: nv.add_rms_norm(x, w), lambda: nv.add_rms_norm_backward(x, x, w, one), lambda: nv.swiglu_checkpoint(x),
             lambda: nv.swiglu_backward(x, *kept), lambda: nv.matvec(x, p[0], s[0]), lambda: nv.grouped_matmul(x, ends, p, s),
             lambda: nv.grouped_wgrad(x, x, ends)):
    try:
        call()
    except ValueError as e:
        assert "current device" in str(e), e
    else:
        raise SystemExit("not refused")
print("refused")
"""


def test_tensors_of_another_device_are_refused():
    """Before anything is launched, on the host: the child takes its device for
    another one."""
    import os
    import subprocess
    import sys

    res = subprocess.run([sys.executable, "-c", ELSEWHERE], capture_output=True, text=True, timeout=100,
                         cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert res.returncode == 0 and "refused" in res.stdout, res.stdout + res.stderr


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("H", [2080, 16640])
@pytest.mark.parametrize("res", [True, False], ids=["residual", "plain"])
@pytest.mark.parametrize("by", [1.0, 2.0 ** 90, 2.0 ** -100], ids=["one", "large", "small"])
def test_norm_codes_next_to_borders_are_exact(H, dtype, res, by):
    """Every y lies within two units of its last place in fp32 from a border
    between two codes, or between two scales: the side that it is on in 64 bits
    counts.  |h| is 1, 5 or 7 with mean square 25, so that the root is known."""
    g = gen(H)
    pick = torch.rand(H // 2, generator=g) < 0.5
    size = torch.stack((torch.where(pick, 1.0, 5.0), torch.where(pick, 7.0, 5.0)), 1).view(-1)
    border = (16 + 2 * torch.randint(0, 7, (H,), generator=g) + 1).double() / 16 * torch.exp2(-torch.randint(0, 9, (H,), generator=g).double())
    border[::32] = 1.75  # of a group's scale
    border = border.view(-1, 32)
    border[:, 1:].clamp_(max=27 / 16)
    w = (border.view(-1) * 5 / size.double()).float()
    # a place off on either side too; always where the quotient is exact (|h| = 1 or 5),
    # since on a border itself the root's last bits in 64 would decide
    side = torch.randint(0, 2, (H,), generator=g) * 2 - 1
    w = torch.where((size == 7) & (torch.rand(H, generator=g) < 0.5), w, torch.nextafter(w, w + side))
    h = size * (torch.randint(0, 2, (6, H), generator=g) * 2 - 1)
    r = torch.randint(-3, 4, (6, H), generator=g).float() if res else torch.zeros(6, H)
    x = (h - r) * by
    codes, scales, _, _ = nv.add_rms_norm(x.to(dtype).cuda(), w.cuda(), (r * by).to(dtype).cuda() if res else None, eps=0.0)
    c, s = R.mx8_codes(h.double() / 5 * w.double())
    assert torch.equal(R.byte(scales), s) and torch.equal(R.byte(codes), c)
