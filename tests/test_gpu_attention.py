"""Attention on an NVFP4 cache on the GPU against its definitions in 64 bits
(tests/attention_ref.py), and what is written to the cache bit for bit against
`quantize` and the oracle: both layouts, both types, odd and empty sizes, strides,
masks that leave rows empty, garbage in slots that no query may see, bad pages,
other streams, captured and replayed steps.  Tolerances count the roundings that
the definitions allow; each is derived where it is used."""
import ctypes
import math

import numpy as np
import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
import oracle
from fp4_block_quantization_nvfp4_amd import _lib as L
from tests import attention_ref as A
from tests import layer_ref as R
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=BF, by=1.0):
    return (torch.randn(*shape, generator=g) * by).to(dtype)


def cuda(t):
    return None if t is None else t.cuda()


# ------------------------------------------------------- norm and rotation

SIZES = [(1, 4, 2, 64, 64), (3, 1, 1, 16, 16), (5, 3, 1, 32, 16), (2, 6, 2, 80, 32), (7, 5, 5, 96, 96), (33, 32, 8, 128, 128),
         (4, 0, 3, 128, 64), (4, 3, 0, 48, 48), (6, 2, 2, 192, 48), (3, 9, 1, 256, 256), (2, 3, 2, 512, 512), (3, 2, 2, 400, 208),
         (2, 2, 2, 64, 0), (700, 2, 1, 112, 80)]


def rows(g, T, Hq, Hk, D, dtype):
    """Queries and keys as views of one projection, of different scale from row to row."""
    x = torch.randn(T, Hq + Hk, D, generator=g) * torch.exp2(torch.randint(-6, 7, (T, Hq + Hk, 1), generator=g).float())
    x = x.to(dtype)
    return x[:, :Hq], x[:, Hq:]


def assert_rounded(got, want, x_size, what):
    """Computed in 64 bits (fewer than 2^12 roundings of terms up to x_size) and rounded once."""
    R.assert_near(got, want, want.abs() * R.half_step(got.dtype) + x_size * 2.0 ** -40 + 1e-38, what)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", SIZES)
def test_norm_rope(T, Hq, Hk, D, rot, interleaved, dtype):
    g = gen(T * D + rot)
    q, k = rows(g, T, Hq, Hk, D, dtype)
    f, mult = nv.rotary_frequencies(rot, factor=4.0, scaling="parts", original_length=512, device="cpu") if rot else (torch.zeros(0, dtype=torch.float64), 1.0)
    p = torch.randint(0, 1 << 20, (T,), generator=g, dtype=torch.int32)
    p[0] = 0
    qw, kw = 1 + 0.3 * torch.randn(D, generator=g), 1 + 0.3 * torch.randn(D, generator=g)
    dq, dk = randn(g, T, Hq, D, dtype=dtype), randn(g, T, Hk, D, dtype=dtype)
    both = torch.cat((q, k), 1).cuda()
    qc, kc = both[:, :Hq], both[:, Hq:]
    for a, b in ((qw, kw), (None, None), (qw, None), (None, kw)):
        how = dict(q_weight=cuda(a), k_weight=cuda(b), interleaved=interleaved, multiplier=mult, eps=1e-5)
        got = nv.norm_rope(qc, kc, p.cuda(), f.cuda(), **how)
        grads = nv.norm_rope_backward(dq.cuda(), dk.cuda(), qc, kc, p.cuda(), f.cuda(), **how)
        for x, w, dz, y, dx, dw, what in ((q, a, dq, got[0], grads[0], grads[2], "q"), (k, b, dk, got[1], grads[1], grads[3], "k")):
            want = A.norm_rope(x, w, p, f, interleaved, mult, 1e-5)
            assert y.is_contiguous() and y.dtype == dtype
            size = want.abs().amax(-1, keepdim=True) if want.numel() else want
            assert_rounded(y, want, size, what)
            gx, gw, terms, wterms = A.norm_rope_gradient(dz, x, w, p, f, interleaved, mult, 1e-5)
            # fp32: each output of the rotation and of the formula has fewer than 16 roundings of terms up to the row's largest
            big = terms.amax(-1, keepdim=True) if terms.numel() else terms
            R.assert_near(dx, gx, gx.abs() * R.half_step(dtype) + 32 * R.U24 * big + 1e-37, f"d{what}")
            assert (dw is None) == (w is None)
            if dw is not None:  # T * heads terms of a few roundings each, summed in some order
                R.assert_near(dw, gw, (T * x.shape[1] + 32) * R.U24 * wterms + 32 * R.U24 * (dz.double().abs().amax(-1).sum() if dz.numel() else 0) + 1e-37,
                              f"d{what} weight")


def test_norm_rope_far_positions():
    """Angles of any position are those of a product in 64 bits."""
    p = torch.tensor([0, 1, 2**20 + 1, 2**24 + 3, 2**30 + 7, 2**31 - 1], dtype=torch.int32)
    f = nv.rotary_frequencies(64, device="cpu")[0]
    x = torch.zeros(6, 1, 64)
    x[..., :32] = 1.0
    got, _ = nv.norm_rope(x.cuda(), x.cuda(), p.cuda(), f.cuda())
    R.assert_near(got, A.norm_rope(x, None, p, f), torch.full((6, 1, 64), 2.0 ** -23), "rotation")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_norm_rope_rows_that_are_not_finite(dtype):
    """They stay in their own rows; a row of zeros has the root of eps."""
    g = gen(3)
    q, k = rows(g, 6, 2, 1, 64, dtype)
    q[1, 0, 3], q[3, 1, 60], k[2] = float("inf"), NAN, 0.0
    p, f = torch.arange(6, dtype=torch.int32), nv.rotary_frequencies(32, device="cpu")[0]
    w = torch.ones(64).cuda()
    qo, ko = nv.norm_rope(q.cuda(), k.cuda(), p.cuda(), f.cuda(), q_weight=w, k_weight=w)
    bad = torch.zeros(6, 2, dtype=torch.bool)
    bad[1, 0] = bad[3, 1] = True
    assert torch.equal(torch.isfinite(qo.cpu().float()).all(-1), ~bad) and (ko[2] == 0).all() and torch.isfinite(ko.float()).all()
    wide = torch.zeros(1, 1, 64)
    wide[0, 0, 0], wide[0, 0, 1] = 3e38, 1e-30
    got, tiny = nv.norm_rope(wide.cuda(), (wide * 0 + 1e-30).cuda(), p[:1].cuda(), f.cuda(), q_weight=w, k_weight=w, eps=0.0)
    assert math.isclose(got[0, 0, 0].item(), 8.0, rel_tol=1e-6) and torch.allclose(tiny.cpu(), torch.ones(1, 1, 64), rtol=1e-6)


def test_norm_rope_gradient_against_differences():
    g = gen(8)
    T, H, D = 3, 2, 96
    q, k, dq, dk = (randn(g, T, H, D, dtype=F32) for _ in range(4))
    w = 1 + 0.1 * torch.randn(D, generator=g)
    p, f = torch.tensor([0, 5, 70000], dtype=torch.int32), nv.rotary_frequencies(64, device="cpu")[0]
    gq, gk, gw, gv = nv.norm_rope_backward(dq.cuda(), dk.cuda(), q.cuda(), k.cuda(), p.cuda(), f.cuda(), q_weight=w.cuda(), k_weight=w.cuda())
    loss = lambda a, b, u, v: ((A.norm_rope(a, u, p, f) * R.f64(dq)).sum() + (A.norm_rope(b, v, p, f) * R.f64(dk)).sum()).item()
    r = lambda *s: torch.randn(*s, dtype=torch.float64, generator=g)
    for _ in range(3):
        a, b, u, v, e = r(T, H, D), r(T, H, D), r(D), r(D), 1e-5
        at = [R.f64(t) for t in (q, k, w, w)]
        slope = (loss(*(x + e * y for x, y in zip(at, (a, b, u, v)))) - loss(*(x - e * y for x, y in zip(at, (a, b, u, v))))) / (2 * e)
        parts = [(R.f64(x), y) for x, y in zip((gq, gk, gw, gv), (a, b, u, v))]
        # fp32 gradients: 100 roundings of the terms' magnitudes; differences: e^2
        assert abs(sum((x * y).sum() for x, y in parts) - slope) <= 100 * R.U24 * sum((x.abs() * y.abs()).sum() for x, y in parts) + 1e-6


def test_norm_rope_many_tokens():
    """More tokens than waves; the weights' gradients join all of them."""
    g = gen(12)
    T, H, D = 9001, 3, 64
    q, dq = randn(g, T, H, D), randn(g, T, H, D)
    k, dk = q[:, :1], dq[:, :1]
    p, f = torch.randint(0, 5000, (T,), generator=g, dtype=torch.int32), nv.rotary_frequencies(64, device="cpu")[0]
    w = 1 + 0.2 * torch.randn(D, generator=g)
    qc, kc = q.cuda(), q.cuda()[:, :1]
    how = dict(q_weight=w.cuda(), k_weight=w.cuda())
    qo, ko = nv.norm_rope(qc, kc, p.cuda(), f.cuda(), **how)
    want = A.norm_rope(q, w, p, f)
    assert_rounded(qo, want, want.abs().amax(-1, keepdim=True), "q")
    assert torch.equal(ko, qo[:, :1])
    first = nv.norm_rope_backward(dq.cuda(), dk.cuda(), qc, kc, p.cuda(), f.cuda(), **how)
    gx, gw, terms, wterms = A.norm_rope_gradient(dq, q, w, p, f)
    R.assert_near(first[0], gx, gx.abs() * 2.0 ** -8 + 32 * R.U24 * terms.amax(-1, keepdim=True), "dq")
    # a lane adds up at most T * H / (768 workgroups) terms and the partial sums are joined in a tree and 16 more: far below T / 4
    R.assert_near(first[2], gw, (T // 4) * R.U24 * wterms, "dq weight")
    again = nv.norm_rope_backward(dq.cuda(), dk.cuda(), qc, kc, p.cuda(), f.cuda(), **how)
    assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk,D", [(2, 0, 64), (0, 3, 48), (9, 2, 128), (17, 1, 64), (2, 5, 256)])
def test_many_tokens_a_wave(Hq, Hk, D, dtype):
    """Tokens past the grid, with sides that have no heads or a ragged last pass: rows are those of calls on parts of the tokens,
    and so is what is written; the weights' gradients are the parts' sums."""
    g = gen(60 + D)
    T, page = 8200, 64
    q, k = rows(g, T, Hq, Hk, D, dtype)
    both, dz = torch.cat((q, k), 1).cuda(), randn(g, T, Hq + Hk, D, dtype=dtype).cuda()
    p, f = torch.randint(0, 1 << 17, (T,), generator=g, dtype=torch.int32).cuda(), nv.rotary_frequencies(D - D % 32)[0]
    for qw, kw in ((torch.rand(D, generator=g).cuda(), torch.rand(D, generator=g).cuda()), (None, torch.rand(D, generator=g).cuda()), (None, None)):
        how = dict(q_weight=qw, k_weight=kw)
        cut = lambda at: (dz[at, :Hq], dz[at, Hq:], both[at, :Hq], both[at, Hq:], p[at], f)
        parts = [slice(a, min(a + 1000, T)) for a in range(0, T, 1000)]
        whole, some = nv.norm_rope_backward(*cut(slice(0, T)), **how), [nv.norm_rope_backward(*cut(at), **how) for at in parts]
        for i in range(2):
            assert torch.equal(whole[i], torch.cat([x[i] for x in some]))
        for i, heads in ((2, Hq), (3, Hk)):
            if whole[i] is not None:
                want = torch.stack([x[i].double() for x in some]).sum(0)
                # each sum's order: T * heads terms, of which a lane has a few hundred at most and trees the others
                size = torch.stack([x[i].double().abs() for x in some]).sum(0) + (T * max(heads, 1)) ** 0.5 * 64
                assert ((whole[i].double() - want).abs() <= 512 * R.U24 * size).all()
    if Hk == 0:
        return
    slots = torch.randperm(T + 100, generator=g)[:T].int().cuda()
    slots[5::7] = -1
    a, b = (nv.PagedCache.empty((T + 163) // page, page, Hk, D) for _ in range(2))
    cut = lambda at: (both[at, :Hq], both[at, Hq:], dz[at, Hq:], p[at], f)
    out = nv.norm_rope_write(*cut(slice(0, T)), a, slots, k_weight=torch.ones(D).cuda())
    got = torch.cat([nv.norm_rope_write(*cut(at), b, slots[at], k_weight=torch.ones(D).cuda()) for at in parts])
    assert torch.equal(out, got) and all(torch.equal(getattr(a, n), getattr(b, n)) for n in ("k", "k_scale", "v", "v_scale"))


# ------------------------------------------------------------------- cache

CACHES = [(1, 1, 16, 16, 2), (5, 2, 64, 32, 3), (70, 3, 96, 16, 9), (33, 8, 128, 64, 2), (40, 5, 208, 128, 1), (17, 2, 512, 16, 4), (300, 1, 256, 256, 2)]


def fresh(pages, page, H, D, amax, g):
    c = nv.PagedCache.empty(pages, page, H, D)
    for t in (c.k, c.k_scale, c.v, c.v_scale):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    if amax:
        c.k_amax, c.v_amax = (torch.rand(H, generator=g) * 6 + 2).cuda(), (torch.rand(H, generator=g) * 6 + 2).cuda()
    return c


def clone(c):
    return nv.PagedCache(c.k.clone(), c.k_scale.clone(), c.v.clone(), c.v_scale.clone(), k_amax=c.k_amax, v_amax=c.v_amax)


def content(c):
    return [t.cpu() for t in (c.k, c.k_scale, c.v, c.v_scale)]


def expect(c, before, k, v, slots):
    """The cache's bytes after rows k, v [T, H, D] went to their slots: quantize head by head."""
    page, (codes_k, scale_k, codes_v, scale_v) = c.k.shape[2], before
    for x, codes, scales, amax in ((k, codes_k, scale_k, c.k_amax), (v, codes_v, scale_v, c.v_amax)):
        for h in range(x.shape[1]):
            p, s = nv.quantize(x[:, h].contiguous(), global_amax=None if amax is None else amax[h:h + 1].clone())
            for t, at in enumerate(slots.tolist()):
                if 0 <= at < codes.shape[0] * page:
                    codes[at // page, h, at % page], scales[at // page, h, at % page] = p[t].cpu(), s[t].cpu()
    return codes_k, scale_k, codes_v, scale_v


def some_slots(g, T, total):
    """Distinct slots in any order, some rows skipped."""
    s = torch.randperm(total, generator=g)[:T].int()
    if T >= 5:
        s[1], s[3] = -1, total
    return s


@pytest.mark.parametrize("amax", [False, True], ids=["single", "amax"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,H,D,page,pages", CACHES)
def test_write_and_read(T, H, D, page, pages, dtype, amax):
    g = gen(T + D)
    pages = max(pages, -(-T // page) + 1)
    c = fresh(pages, page, H, D, amax, g)
    x = torch.randn(T, 2 * H, D, generator=g) * torch.exp2(torch.randint(-8, 5, (T, 2 * H, D // 16, 1), generator=g).float()).expand(-1, -1, -1, 16).reshape(T, 2 * H, D)
    x = x.to(dtype).cuda()
    k, v = x[:, :H], x[:, H:]
    if T > 4 and D > 16:
        k[0, 0, :16] = 0.0
        k[2, 0, 1], v[2, 0, 5], v[4, 0, 17] = NAN, float("inf"), -float("inf")
        v[2, 0, 6] = -NAN
    slots = some_slots(g, T, pages * page)
    before = content(c)
    want = expect(c, [t.clone() for t in before], k, v, slots)
    nv.write_cache(c, k, v, slots.cuda())
    for got, w, what in zip(content(c), want, ("keys", "key scales", "values", "value scales")):
        assert torch.equal(got, w), what
    for out in (BF, F32):
        rk, rv = nv.read_cache(c, slots.cuda(), out_dtype=out)
        for got, codes, scales, a in ((rk, c.k, c.k_scale, c.k_amax), (rv, c.v, c.v_scale, c.v_amax)):
            for h in range(H):
                flat = lambda t: t[:, h].reshape(pages * page, -1).contiguous()
                dense = nv.dequantize(flat(codes), flat(scales), pages * page, D, global_amax=None if a is None else a[h:h + 1].clone(), out_dtype=out)
                ok = (slots >= 0) & (slots < pages * page)
                assert torch.equal(got[:, h].cpu()[ok], dense.cpu()[slots[ok].long()])
                assert (got[:, h].cpu()[~ok] == 0).all()


def test_write_against_the_oracle():
    g = gen(2)
    k, v = randn(g, 40, 2, 64, dtype=F32, by=3.0), randn(g, 40, 2, 64, dtype=F32)
    c = nv.PagedCache.empty(4, 16, 2, 64)
    nv.write_cache(c, k.cuda(), v.cuda(), torch.arange(40, dtype=torch.int32).cuda())
    for x, codes, scales in ((k, c.k, c.k_scale), (v, c.v, c.v_scale)):
        p, s = oracle.quantize(x.numpy().reshape(80, 64))
        at = lambda t: t.cpu().transpose(1, 2).reshape(64, 2, -1)[:40].reshape(80, -1).numpy()
        assert np.array_equal(at(codes), p) and np.array_equal(at(scales), s)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "pairs"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [s for s in SIZES if s[2] > 0])
def test_norm_rope_write_is_norm_rope_and_write(T, Hq, Hk, D, rot, interleaved, dtype):
    g = gen(T + 2 * D)
    q, k = rows(g, T, Hq, Hk, D, dtype)
    v = randn(g, T, Hk, D, dtype=dtype).cuda()
    all_ = torch.cat((q, k), 1).cuda()
    q, k = all_[:, :Hq], all_[:, Hq:]
    f = (nv.rotary_frequencies(rot, device="cpu")[0] if rot else torch.zeros(0, dtype=torch.float64)).cuda()
    p = torch.randint(0, 1 << 17, (T,), generator=g, dtype=torch.int32).cuda()
    w = (1 + 0.3 * torch.randn(2, D, generator=g)).cuda()
    pages = -(-T // 16) + 1
    slots = some_slots(g, T, pages * 16).cuda()
    for how in (dict(q_weight=w[0], k_weight=w[1]), dict(), dict(q_weight=w[0]), dict(k_weight=w[1], multiplier=1.25)):
        c = fresh(pages, 16, Hk, D, T % 2 == 0, g)
        d = clone(c)
        got = nv.norm_rope_write(q, k, v, p, f, c, slots, interleaved=interleaved, **how)
        qo, ko = nv.norm_rope(q, k, p, f, interleaved=interleaved, **how)
        nv.write_cache(d, ko, v, slots)
        assert torch.equal(got, qo)
        for a, b, what in zip(content(c), content(d), ("keys", "key scales", "values", "value scales")):
            assert torch.equal(a, b), what


def test_cache_past_four_gigabytes():
    """Slots whose bytes lie past 2^32: nothing wraps."""
    pages, page, H, D = 70000, 1024, 1, 128  # 4.6 GB of codes of keys
    c = nv.PagedCache(*(torch.empty(pages, H, page, n, dtype=torch.uint8, device="cuda") for n in (D // 2, D // 16, D // 2, D // 16)))
    g = gen(4)
    k, v = randn(g, 40, H, D).cuda(), randn(g, 40, H, D).cuda()
    first = torch.randint(0, 1000, (20,), generator=g) * 7
    slots = torch.cat((first.unique(), pages * page - 1 - first.unique())).int()[:40].cuda()
    n = len(slots)
    nv.write_cache(c, k[:n], v[:n], slots)
    small = nv.PagedCache.empty(64, 16, H, D)
    nv.write_cache(small, k[:n], v[:n], torch.arange(n, dtype=torch.int32).cuda())
    for a, b in zip(nv.read_cache(c, slots), nv.read_cache(small, torch.arange(n, dtype=torch.int32).cuda())):
        assert torch.equal(a, b)
    table = torch.tensor([[0], [pages - 1]], dtype=torch.int32).cuda()
    c.k_scale[0].fill_(0x38), c.v_scale[0].fill_(0x38), c.k_scale[-1].fill_(0x38), c.v_scale[-1].fill_(0x38)
    q = randn(g, 2, 4, D).cuda()
    out, lse = nv.cache_attention(q, c, table, torch.tensor([1000, 1024], dtype=torch.int32).cuda())
    part = nv.PagedCache(*(t[[0, -1]].contiguous() for t in (c.k, c.k_scale, c.v, c.v_scale)))
    want = nv.cache_attention(q, part, torch.tensor([[0], [1]], dtype=torch.int32).cuda(), torch.tensor([1000, 1024], dtype=torch.int32).cuda())
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# --------------------------------------------------------------- attention


def filled(g, pages, page, H, D, amax=True, span=(0x28, 0x44)):
    """A cache of any codes and scales around one."""
    c = nv.PagedCache.empty(pages, page, H, D)
    for t in (c.k, c.v):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.randint(*span, t.shape, generator=g, dtype=torch.uint8))
    if amax:
        c.k_amax, c.v_amax = (2688 * (0.05 + 0.1 * torch.rand(H, generator=g))).cuda(), (2688 * (0.5 + torch.rand(H, generator=g))).cuda()
    else:
        c.k_scale.sub_(0x18)
    return c


def tables(g, lens, page, extra=1):
    """Pages of each sequence, in any order; -1 behind the last; the number of pages."""
    need = [-(-max(l, 0) // page) for l in lens]
    pages = sum(need) + extra
    order = torch.randperm(pages, generator=g).int()
    t = torch.full((len(lens), max(max(need, default=0), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        t[b, :n] = order[at:at + n]
        at += n
    return t, pages


def poison(c, table, lens):
    """NaN scales and any codes in every slot that no sequence has."""
    page = c.k.shape[2]
    free = torch.ones(c.k.shape[0], page, dtype=torch.bool)
    for b, l in enumerate(lens):
        for j in range(max(l, 0)):
            free[table[b, j // page], j % page] = False
    hit = free[:, None, :, None].cuda()
    for t in (c.k_scale, c.v_scale):
        t.copy_(torch.where(hit, torch.full_like(t, 0x7F), t))


def check_attention(q, c, table, lens, ends, causal, scale=None, what=""):
    lens_t = torch.tensor(lens, dtype=torch.int32)
    ends_t = None if ends is None else torch.tensor(ends, dtype=torch.int32)
    out, lse = nv.cache_attention(q, c, table.cuda(), lens_t.cuda(), cuda(ends_t), scale=scale, causal=causal)
    assert out.dtype == BF and out.shape == q.shape and lse.dtype == F32 and lse.shape == q.shape[:2]
    keys, values = A.cache_values(c.k, c.k_scale, c.k_amax), A.cache_values(c.v, c.v_scale, c.v_amax)
    want, wl, off, loff = A.attention(q, keys, values, table, lens_t, ends_t, scale, causal)
    R.assert_near(lse, wl, loff, f"{what} lse")
    R.assert_near(out, want, off, f"{what} out")
    return out, lse


HEADS = [(1, 1, 32), (4, 2, 64), (15, 5, 96), (32, 8, 128), (8, 8, 64), (16, 1, 160), (7, 1, 192), (40, 2, 256), (12, 4, 224)]


@pytest.mark.parametrize("Hq,Hk,D", HEADS)
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(Hq, Hk, D, page):
    g = gen(Hq * D + page)
    lens = [1, 0, 17, 127, 128, 129, 500, 16, 1030, 2]
    table, pages = tables(g, lens, page)
    c = filled(g, pages, page, Hk, D, amax=page != 64)
    poison(c, table, lens)
    check_attention(randn(g, len(lens), Hq, D).cuda(), c, table, lens, None, True)
    check_attention(randn(g, len(lens), Hq, D, by=20.0).cuda(), c, table, lens, None, False, scale=0.3)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hk,D", HEADS)
def test_ragged_queries(Hq, Hk, D, causal):
    """Few and many queries in one batch, sequences without queries or keys, keys fewer than queries (rows that see none), rows behind the last sequence."""
    g = gen(Hq + D)
    n = [3, 0, 130, 1, 64, 5, 37, 0, 2, 200]
    lens = [300, 77, 130, 1, 900, 2, 20, 0, 0, 231]
    T = sum(n) + 9
    ends = torch.cumsum(torch.tensor(n), 0).tolist()
    table, pages = tables(g, lens, 32)
    c = filled(g, pages, 32, Hk, D)
    poison(c, table, lens)
    out, lse = check_attention(randn(g, T, Hq, D).cuda(), c, table, lens, ends, causal)
    assert (out[-9:] == 0).all() and (lse[-9:] == -math.inf).all()


@pytest.mark.parametrize("G,n,L", [(1, 1, 1), (1, 31, 64), (4, 8, 63), (4, 9, 65), (8, 16, 16), (2, 65, 191), (1, 128, 128), (1, 129, 257), (3, 43, 512), (16, 3, 4096)])
@pytest.mark.parametrize("causal", [True, False])
def test_one_sequence(G, n, L, causal):
    """Either side of the units' and tiles' sizes."""
    g = gen(G * 1000 + n)
    table, pages = tables(g, [L], 64)
    c = filled(g, pages, 64, 2, 128)
    poison(c, table, [L])
    check_attention(randn(g, n, 2 * G, 128).cuda(), c, table, [L], [n], causal)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long_sequences_are_split(D):
    """One long sequence among short ones: many workgroups share it, and its parts are joined."""
    g = gen(D)
    lens = [3, 20000, 1, 0, 129, 4000]
    table, pages = tables(g, lens, 128)
    c = filled(g, pages, 128, 2, D)
    q = randn(g, len(lens), 8, D).cuda()
    first = check_attention(q, c, table, lens, None, True)
    for _ in range(3):  # the sums' order is fixed
        out, lse = nv.cache_attention(q, c, table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("D,n,L", [(96, [300, 129], [300, 700]), (128, [513], [513]), (64, [300], [900]), (256, [140, 190], [140, 900])])
def test_many_heads(D, n, L):
    """Enough units for workgroups of eight waves, which heads over 64 take."""
    g = gen(D)
    table, pages = tables(g, L, 64)
    c = filled(g, pages, 64, 128 if D < 256 else 16, D)
    poison(c, table, L)
    check_attention(randn(g, sum(n), 128 if D < 256 else 16, D).cuda(), c, table, L, torch.cumsum(torch.tensor(n), 0).tolist(), True)


def test_many_sequences():
    """More than a wave's 64 at a time, each with a few keys."""
    g = gen(9)
    B = 333
    lens = torch.randint(0, 300, (B,), generator=g).tolist()
    n = torch.randint(0, 4, (B,), generator=g)
    table, pages = tables(g, lens, 16)
    c = filled(g, pages, 16, 2, 64)
    check_attention(randn(g, B, 4, 64).cuda(), c, table, lens, None, True)
    check_attention(randn(g, int(n.sum()) + 3, 4, 64).cuda(), c, table, lens, torch.cumsum(n, 0).tolist(), True)


def test_sharp_and_flat_scores():
    """One key has all the weight; all keys are alike; scores far apart, whose small weights count in the sum."""
    g = gen(10)
    table, pages = tables(g, [2000], 64)
    c = filled(g, pages, 64, 1, 64, amax=False)
    for by in (0.0, 1e-3, 30.0, 3e4):
        check_attention(randn(g, 1, 4, 64, by=by).cuda(), c, table, [2000], None, True, what=f"by {by}")
        check_attention(randn(g, 70, 4, 64, by=by).cuda(), c, table, [2000], [70], True, what=f"tiles by {by}")
    tiny = randn(g, 1, 4, 64, dtype=F32, by=1e-35).bfloat16().cuda()
    check_attention(tiny, c, table, [2000], None, True, what="tiny")
    check_attention(tiny, c, table, [2000], None, True, scale=1e33, what="tiny, large scale")


def test_rows_that_are_not_finite():
    """A NaN or an infinity in a query stays in its row."""
    g = gen(11)
    table, pages = tables(g, [200], 64)
    c = filled(g, pages, 64, 2, 64)
    for n in (4, 80):
        q = randn(g, n, 4, 64)
        clean = nv.cache_attention(q.cuda(), c, table.cuda(), torch.tensor([200], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda())
        q[1, 2, 5], q[3, 0, 63] = NAN, float("inf")
        out, lse = nv.cache_attention(q.cuda(), c, table.cuda(), torch.tensor([200], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda())
        bad = torch.zeros(n, 4, dtype=torch.bool)
        bad[1, 2] = bad[3, 0] = True
        keep = ~bad.cuda()
        assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])
        assert torch.isnan(out[1, 2]).all() and torch.isnan(lse[1, 2]) and torch.isnan(out[3, 0].float()).any()


@pytest.mark.parametrize("n,L,D", [(5, 40, 64), (40, 150, 128), (100, 200, 256), (300, 400, 96), (300, 300, 64), (150, 700, 160)])
@pytest.mark.parametrize("what", ["k_scale", "v_scale"])
def test_nan_in_keys_that_are_hidden(n, L, D, what):
    """A NaN scale of a key or a value reaches the queries that see it, and no other."""
    g = gen(50 + D)
    table, pages = tables(g, [L], 16)
    c = filled(g, pages, 16, 2, D)
    q, lens, ends = randn(g, n, 4, D).cuda(), torch.tensor([L], dtype=torch.int32).cuda(), torch.tensor([n], dtype=torch.int32).cuda()
    want = nv.cache_attention(q, c, table.cuda(), lens, ends)
    j = L - n // 2  # queries from here on see it
    getattr(c, what)[table[0, j // 16], 1, j % 16, D // 16 - 1] = 0x7F if n % 2 else 0xFF
    out, lse = nv.cache_attention(q, c, table.cuda(), lens, ends)
    first = j - (L - n)
    assert torch.equal(out[:first], want[0][:first]) and torch.equal(lse[:first], want[1][:first])
    assert torch.equal(out[:, :2], want[0][:, :2]) and torch.equal(lse[:, :2], want[1][:, :2])
    assert torch.isnan(out[first:, 2:]).all() and torch.isnan(lse[first:, 2:]).all()


def test_bad_pages_and_lengths():
    """Pages that are not in the cache, and lengths past the table's rows, give NaN where a query sees them; ends in any order stay in range."""
    g = gen(13)
    lens = [100, 100, 40, 100]
    table, pages = tables(g, lens, 16)
    c = filled(g, pages, 16, 2, 64)
    table[0, 3], table[1, 0], table[3, 6] = -5, 1 << 30, pages
    length = torch.tensor([100, 100, 1 << 30, 100], dtype=torch.int32).cuda()
    q = randn(g, 4, 4, 64).cuda()
    out, lse = nv.cache_attention(q, c, table.cuda(), length)
    assert torch.isnan(out).all() and torch.isnan(lse).all()
    # queries that do not see the bad page (key 48 of 100) are as without it
    q = randn(g, 100, 4, 64).cuda()
    out, lse = nv.cache_attention(q, c, table[:1].cuda(), length[:1], torch.tensor([100], dtype=torch.int32).cuda())
    good = table[:1].clone()
    good[0, 3] = 0
    want, wl = nv.cache_attention(q, c, good.cuda(), length[:1], torch.tensor([100], dtype=torch.int32).cuda())
    assert torch.equal(out[:48], want[:48]) and torch.equal(lse[:48], wl[:48]) and torch.isnan(out[48:]).all() and torch.isnan(lse[48:]).all()
    good, _ = tables(gen(1), lens, 16)
    for ends in ([50, 20, 1000, 3], [-4, -1, 7, 7], [0, 0, 0, 0], [100, 100, 100, 100]):
        check_attention(q, c, good, [100, 100, 40, -3], ends, True)


def test_strides_and_alignment():
    g = gen(14)
    table, pages = tables(g, [90, 33], 32)
    c = filled(g, pages, 32, 2, 64)
    lens, ends = torch.tensor([90, 33], dtype=torch.int32).cuda(), torch.tensor([40, 60], dtype=torch.int32).cuda()
    q = randn(g, 60, 4, 64)
    want = nv.cache_attention(q.cuda(), c, table.cuda(), lens, ends)
    wide = torch.zeros(60, 9, 128, dtype=BF, device="cuda")
    wide[:, 1::2, 8:72] = q.cuda()
    by_head = q.cuda().transpose(0, 1).contiguous().transpose(0, 1)
    flipped = torch.zeros(4, 60, 72, dtype=BF, device="cuda")[:, :, :64].transpose(0, 1)
    flipped.copy_(q)
    for view in (wide[:, 1::2, 8:72], by_head, flipped):
        assert not view.is_contiguous()
        got = nv.cache_attention(view, c, table.cuda(), lens, ends)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    p, f = torch.arange(60, dtype=torch.int32).cuda(), nv.rotary_frequencies(64)[0]
    want = nv.norm_rope(q.cuda(), q.cuda(), p, f)
    for view in (wide[:, 1::2, 8:72], by_head, flipped):
        got = nv.norm_rope(view, view, p, f)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    one = torch.zeros(1, 1, 200, dtype=BF, device="cuda")[:, :, 8:72].expand(1, 1, 64)
    assert nv.norm_rope(one, one, p[:1], f)[0].shape == (1, 1, 64)
    same = q.cuda()[:1].expand(60, 4, 64)  # a broadcast input
    assert torch.equal(nv.norm_rope(same, same, p, f)[0], nv.norm_rope(same.contiguous(), same.contiguous(), p, f)[0])


def test_refusals():
    g = gen(15)
    c = filled(g, 3, 16, 2, 64)
    q, i = randn(g, 3, 4, 64).cuda(), torch.tensor([1, 2, 3], dtype=torch.int32).cuda()
    k, f = q[:, :2], nv.rotary_frequencies(64)[0]
    table = torch.zeros(3, 1, dtype=torch.int32).cuda()
    value = lambda match, call: _refused(ValueError, match, call)
    value("bfloat16 is required", lambda: nv.cache_attention(q.float(), c, table, i))
    value("head size", lambda: nv.cache_attention(q[..., :32], c, table, i))
    value("multiple of the cache's heads", lambda: nv.cache_attention(q[:, :3], c, table, i))
    value("multiples of 16 bytes", lambda: nv.cache_attention(torch.zeros(3, 4, 68, dtype=BF, device="cuda")[..., :64], c, table, i))
    value("contiguous", lambda: nv.cache_attention(torch.zeros(3, 4, 128, dtype=BF, device="cuda")[..., ::2], c, table, i))
    value("one query for each", lambda: nv.cache_attention(q[:2], c, table, i))
    value("lens", lambda: nv.cache_attention(q, c, table, i[:2]))
    value("lens", lambda: nv.cache_attention(q, c, table, i.long()))
    value("ends", lambda: nv.cache_attention(q, c, table, i, i[:2]))
    value("table", lambda: nv.cache_attention(q, c, table.long(), i))
    value("table", lambda: nv.cache_attention(q, c, table[0], i))
    value("3-D", lambda: nv.cache_attention(q[0], c, table, i))
    value("slots", lambda: nv.write_cache(c, k, k, i[:2]))
    value("v must be", lambda: nv.write_cache(c, k, q, i))
    value("cache's heads", lambda: nv.write_cache(c, q, q[:, :2], i))
    value("k must be", lambda: nv.norm_rope_write(q, q, q, i, f, c, i))
    value("k must be", lambda: nv.norm_rope(q, k.float(), i, f))
    value("positions", lambda: nv.norm_rope(q, k, i.long(), f))
    value("freqs", lambda: nv.norm_rope(q, k, i, f.float()))
    value("q_weight", lambda: nv.norm_rope(q, k, i, f, q_weight=torch.ones(32).cuda()))
    value("dq must be", lambda: nv.norm_rope_backward(k, k, q, k, i, f))
    value("out_dtype", lambda: nv.read_cache(c, i, out_dtype=torch.float16))
    value("cache.v_scale", lambda: nv.read_cache(nv.PagedCache(c.k, c.k_scale, c.v, c.v_scale[:1]), i))
    value("k_amax", lambda: nv.read_cache(nv.PagedCache(c.k, c.k_scale, c.v, c.v_scale, k_amax=torch.ones(1).cuda()), i))
    none = nv.PagedCache.empty(3, 16, 0, 64)
    value("heads >= 1", lambda: nv.cache_attention(q, none, table, i))
    value("heads >= 1", lambda: nv.write_cache(none, q[:, :0], q[:, :0], i))
    status = lambda call: _refused(nv.NVFP4Error, "status", call)
    status(lambda: nv.cache_attention(q, c, table, i, scale=-1.0))
    status(lambda: nv.norm_rope(q, k, i, nv.rotary_frequencies(66)[0]))
    status(lambda: nv.norm_rope(q, k, i, nv.rotary_frequencies(24)[0]))
    status(lambda: nv.norm_rope(q, k, i, f, eps=-1.0))
    odd = filled(g, 2, 16, 2, 48, amax=False)
    status(lambda: nv.cache_attention(q[..., :48].contiguous(), odd, table, i))
    status(lambda: nv.read_cache(nv.PagedCache(*(torch.zeros(2, 1, 24, n, dtype=torch.uint8, device="cuda") for n in (8, 1, 8, 1))), i))


def _refused(kind, match, call):
    with pytest.raises(kind, match=match):
        call()


def test_empty_calls():
    c = nv.PagedCache.empty(2, 16, 2, 64)
    none, i = torch.zeros(0, 4, 64, dtype=BF, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    f, w = nv.rotary_frequencies(64)[0], torch.ones(64, device="cuda")
    q, k = nv.norm_rope(none, none[:, :2], i, f, q_weight=w)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    grads = nv.norm_rope_backward(none, none[:, :2], none, none[:, :2], i, f, q_weight=w, k_weight=w)
    assert grads[0].shape == (0, 4, 64) and (grads[2] == 0).all() and (grads[3] == 0).all()
    assert nv.norm_rope_write(none, none[:, :2], none[:, :2], i, f, c, i).shape == (0, 4, 64)
    nv.write_cache(c, none[:, :2], none[:, :2], i)
    assert nv.read_cache(c, i)[0].shape == (0, 2, 64)
    out, lse = nv.cache_attention(none, c, torch.zeros(0, 1, dtype=torch.int32, device="cuda"), i)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    out, lse = nv.cache_attention(torch.ones(3, 4, 64, dtype=BF, device="cuda"), c, torch.zeros(0, 1, dtype=torch.int32, device="cuda"), i, i)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_workspace_of_no_bytes():
    """Where none is needed, one that is there is left as it was."""
    g = gen(31)
    table, pages = tables(g, [40, 64, 0], 16, extra=0)
    c, q = filled(g, pages, 16, 2, 64), randn(g, 40, 4, 64).cuda()
    table = table[:, :4].contiguous().cuda()
    lens, ends = torch.tensor([40, 64, 0], dtype=torch.int32).cuda(), torch.tensor([38, 39, 40], dtype=torch.int32).cuda()
    want = nv.cache_attention(q, c, table, lens, ends)
    P = lambda t: None if t is None else t.data_ptr()
    heads = L.Heads(P(q), 4, q.stride(0), q.stride(1))
    view = L.Cache(P(c.k), P(c.k_scale), P(c.v), P(c.v_scale), P(c.k_amax), P(c.v_amax), c.k.shape[0], 16, 2, 64)
    assert L.lib().nvfp4_cache_attention_workspace_bytes(40, 4, ctypes.byref(view), 3, 4) == 0
    space = torch.full((1 << 24,), 7, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(40, 4, device="cuda")
    st = L.lib().nvfp4_cache_attention(ctypes.byref(heads), 40, ctypes.byref(view), P(table), 3, 4, P(lens), P(ends), 0.125, 1, P(out), P(lse), P(space), 0, torch.cuda.current_stream().cuda_stream)
    assert st == L.OK
    torch.cuda.synchronize()
    assert (space == 7).all() and torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ------------------------------------------------------- a run of them together


class Layer:
    """Attention of a decoder's layer: norms and rotation, the cache, attention over it."""

    def __init__(self, g, Hq, Hk, D, pages, page):
        self.Hq, self.Hk, self.D = Hq, Hk, D
        self.qw, self.kw = ((1 + 0.2 * torch.randn(D, generator=g)).cuda() for _ in range(2))
        self.freqs, self.mult = nv.rotary_frequencies(D, factor=4.0, scaling="parts", original_length=256)
        self.cache = nv.PagedCache.empty(pages, page, Hk, D, k_amax=torch.full((Hk,), 8.0).cuda(), v_amax=torch.full((Hk,), 6.0).cuda())

    def step(self, qkv, positions, slots, table, lens, ends):
        q, k, v = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + self.Hk], qkv[:, self.Hq + self.Hk:]
        q = nv.norm_rope_write(q, k, v, positions, self.freqs, self.cache, slots, q_weight=self.qw, k_weight=self.kw, multiplier=self.mult)
        return nv.cache_attention(q, self.cache, table, lens, ends)


def test_prompt_then_tokens():
    """Prompts, then tokens one by one, against the same steps in 64 bits on what the cache holds."""
    g = gen(20)
    Hq, Hk, D, page = 8, 2, 64, 16
    prompt = [37, 90, 1]
    table, pages = tables(g, [p + 8 for p in prompt], page)
    layer = Layer(g, Hq, Hk, D, pages, page)
    slot = lambda b, j: int(table[b, j // page]) * page + j % page
    done = [0, 0, 0]
    for count in (prompt, [1, 1, 1], [2, 0, 3], [1, 1, 1]):
        where = [(b, done[b] + i) for b, n in enumerate(count) for i in range(n)]
        done = [a + n for a, n in zip(done, count)]
        T = len(where)
        qkv = randn(g, T, Hq + 2 * Hk, D)
        p = torch.tensor([j for _, j in where], dtype=torch.int32)
        slots = torch.tensor([slot(b, j) for b, j in where], dtype=torch.int32)
        lens, ends = torch.tensor(done, dtype=torch.int32), torch.cumsum(torch.tensor(count), 0).int()
        out, lse = layer.step(qkv.cuda(), p.cuda(), slots.cuda(), table.cuda(), lens.cuda(), ends.cuda())
        f = layer.freqs.cpu()
        q = A.norm_rope(qkv[:, :Hq], layer.qw, p, f, False, layer.mult).bfloat16()
        k = A.norm_rope(qkv[:, Hq:Hq + Hk], layer.kw, p, f, False, layer.mult).bfloat16()
        rk, rv = nv.read_cache(layer.cache, slots.cuda(), out_dtype=F32)
        # a 4-bit value is off by up to a quarter of the block's largest, and the block's scale by 2^-4 of itself
        for got, want in ((rk, k), (rv, qkv[:, Hq + Hk:])):
            top = R.f64(want).view(T, Hk, -1, 16).abs().amax(-1).repeat_interleave(16, -1)
            R.assert_near(got, R.f64(want), top * (1 / 6 + 2.0 ** -4) + 8 * 2.0 ** -9 / 448, "cache")
        c = layer.cache
        want, wl, off, loff = A.attention(q, A.cache_values(c.k, c.k_scale, c.k_amax), A.cache_values(c.v, c.v_scale, c.v_amax), table, lens, ends)
        R.assert_near(out, want, off, "out")
        R.assert_near(lse, wl, loff, "lse")


def test_streams_and_replays():
    """Captured steps replayed with new inputs, eager work between, on another stream, two graphs that share nothing but the cache's sizes."""
    g = gen(21)
    Hq, Hk, D, page = 8, 2, 128, 16
    lens = [700, 33, 150, 1]
    table, pages = tables(g, lens, page)
    a, b = Layer(g, Hq, Hk, D, pages, page), Layer(g, Hq, Hk, D, pages, page)
    slots = torch.tensor([int(table[i, (l - 1) // page]) * page + (l - 1) % page for i, l in enumerate(lens)], dtype=torch.int32).cuda()
    p, table, length = torch.tensor([l - 1 for l in lens], dtype=torch.int32).cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    for layer in (a, b):
        filled_ = filled(g, pages, page, Hk, D)
        for name in ("k", "k_scale", "v", "v_scale"):
            getattr(layer.cache, name).copy_(getattr(filled_, name))
    qkv, more = torch.zeros(4, Hq + 2 * Hk, D, dtype=BF, device="cuda"), torch.zeros(70, Hq, D, dtype=BF, device="cuda")
    ends = torch.tensor([3, 3, 60, 64], dtype=torch.int32).cuda()
    train = torch.zeros(90, Hq, D, dtype=BF, device="cuda")
    pos = torch.arange(90, dtype=torch.int32).cuda()
    run = lambda layer: (*layer.step(qkv, p, slots, table, length, None), *nv.cache_attention(more, layer.cache, table, length, ends),
                         *nv.norm_rope_backward(train, train[:, :Hk], train, train[:, :Hk], pos, layer.freqs, q_weight=layer.qw, k_weight=layer.kw))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(a), run(b)
    torch.cuda.synchronize()
    graphs = []
    for layer in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run(layer)
        graphs.append((graph, got, layer))
    for i in range(5):
        qkv.copy_(randn(g, *qkv.shape))
        more.copy_(randn(g, *more.shape))
        train.copy_(randn(g, *train.shape))
        for graph, got, layer in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for graph, got, layer in graphs:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                want = run(layer)
            side.synchronize()
            for x, y in zip(got, want):
                assert torch.equal(x, y), i


def test_example_runs():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_layer.py")
    spec = importlib.util.spec_from_file_location("attention_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    out, last, cross, grads, layer = mod.main(prompts=(70, 0, 1), heads=4, kv_heads=2, dim=64, tokens=2)
    assert out.shape == (71, 4, 64) and last.shape == cross.shape == (3, 4, 64) and layer.lens.tolist() == [72, 2, 3]
    assert [tuple(t.shape) for t in grads] == [(71, 4, 64), (71, 2, 64), (64,), (64,)]
    assert all(torch.isfinite(t).all() and t.any() for t in (out, last, cross, *grads))
