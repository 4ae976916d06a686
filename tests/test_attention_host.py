"""Attention on an NVFP4 cache without a GPU: bad arguments are refused on the host
with the documented status before anything is launched (fake, never-dereferenced
device addresses), the binding refuses CPU tensors, launches stay inside the
dispatch limits, and the 64-bit definitions that the GPU tests use hold against
values worked out by hand and, the gradient, against differences."""
import ctypes
import math
import random

import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv
from fp4_block_quantization_nvfp4_amd import _lib as L
from tests import attention_ref as A

X = 1 << 20  # a fake, 256-byte-aligned device address (never dereferenced)
BIG = 1 << 40
ref = ctypes.byref


def heads(at=X, heads=4, token=512, head=64):
    return L.Heads(at, heads, token, head)


def cache(k=X, ks=X, v=X, vs=X, ka=X, va=X, pages=8, page=16, heads=2, dim=64):
    return L.Cache(k, ks, v, vs, ka, va, pages, page, heads, dim)


def rope(positions=X, freqs=X, rotated=32, interleaved=0, multiplier=1.0, eps=1e-6, qw=X, kw=X):
    return L.Rope(positions, freqs, rotated, interleaved, multiplier, eps, qw, kw)


ROWS = [
    (dict(q=heads(at=None)), L.E_NULL), (dict(q=heads(at=X + 8)), L.E_ALIGN), (dict(q=heads(token=4)), L.E_ALIGN),
    (dict(q=heads(head=12)), L.E_ALIGN), (dict(q=heads(heads=-1)), L.E_SHAPE), (dict(q=heads(heads=65537)), L.E_RANGE),
    (dict(q=heads(token=BIG + 8)), L.E_RANGE), (dict(q=heads(head=-BIG - 8)), L.E_RANGE), (dict(q=None), L.E_NULL),
    (dict(T=-1), L.E_SHAPE), (dict(T=1 << 31), L.E_RANGE), (dict(T=1 << 26), L.E_RANGE), (dict(dt=2), L.E_DTYPE),
]
ROPE = [
    (dict(r=None), L.E_NULL), (dict(r=rope(rotated=24)), L.E_SHAPE), (dict(r=rope(rotated=-16)), L.E_SHAPE),
    (dict(r=rope(rotated=80)), L.E_SHAPE), (dict(r=rope(eps=-1.0)), L.E_ARG), (dict(r=rope(eps=float("nan"))), L.E_ARG),
    (dict(r=rope(multiplier=float("inf"))), L.E_ARG), (dict(r=rope(positions=None)), L.E_NULL), (dict(r=rope(freqs=None)), L.E_NULL),
    (dict(r=rope(positions=X + 2)), L.E_ALIGN), (dict(r=rope(freqs=X + 4)), L.E_ALIGN), (dict(r=rope(qw=X + 4)), L.E_ALIGN),
    (dict(r=rope(kw=X + 8)), L.E_ALIGN),
]


def at(x):
    return None if x is None else ref(x)


@pytest.mark.parametrize("kw,status", ROWS + ROPE + [
    (dict(k=heads(at=None)), L.E_NULL), (dict(k=heads(token=2)), L.E_ALIGN), (dict(D=8), L.E_SHAPE), (dict(D=72), L.E_SHAPE),
    (dict(D=528), L.E_RANGE), (dict(qo=None), L.E_NULL), (dict(ko=None), L.E_NULL), (dict(qo=X + 8), L.E_ALIGN), (dict(ko=X + 4), L.E_ALIGN),
    (dict(T=0, q=heads(at=None), k=heads(at=None), qo=None, ko=None), L.OK),
    (dict(q=heads(at=None, heads=0), k=heads(at=None, heads=0), qo=None, ko=None), L.OK)])
def test_norm_rope_rejects(kw, status):
    a = dict(q=heads(), k=heads(), dt=L.BF16, T=4, D=64, r=rope(), qo=X, ko=X) | kw
    assert L.lib().nvfp4_norm_rope(at(a["q"]), at(a["k"]), a["dt"], a["T"], a["D"], at(a["r"]), a["qo"], a["ko"], None) == status


@pytest.mark.parametrize("kw,status", ROWS + ROPE + [
    (dict(dq=heads(heads=3)), L.E_SHAPE), (dict(dk=heads(heads=5)), L.E_SHAPE), (dict(dq=heads(at=None)), L.E_NULL),
    (dict(dk=heads(at=X + 2)), L.E_ALIGN), (dict(qo=None), L.E_NULL), (dict(ko=None), L.E_NULL), (dict(dw=None), L.E_NULL),
    (dict(ws=None), L.E_NULL), (dict(n=2 * 64 * 4 - 1), L.E_ARG), (dict(dw=X + 8), L.E_ALIGN), (dict(ws=X + 8), L.E_ALIGN),
    (dict(qo=X + 8), L.E_ALIGN), (dict(T=0, r=rope(qw=None, kw=None), dw=None, ws=None, qo=None, ko=None), L.OK),
    (dict(T=0, dw=None), L.E_NULL)])
def test_norm_rope_backward_rejects(kw, status):
    a = dict(q=heads(), k=heads(), dq=heads(), dk=heads(), dt=L.BF16, T=4, D=64, r=rope(), qo=X, ko=X, dw=X, ws=X) | kw
    n = a.get("n", L.lib().nvfp4_norm_rope_backward_workspace_bytes(a["T"], a["D"]))
    assert L.lib().nvfp4_norm_rope_backward(at(a["dq"]), at(a["dk"]), at(a["q"]), at(a["k"]), a["dt"], a["T"], a["D"], at(a["r"]),
                                            a["qo"], a["ko"], a["dw"], a["ws"], n, None) == status


def test_norm_rope_backward_without_weights_reads_no_inputs():
    """Strides and addresses of the inputs matter only where a weight needs them."""
    none = heads(at=None, token=3)
    r = rope(qw=None, kw=None)
    assert L.lib().nvfp4_norm_rope_backward(ref(heads(at=None)), ref(heads()), ref(none), ref(none), L.BF16, 4, 64, ref(r), X, X, None, None,
                                            0, None) == L.E_NULL  # the gradients are needed
    assert L.lib().nvfp4_norm_rope_backward(ref(heads()), ref(heads()), ref(none), ref(none), L.BF16, 4, 64, ref(rope(kw=None)), X, X, X, X,
                                            4096, None) == L.E_NULL


CACHE = [
    (dict(c=None), L.E_NULL), (dict(c=cache(pages=-1)), L.E_SHAPE), (dict(c=cache(page=8)), L.E_SHAPE), (dict(c=cache(page=48)), L.E_SHAPE),
    (dict(c=cache(page=1 << 17)), L.E_SHAPE), (dict(c=cache(heads=0)), L.E_SHAPE), (dict(c=cache(dim=24)), L.E_SHAPE),
    (dict(c=cache(dim=0)), L.E_SHAPE), (dict(c=cache(dim=528)), L.E_RANGE), (dict(c=cache(pages=1 << 27)), L.E_RANGE),
    (dict(c=cache(heads=65537)), L.E_RANGE), (dict(c=cache(k=None)), L.E_NULL), (dict(c=cache(ks=None)), L.E_NULL),
    (dict(c=cache(v=None)), L.E_NULL), (dict(c=cache(vs=None)), L.E_NULL), (dict(c=cache(k=X + 8)), L.E_ALIGN),
    (dict(c=cache(v=X + 4)), L.E_ALIGN), (dict(c=cache(ks=X + 1)), L.E_ALIGN), (dict(c=cache(vs=X + 1)), L.E_ALIGN),
    (dict(c=cache(ka=X + 2)), L.E_ALIGN), (dict(c=cache(va=X + 1)), L.E_ALIGN),
]
WRITE = CACHE + [
    (dict(k=None), L.E_NULL), (dict(v=None), L.E_NULL), (dict(k=heads(heads=3)), L.E_SHAPE), (dict(v=heads(heads=1)), L.E_SHAPE),
    (dict(k=heads(heads=2, at=None)), L.E_NULL), (dict(v=heads(heads=2, at=X + 8)), L.E_ALIGN), (dict(v=heads(heads=2, token=3)), L.E_ALIGN),
    (dict(dt=2), L.E_DTYPE), (dict(slots=None), L.E_NULL), (dict(slots=X + 2), L.E_ALIGN), (dict(T=-1), L.E_SHAPE), (dict(T=1 << 31), L.E_RANGE),
    (dict(T=1 << 27), L.E_RANGE), (dict(T=0, slots=None), L.OK),
]


@pytest.mark.parametrize("kw,status", WRITE)
def test_write_cache_rejects(kw, status):
    a = dict(k=heads(heads=2), v=heads(heads=2), dt=L.BF16, T=4, c=cache(), slots=X) | kw
    assert L.lib().nvfp4_write_cache(at(a["k"]), at(a["v"]), a["dt"], a["T"], at(a["c"]), a["slots"], None) == status


@pytest.mark.parametrize("kw,status", WRITE + ROPE + ROWS[:8] + [(dict(qo=None), L.E_NULL), (dict(qo=X + 8), L.E_ALIGN)])
def test_norm_rope_write_rejects(kw, status):
    a = dict(q=heads(), k=heads(heads=2), v=heads(heads=2), dt=L.BF16, T=4, r=rope(), c=cache(), slots=X, qo=X) | kw
    assert L.lib().nvfp4_norm_rope_write(at(a["q"]), at(a["k"]), at(a["v"]), a["dt"], a["T"], at(a["r"]), at(a["c"]), a["slots"], a["qo"],
                                         None) == status


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(T=-1), L.E_SHAPE), (dict(T=1 << 31), L.E_RANGE), (dict(T=1 << 27), L.E_RANGE), (dict(dt=2), L.E_DTYPE), (dict(slots=None), L.E_NULL),
    (dict(k=None), L.E_NULL), (dict(v=None), L.E_NULL), (dict(slots=X + 1), L.E_ALIGN), (dict(k=X + 8), L.E_ALIGN), (dict(v=X + 8), L.E_ALIGN),
    (dict(T=0, slots=None, k=None, v=None), L.OK)])
def test_read_cache_rejects(kw, status):
    a = dict(c=cache(), slots=X, T=4, k=X, v=X, dt=L.BF16) | kw
    assert L.lib().nvfp4_read_cache(at(a["c"]), a["slots"], a["T"], a["k"], a["v"], a["dt"], None) == status


@pytest.mark.parametrize("kw,status", CACHE[:10] + CACHE[11:] + [
    (dict(q=None), L.E_NULL), (dict(q=heads(heads=3)), L.E_SHAPE), (dict(q=heads(at=None)), L.E_NULL), (dict(q=heads(at=X + 8)), L.E_ALIGN),
    (dict(q=heads(token=4)), L.E_ALIGN), (dict(q=heads(heads=-2)), L.E_SHAPE), (dict(c=cache(dim=48)), L.E_SHAPE), (dict(c=cache(dim=288)), L.E_RANGE),
    (dict(T=-1), L.E_SHAPE), (dict(T=1 << 31), L.E_RANGE), (dict(B=-1), L.E_SHAPE), (dict(width=0), L.E_SHAPE), (dict(width=(1 << 26) + 1), L.E_RANGE),
    (dict(B=(1 << 20) + 1), L.E_RANGE), (dict(B=1 << 20, c=cache(heads=8), q=heads(heads=8)), L.E_RANGE),
    (dict(B=1 << 15, width=1 << 17), L.E_RANGE), (dict(ends=None), L.E_SHAPE), (dict(scale=0.0), L.E_ARG), (dict(scale=-1.0), L.E_ARG),
    (dict(scale=float("inf")), L.E_ARG), (dict(scale=float("nan")), L.E_ARG), (dict(table=None), L.E_NULL), (dict(lens=None), L.E_NULL),
    (dict(out=None), L.E_NULL), (dict(lse=None), L.E_NULL), (dict(ws=None), L.E_NULL), (dict(n=100), L.E_ARG), (dict(table=X + 2), L.E_ALIGN),
    (dict(lens=X + 1), L.E_ALIGN), (dict(ends=X + 2), L.E_ALIGN), (dict(out=X + 8), L.E_ALIGN), (dict(lse=X + 2), L.E_ALIGN), (dict(ws=X + 8), L.E_ALIGN),
    (dict(T=0, table=None, lens=None, out=None, lse=None, ws=None), L.OK), (dict(q=heads(heads=0), out=None, ws=None), L.OK)])
def test_cache_attention_rejects(kw, status):
    a = dict(q=heads(), T=6, c=cache(), table=X, B=3, width=40, lens=X, ends=X, scale=0.125, out=X, lse=X, ws=X) | kw
    Hq = a["q"].heads if a["q"] else 4
    n = a.get("n", L.lib().nvfp4_cache_attention_workspace_bytes(a["T"], Hq, at(a["c"]), a["B"], a["width"]))
    assert L.lib().nvfp4_cache_attention(at(a["q"]), a["T"], at(a["c"]), a["table"], a["B"], a["width"], a["lens"], a["ends"], a["scale"], 1,
                                         a["out"], a["lse"], a["ws"], n, None) == status


def test_cpu_tensors_are_refused():
    x = torch.zeros(3, 2, 32, dtype=torch.bfloat16)
    i, f = torch.zeros(3, dtype=torch.int32), torch.ones(16, dtype=torch.float64)
    c = nv.PagedCache.empty(2, 16, 2, 32, device="cpu")
    assert c.k.shape == (2, 2, 16, 16) and c.v_scale.shape == (2, 2, 16, 2)
    for call in (lambda: nv.norm_rope(x, x, i, f), lambda: nv.norm_rope_backward(x, x, x, x, i, f),
                 lambda: nv.norm_rope_write(x, x, x, i, f, c, i), lambda: nv.write_cache(c, x, x, i), lambda: nv.read_cache(c, i),
                 lambda: nv.cache_attention(x, c, torch.zeros(3, 1, dtype=torch.int32), i)):
        with pytest.raises(ValueError, match="device tensor"):
            call()


# ----------------------------------------------------------------- launches

ROPE_K, ROPE_BWD, ROPE_SUM, READ, SPLIT, TILES, JOIN = range(7)


def plan(entry, T, Hq=4, Hk=2, D=64, B=1, keys=16):
    out = (ctypes.c_int64 * 16)()
    st = L.lib().nvfp4_selftest_attention_plan(entry, T, Hq, Hk, D, B, keys, out)
    return st, [list(out[4 * i:4 * i + 4]) for i in range(4)]


def ceil(a, b):
    return -(-a // b)


def check_limits(launch, what):
    _, x, y, lanes = launch
    assert 1 <= x < 1 << 31 and x * lanes < 1 << 32 and 1 <= y <= 65535 and 64 <= lanes <= 1024 and lanes % 64 == 0, (what, launch)


def test_launches_stay_in_the_limits():
    rng = random.Random(3)
    got = {}
    top = [(0, (1 << 31) - 1, 0, 1, 16 // 16 * 16), (4, 1 << 29, 1, 1, 16), (3, 1 << 29, 1, 1, 16), (1, 1 << 29, 1, 1, 16)]
    for i in range(6000):
        entry = rng.randrange(7)
        Hk = int(2 ** rng.uniform(0, 8))
        Hq = Hk * int(2 ** rng.uniform(0, 7)) if entry >= 5 else int(2 ** rng.uniform(0, 12))
        D = 32 * rng.randint(1, 8) if entry >= 5 else 16 * rng.randint(1, 32)
        T, B, keys = int(2 ** rng.uniform(0, 31)), int(2 ** rng.uniform(0, 20)), 16 * int(2 ** rng.uniform(0, 26))
        if i < len(top):
            entry, T, Hq, Hk, D = top[i]
        if entry == 6:
            T = B
        st, launches = plan(entry, T, Hq, Hk, D, B, keys)
        if st != L.OK:
            assert st == L.E_RANGE
            continue
        what = (entry, T, Hq, Hk, D, B, keys)
        for l in launches:
            if l[1]:
                check_limits(l, what)
                got[l[0]] = got.get(l[0], 0) + 1
        first = launches[0]
        if entry in (0, 2, 3):
            assert first[0] == ROPE_K
        if entry == 4:
            assert first[1] * 256 >= T * Hk * (D // 16) and first[2] == 2
        if entry >= 5:
            split, tiles, join, _ = launches
            c, G = cache(heads=Hk, dim=D), Hq // Hk
            need = L.lib().nvfp4_cache_attention_workspace_bytes(T, Hq, ref(c), B, keys // 16)
            assert (join[1] > 0) == (keys > 64)
            least = (keys > 64) * split[1] * 4 * (2 * (16 * D + 32) * 4 + 32)
            assert need >= least and least % 16 == 0
            joined = 4 * split[1]
            if tiles[1]:  # units of any split of T queries over B sequences and those of none, each in as many parts
                rows = tiles[3] // 2
                units = (ceil(T * G, rows) + B) * Hk
                assert entry == 5 and rows in (128, 256) and tiles[1] % units == 0
                parts = tiles[1] // units
                assert 1 <= parts <= 16
                if parts > 1:
                    assert need >= least + units * (32 + parts * rows * (D + 2) * 4) and units * parts <= 1024 and keys > 64
                    joined += units * rows // 16
            else:
                assert entry == 6 or T * G <= 128
            assert join[1] == (joined if keys > 64 else 0)
    assert set(got) == set(range(7)) and min(got.values()) > 20


def test_plan_refusals():
    assert plan(7, 4)[0] == L.E_ARG and plan(-1, 4)[0] == L.E_ARG and plan(0, 4, D=24)[0] == L.E_SHAPE
    assert plan(5, 4, Hq=3)[0] == L.E_SHAPE and plan(5, 4, D=48)[0] == L.E_SHAPE and plan(5, 4, D=288)[0] == L.E_RANGE
    assert plan(0, 1 << 31)[0] == L.E_RANGE and plan(5, 4, keys=(1 << 30) + 16)[0] == L.E_RANGE
    assert L.lib().nvfp4_selftest_attention_plan(0, 4, 4, 2, 64, 1, 16, None) == L.E_NULL


# ------------------------------------------------- frequencies and definitions


def test_frequencies():
    f, m = nv.rotary_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and m == 1.0 and f[0] == 1.0 and math.isclose(f[31], 10000.0 ** (-62 / 64), rel_tol=1e-14)
    g, m = nv.rotary_frequencies(64, factor=8, scaling="linear", device="cpu")
    assert torch.allclose(g, f / 8, rtol=1e-15, atol=0) and m == 1.0
    g, m = nv.rotary_frequencies(64, factor=8, scaling="base", device="cpu")
    assert g[0] == 1.0 and math.isclose(g[31], f[31] / 8, rel_tol=1e-12) and m == 1.0
    g, m = nv.rotary_frequencies(64, factor=8, scaling="parts", original_length=4096, device="cpu")
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(g[turns > 40], f[turns > 40]) and torch.allclose(g[turns < 0.8], f[turns < 0.8] / 8, rtol=1e-15, atol=0)
    assert ((g <= f) & (g >= f / 8)).all() and math.isclose(m, 0.1 * math.log(8) + 1)
    assert nv.rotary_frequencies(0, device="cpu")[0].numel() == 0
    for bad in (dict(dim=3), dict(dim=-2), dict(dim=8, base=0.0), dict(dim=8, factor=0.5), dict(dim=8, scaling="other"), dict(dim=8, scaling="parts", factor=2)):
        with pytest.raises(ValueError):
            nv.rotary_frequencies(**bad, device="cpu")


def test_rotation_definition():
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0]]], dtype=torch.float64)
    p, f = torch.tensor([1]), torch.tensor([math.pi / 2, math.pi], dtype=torch.float64)
    half = A.rotate(x, p, f, False)
    assert torch.allclose(half, torch.tensor([[[-3.0, -2.0, 1.0, -4.0, 5.0]]], dtype=torch.float64), atol=1e-12)
    pairs = A.rotate(x, p, f, True, multiplier=2.0)
    assert torch.allclose(pairs, torch.tensor([[[-4.0, 2.0, -6.0, -8.0, 5.0]]], dtype=torch.float64), atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_against_differences(interleaved):
    g = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(*s, dtype=torch.float64, generator=g)
    x, w, dz = r(3, 2, 32), r(32), r(3, 2, 32)
    p, f = torch.tensor([0, 7, 90001]), nv.rotary_frequencies(16, device="cpu")[0]
    dx, dw, _, _ = A.norm_rope_gradient(dz, x, w, p, f, interleaved, 1.3)
    loss = lambda x, w: (A.norm_rope(x, w, p, f, interleaved, 1.3) * dz).sum()
    for _ in range(4):
        a, b, e = r(3, 2, 32), r(32), 1e-5
        slope = (loss(x + e * a, w + e * b) - loss(x - e * a, w - e * b)) / (2 * e)
        assert math.isclose(slope, (dx * a).sum() + (dw * b).sum(), rel_tol=1e-7, abs_tol=1e-8)


def test_attention_definition():
    """Two keys of weights 1/4 and 3/4; a query that sees none; pages in any order."""
    k = torch.zeros(2, 1, 16, 32, dtype=torch.float64)
    v = torch.zeros(2, 1, 16, 32, dtype=torch.float64)
    k[1, 0, 1, 0] = math.log(3)
    v[1, 0, 0, 5], v[1, 0, 1, 5] = 4.0, 8.0
    q = torch.zeros(3, 1, 32, dtype=torch.bfloat16)
    q[:, 0, 0] = 1.0
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    out, lse, _, _ = A.attention(q, k, v, table, torch.tensor([2]), torch.tensor([3]), scale=1.0)
    assert out[0].abs().max() == 0 and lse[0, 0] == -math.inf
    assert out[1, 0, 5] == 4.0 and lse[1, 0] == 0.0
    assert math.isclose(out[2, 0, 5], 7.0) and math.isclose(lse[2, 0], math.log(4))
    out, _, _, _ = A.attention(q, k, v, table, torch.tensor([2]), torch.tensor([3]), scale=1.0, causal=False)
    assert torch.allclose(out[:, 0, 5], torch.full((3,), 7.0, dtype=torch.float64))
