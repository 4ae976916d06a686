"""The operators of attention whose keys and values are stored in NVFP4, as cases
to be measured: norms of queries and keys for each head with the rotation of
their positions, with gradients; a paged cache that is quantized as it is
written, and read back; attention over that cache, for single tokens, prompts
and an encoder's states.

`own` false: plain torch operations in 32 bits (angles, and values that are
about to be quantized, in 64).  `own` true: this repository's kernels.  Both
take what `prepare` makes.

Cache: `pages` pages of `page` slots for each of Hk heads.  A slot's row of D
elements is held as e2m1 codes, two per byte, the even element in the low
nibble [pages, Hk, page, D / 2], and an e4m3 scale for 16 elements [pages, Hk,
page, D / 16]; the second-level scale is amax / (6 * 448) for each head, or none.
A sequence's keys lie in the slots of its row of the page table, in order.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6
FLT_MAX = 3.4028234663852886e38
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one new token's queries and keys while serving: latency counts
        dict(name="positions, one token", op="rope", T=1, Hq=32, Hk=8, D=128, R=128, layout="half", far=32768, norm=True, dtype="bf16", train=False),
        # a training step's queries and keys, with the gradients of both and of the norms' weights
        dict(name="positions, training", op="rope", T=8192, Hq=32, Hk=8, D=128, R=128, layout="half", far=8192, norm=True, dtype="bf16", train=True),
        # 32 bits, a part of an odd head rotated, interleaved pairs, positions of a long context
        dict(name="positions, odd, training", op="rope", T=1021, Hq=6, Hk=2, D=80, R=32, layout="interleaved", far=1000000, norm=True, dtype="f32", train=True),
        # a decoding step of 64 sequences: norms, rotation and the cache's new rows in one call, then those rows read back
        dict(name="cache, decoding", op="cache", T=64, Hq=32, Hk=8, D=128, R=128, layout="half", far=32768, page=64, amax=True, fused=True, dtype="bf16"),
        # a prompt's keys and values
        dict(name="cache, prompt", op="cache", T=16384, Hq=0, Hk=8, D=128, R=0, layout="half", far=1, page=64, amax=False, fused=False, dtype="bf16"),
        # odd sizes: small pages, keys without a second-level scale, a quarter of the head rotated, padded rows that are not written
        dict(name="cache, odd", op="cache", T=777, Hq=9, Hk=3, D=192, R=48, layout="half", far=100000, page=16, amax=False, fused=True, dtype="bf16"),
        # one new token of one conversation: latency counts
        dict(name="attention, one sequence", op="attention", B=1, n=1, keys=1000, Hq=32, Hk=8, D=128, page=64, amax=True, causal=True),
        # a decoding step of 64 conversations of different lengths
        dict(name="attention, decoding", op="attention", B=64, n=1, keys=8192, Hq=32, Hk=8, D=128, page=64, amax=True, causal=True),
        # two long documents
        dict(name="attention, long", op="attention", B=2, n=1, keys=131072, Hq=32, Hk=8, D=128, page=256, amax=True, causal=True),
        # prompts that fill the cache for the first time
        dict(name="attention, prompt", op="attention", B=2, n=8192, keys=8192, Hq=32, Hk=8, D=128, page=64, amax=True, causal=True),
        # ragged pieces of prompts behind what is in the cache, odd heads, small pages; sequences without queries or keys
        dict(name="attention, odd", op="attention", B=7, n=301, keys=1999, Hq=15, Hk=5, D=96, page=16, amax=False, causal=True),
        # a decoder's tokens over the states of an encoder
        dict(name="attention, encoder", op="attention", B=16, n=64, keys=1500, Hq=16, Hk=16, D=64, page=64, amax=True, causal=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope", "cache", "attention", "attention"))
    Hk = rng.choice((1, 2, 3, 4, 5, 8, 16))
    Hq = Hk * rng.choice((1, 2, 3, 4, 7, 8))
    if op != "attention":
        D = 16 * rng.randint(2, 16)
        fused = op == "rope" or rng.random() < 0.7
        c = dict(op=op, T=_log(rng, 1, (8192 * 40 * 128) // ((Hq + Hk) * D)), Hq=Hq if fused else 0, Hk=Hk, D=D, R=16 * rng.randint(1, D // 16) if fused else 0,
                 layout=rng.choice(("half", "interleaved")), far=_log(rng, 100, 1000000))
        if op == "rope":
            return dict(c, norm=rng.random() < 0.8, dtype=rng.choice(("bf16", "f32")) if c["T"] * (Hq + Hk) * D < 1 << 24 else "bf16", train=rng.random() < 0.6)
        return dict(c, page=rng.choice((16, 32, 64, 128)), amax=rng.random() < 0.5, fused=fused, dtype=rng.choice(("bf16", "bf16", "f32")))
    D, page = 32 * rng.randint(1, 8), rng.choice((16, 32, 64, 128, 256))
    causal = rng.random() < 0.7
    if rng.random() < 0.5:  # single tokens, or a few each
        n = rng.choice((1, 1, 1, 2, 5))
        B = _log(rng, 1, 64)
        keys = _log(rng, 1, max(2, (1 << 28) // (B * Hk * D)))
        keys = min(keys, 131072)
    else:
        B = _log(rng, 1, 8)
        n = _log(rng, 1, 4096)
        keys = max(n, _log(rng, 16, 8192)) if causal else _log(rng, 16, 8192)
        while B * n * keys * Hq * D > 2 * 8192 * 4096 * 32 * 128 or B * keys * Hk * D > 1 << 28:
            B, n = (B + 1) // 2, (n + 1) // 2
    return dict(op=op, B=B, n=n, keys=keys, Hq=Hq, Hk=Hk, D=D, page=page, amax=rng.random() < 0.5, causal=causal)


# ------------------------------------------------------------------ inputs


def _freqs(R):
    """Angle of one step for each pair, 64 bits."""
    return torch.tensor([10000.0 ** (-2 * i / R) for i in range(R // 2)], dtype=torch.float64, device="cuda")


def _counts(case, seed):
    """Queries and keys of each sequence: the case's own numbers for one of them, fewer for the others, in an order that goes by the seed.
    Of several pieces of prompts one has no query and one no key."""
    c = torch.Generator().manual_seed(case["B"] * 1009 + case["keys"])
    B, n, keys = case["B"], case["n"], case["keys"]
    part = 0.2 + 0.8 * torch.rand(2, B, generator=c)
    part[:, 0] = 1.0
    ns = [n] * B if n <= 5 else [max(1, round(n * p)) for p in part[0].tolist()]
    ks = [max(1, round(keys * p)) for p in part[1].tolist()]
    if case["causal"]:
        ks = [max(a, b) for a, b in zip(ns, ks)] if n < keys else list(ns)
    if B >= 5 and 5 < n < keys:
        ns[2], ks[3] = 0, 0
    order = torch.randperm(B, generator=torch.Generator().manual_seed(seed * 11 + 5)).tolist()
    return [ns[i] for i in order], [ks[i] for i in order]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 13 + 1)
    s = dict(case)

    def rand(*shape, dtype="bf16", by=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * by).to(DTYPE[dtype])

    def whole(hi, *shape):
        return torch.randint(hi, shape, device="cuda", generator=g, dtype=torch.int32)

    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if case["op"] == "attention":
        ns, ks = _counts(case, seed)
        page = case["page"]
        wide = max(1, (max(ks) + page - 1) // page)
        pages = sum((k + page - 1) // page for k in ks) + 1
        order, at = torch.randperm(pages, device="cuda", generator=g).int(), 0
        s["table"] = torch.full((len(ks), wide), -1, dtype=torch.int32, device="cuda")
        for b, k in enumerate(ks):  # rows past a sequence's last page stay -1
            m = (k + page - 1) // page
            s["table"][b, :m] = order[at:at + m]
            at += m
        for x, by in (("k", 1.0), ("v", 0.5)):
            amax = 4.5 * by * (1 + torch.rand(Hk, device="cuda", generator=g)) if case["amax"] else None
            parts = [_quantize(rand(min(512, pages - i), Hk, page, D, by=by).float(), None if amax is None else amax.view(-1, 1, 1)) for i in range(0, pages, 512)]
            s[x], s[x + "_scale"] = (torch.cat(p).contiguous() for p in zip(*parts))
            s[x + "_amax"] = amax
        # queries about as sharp as trained ones: most of the weight on some tens of keys
        s["q"] = rand(sum(ns), Hq, D, by=1.5)
        s["lens"] = torch.tensor(ks, dtype=torch.int32, device="cuda")
        s["ends"] = None if all(n == 1 for n in ns) else torch.cumsum(torch.tensor(ns), 0).int().cuda()
        s["counts"] = list(zip(ns, ks))
        return s
    T, dt = case["T"], case["dtype"]
    # one projection gives queries, keys and values of a token side by side
    qkv = rand(T, Hq + 2 * Hk, D, dtype=dt, by=1.5)
    s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    s["positions"] = whole(case["far"], T)
    s["freqs"] = _freqs(case["R"])
    weights = case.get("norm", case.get("fused"))
    s["q_weight"], s["k_weight"] = ((1 + 0.2 * rand(D, dtype="f32")) if weights else None for _ in range(2))
    if case["op"] == "rope":
        if case["train"]:
            s["dq"], s["dk"] = rand(T, Hq, D, dtype=dt), rand(T, Hk, D, dtype=dt)
        return s
    pages = (T + case["page"] - 1) // case["page"] + 3
    slots = torch.randperm(pages, device="cuda", generator=g).repeat_interleave(case["page"]) * case["page"]
    slots = (slots + torch.arange(case["page"], device="cuda").repeat(pages))[:T].int()
    if T >= 500 and case["page"] == 16:  # padding between prompts
        slots[whole(T, T // 50).long()] = -1
    s["slots"] = slots.contiguous()
    for x in "kv":
        s[x + "_cache"] = torch.zeros(pages, Hk, case["page"], D // 2, dtype=torch.uint8, device="cuda")
        s[x + "_scale"] = torch.zeros(pages, Hk, case["page"], D // 16, dtype=torch.uint8, device="cuda")
        s[x + "_amax"] = 6 + 2 * torch.rand(Hk, device="cuda", generator=g) if case["amax"] else None
    return s


# -------------------------------------------------------------- plain forms


def _quantize(x, amax=None):
    """32-bit rows [..., D] -> codes [..., D / 2], scale bytes [..., D / 16]; amax with the rows' leading dimensions."""
    b = x.view(*x.shape[:-1], -1, 16)
    a = b.abs().amax(-1)
    if amax is None:
        dec, sigma = 1.0, a / 6
    else:
        dec = amax / 2688.0
        sigma = a * ((2688.0 / amax).clamp(max=FLT_MAX) * torch.tensor(1 / 6, device=x.device))
    scale = sigma.clamp(max=448.0).to(F8)
    rho = (1.0 / (scale.float() * dec)).clamp(max=FLT_MAX)
    v = (b.abs() * rho.unsqueeze(-1)).clamp(max=6.0)
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    v = torch.round(v / step) * step  # ties to even: the grid's even codes are the even multiples
    grid = torch.tensor(E2M1, device=x.device)
    code = torch.bucketize(v, grid).to(torch.uint8) | (torch.signbit(b).to(torch.uint8) << 3)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _values(codes, scales, amax=None):
    """32-bit values; amax with the rows' leading dimensions."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = grid[torch.stack((codes & 15, codes >> 4), -1).long()].flatten(-2)
    v = v * scales.view(F8).float().repeat_interleave(16, -1)
    return v if amax is None else v * (amax / 2688.0)


def _rotate(y, cos, sin, layout, back=False):
    """Pairs of the first 2 * cos.shape[-1] elements of y [T, H, D] turned by their angles (back: the other way)."""
    R = 2 * cos.shape[-1]
    if R == 0:
        return y
    a, b = (y[..., :R // 2], y[..., R // 2:R]) if layout == "half" else (y[..., 0:R:2], y[..., 1:R:2])
    cos, sin = cos.unsqueeze(1), (-sin if back else sin).unsqueeze(1)
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.cat((a, b), -1) if layout == "half" else torch.stack((a, b), -1).flatten(-2)
    return torch.cat((turned, y[..., R:]), -1)


def _angles(s, wide):
    a = s["positions"].double().unsqueeze(1) * s["freqs"]
    return (torch.cos(a), torch.sin(a)) if wide else (torch.cos(a).float(), torch.sin(a).float())


def _norm_rope(x, w, cos, sin, layout, wide):
    y = x.double() if wide else x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
    return _rotate(y, cos, sin, layout).to(x.dtype)


def _plain_rope(s):
    cos, sin = _angles(s, False)
    out = dict(q=_norm_rope(s["q"], s["q_weight"], cos, sin, s["layout"], False), k=_norm_rope(s["k"], s["k_weight"], cos, sin, s["layout"], False))
    if s["train"]:
        for x in "qk":
            dy, w, v = _rotate(s["d" + x].float(), cos, sin, s["layout"], True), s[x + "_weight"], s[x].float()
            if w is not None:
                rstd = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
                n = v * rstd
                out[f"d{x}_weight"] = (dy * n).sum((0, 1))
                d = dy * w
                dy = rstd * (d - n * (d * n).mean(-1, keepdim=True))
            out["d" + x] = dy.to(s[x].dtype)
    return out


def _plain_cache(s):
    out, k = {}, s["k"]
    if s["fused"]:
        cos, sin = _angles(s, True)
        out["q"] = _norm_rope(s["q"], s["q_weight"], cos, sin, s["layout"], True)
        k = _norm_rope(k, s["k_weight"], cos, sin, s["layout"], True)
    written = s["slots"] >= 0
    at = s["slots"].clamp(min=0).long()
    for x, rows in (("k", k), ("v", s["v"])):
        amax = None if s[x + "_amax"] is None else s[x + "_amax"].view(-1, 1)
        codes, scales = _quantize(rows.float(), amax)
        cache, scale = s[x + "_cache"], s[x + "_scale"]
        page, slot = at[written] // s["page"], at[written] % s["page"]
        cache[page, :, slot], scale[page, :, slot] = codes[written], scales[written]
        got = _values(cache[at // s["page"], :, at % s["page"]], scale[at // s["page"], :, at % s["page"]], None if amax is None else amax)
        out[x] = torch.where(written.view(-1, 1, 1), got, 0.0).to(DTYPE[s["dtype"]])
    return out


def _plain_attention(s):
    Hq, Hk, D, page = s["Hq"], s["Hk"], s["D"], s["page"]
    G, t, outs, lses = Hq // Hk, 0, [], []
    for b, (n, L) in enumerate(s["counts"]):
        if n == 0:
            continue
        q = s["q"][t:t + n].float()
        t += n
        if L == 0:
            outs.append(torch.zeros(n, Hq, D, device=q.device))
            lses.append(torch.full((n, Hq), -math.inf, device=q.device))
            continue
        pages = s["table"][b, :(L + page - 1) // page].long()
        k, v = (_values(s[x][pages], s[x + "_scale"][pages], None if s[x + "_amax"] is None else s[x + "_amax"].view(-1, 1, 1)).transpose(0, 1).reshape(Hk, -1, D)[:, :L]
                for x in "kv")
        seen = None
        if s["causal"] and n > 1:
            seen = torch.arange(L, device=q.device) <= torch.arange(n, device=q.device).unsqueeze(1) + (L - n)
        o, l = torch.empty(n, Hq, D, device=q.device), torch.empty(n, Hq, device=q.device)
        for h in range(Hk):  # a head's scores at a time
            rows = q[:, h * G:(h + 1) * G].transpose(0, 1)  # [G, n, D]
            for i in range(0, G, 1 if n * L > 1 << 22 else G):
                part = rows[i:i + (1 if n * L > 1 << 22 else G)].contiguous()
                score = (part.view(-1, D) @ k[h].t()).view(-1, n, L) * D ** -0.5
                if seen is not None:
                    score = torch.where(seen, score, -math.inf)
                top = score.amax(-1, keepdim=True)
                p = torch.exp(score - top)
                total = p.sum(-1, keepdim=True)
                o[:, h * G + i:h * G + i + len(part)] = ((p.view(-1, L) @ v[h]).view(-1, n, D) / total).transpose(0, 1)
                l[:, h * G + i:h * G + i + len(part)] = (top + torch.log(total)).squeeze(-1).t()
        outs.append(o)
        lses.append(l)
    return dict(out=torch.cat(outs).bfloat16(), lse=torch.cat(lses))


# ------------------------------------------------------------ the framework


def _own(s):
    import fp4_block_quantization_nvfp4_amd as nv

    if s["op"] == "attention":
        cache = nv.PagedCache(s["k"], s["k_scale"], s["v"], s["v_scale"], k_amax=s["k_amax"], v_amax=s["v_amax"])
        out, lse = nv.cache_attention(s["q"], cache, s["table"], s["lens"], s["ends"], causal=s["causal"])
        return dict(out=out, lse=lse)
    how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], interleaved=s["layout"] == "interleaved", eps=EPS)
    if s["op"] == "rope":
        q, k = nv.norm_rope(s["q"], s["k"], s["positions"], s["freqs"], **how)
        out = dict(q=q, k=k)
        if s["train"]:
            dq, dk, dqw, dkw = nv.norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"], s["freqs"], **how)
            out.update(dq=dq, dk=dk)
            if dqw is not None:
                out.update(dq_weight=dqw, dk_weight=dkw)
        return out
    cache = nv.PagedCache(s["k_cache"], s["k_scale"], s["v_cache"], s["v_scale"], k_amax=s["k_amax"], v_amax=s["v_amax"])
    out = {}
    if s["fused"]:
        out["q"] = nv.norm_rope_write(s["q"], s["k"], s["v"], s["positions"], s["freqs"], cache, s["slots"], **how)
    else:
        nv.write_cache(cache, s["k"], s["v"], s["slots"])
    out["k"], out["v"] = nv.read_cache(cache, s["slots"], out_dtype=DTYPE[s["dtype"]])
    return out


def run(state):
    if own:
        return _own(state)
    return {"rope": _plain_rope, "cache": _plain_cache, "attention": _plain_attention}[state["op"]](state)


def work(case):
    """Inputs read once and outputs written once, whatever stays on the way between a case's calls; a multiply-add is two operations.
    Of attention the pairs of a query and a key that it sees."""
    size, Hq, Hk, D = {"bf16": 2, "f32": 4}, case["Hq"], case["Hk"], case["D"]
    if case["op"] == "rope":
        n = case["T"] * (Hq + Hk) * D
        return dict(bytes=n * size[case["dtype"]] * (4 if case["train"] else 2) + 4 * case["T"], flops=n * (24 if case["train"] else 9))
    if case["op"] == "cache":
        b, T = size[case["dtype"]], case["T"]
        n = T * (2 * Hq + 2 * Hk + 2 * Hk) * D * b + 2 * T * Hk * (D // 2 + D // 16) + 8 * T
        return dict(bytes=n, flops=T * (9 * Hq + 19 * Hk + 10 * Hk) * D)
    ns, ks = _counts(case, 0)
    pairs = sum(n * L - (n * (n - 1) // 2 if case["causal"] else 0) for n, L in zip(ns, ks) if L)
    rows = sum(L for n, L in zip(ns, ks) if n)
    return dict(bytes=rows * Hk * 2 * (D // 2 + D // 16) + sum(ns) * Hq * (4 * D + 4), flops=4 * D * Hq * pairs)


# -------------------------------------------------------------- in 64 bits


def _f32(v):
    """A step that the format defines in 32 bits, taken from 64."""
    return v.float().double()


def _exact_quantized(x, amax):
    """Values in 64 bits that the cache holds for rows x [T, H, D]; amax [H] or None.  The format's own steps are 32-bit ones, each rounded once."""
    b = x.double().reshape(*x.shape[:-1], -1, 16)
    a = b.abs().amax(-1)
    if amax is None:
        dec, sigma = torch.ones((), dtype=torch.float64, device=x.device), _f32(a / 6)
    else:
        A = amax.double().view(-1, 1)
        dec, enc = _f32(A / 2688), _f32(2688 / A).clamp(max=FLT_MAX)
        sigma = _f32(a * _f32(enc * _f32(torch.tensor(1 / 6, dtype=torch.float64, device=x.device))))
    sigma = sigma.clamp(max=448.0)
    unit = torch.exp2(torch.floor(torch.log2(sigma.clamp(min=2.0 ** -6))) - 3)
    scale = (torch.round(sigma / unit) * unit).clamp(max=448.0)
    rho = torch.where(scale > 0, _f32(1 / _f32(scale * dec)), math.inf).clamp(max=FLT_MAX)
    v = _f32(b * rho.unsqueeze(-1))
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    far = (v.abs().clamp(max=6.0).unsqueeze(-1) - grid).abs()
    far = far + torch.tensor([0.0, 1e-12] * 4, dtype=torch.float64, device=x.device)  # between two as near, the even code
    got = grid[far.argmin(-1)] * torch.where(torch.signbit(b), -1.0, 1.0)
    return (got * (scale * (dec if amax is not None else 1.0)).unsqueeze(-1)).reshape(x.shape)


def _turn(y, position, freqs, layout, back=False):
    """Rotation as a product of complex numbers, in 64 bits."""
    R = 2 * len(freqs)
    y = y.double()
    if R == 0:
        return y
    angle = position.double()[:, None] * freqs[None]
    unit = torch.polar(torch.ones_like(angle), -angle if back else angle)[:, None]
    got = y.clone()
    if layout == "half":
        z = torch.complex(y[..., :R // 2].contiguous(), y[..., R // 2:R].contiguous()) * unit
        got[..., :R // 2], got[..., R // 2:R] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:R:2].contiguous(), y[..., 1:R:2].contiguous()) * unit
        got[..., 0:R:2], got[..., 1:R:2] = z.real, z.imag
    return got


def _exact_rows(x, w, position, freqs, layout):
    y = x.double()
    if w is not None:
        y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + EPS) * w.double()
    return _turn(y, position, freqs, layout)


def exact(case, seed):
    s = prepare(case, seed)
    D, layout = case["D"], case.get("layout")
    if case["op"] == "rope":
        where = (s["positions"], s["freqs"], layout)
        out = dict(q=_exact_rows(s["q"], s["q_weight"], *where), k=_exact_rows(s["k"], s["k_weight"], *where))
        if case["train"]:
            for x in "qk":
                dy, w, v = _turn(s["d" + x], *where, back=True), s[x + "_weight"], s[x].double()
                if w is not None:
                    root = torch.sqrt(v.square().sum(-1) / D + EPS)
                    out[f"d{x}_weight"] = torch.einsum("thd,thd,th->d", dy, v, 1 / root)
                    d = dy * w.double()
                    dy = d / root[..., None] - v * (torch.einsum("thd,thd->th", d, v) / D / root ** 3)[..., None]
                out["d" + x] = dy
        return out
    if case["op"] == "cache":
        out, k = {}, s["k"]
        if case["fused"]:
            where = (s["positions"], s["freqs"], layout)
            out["q"] = _exact_rows(s["q"], s["q_weight"], *where)
            k = _exact_rows(k, s["k_weight"], *where).to(k.dtype)  # the cache holds what the rows' own type holds
        kept = (s["slots"] >= 0).double()[:, None, None]
        out["k"], out["v"] = _exact_quantized(k, s["k_amax"]) * kept, _exact_quantized(s["v"], s["v_amax"]) * kept
        return out
    Hq, Hk, page = case["Hq"], case["Hk"], case["page"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=out.device)
    mag = torch.tensor(E2M1, dtype=torch.float64, device=out.device)
    first = 0
    for b, (n, L) in enumerate(s["counts"]):
        mine = slice(first, first + n)
        first += n
        if n == 0 or L == 0:
            continue
        j = torch.arange(L, device=out.device)
        at, slot = s["table"][b].long()[j // page], j % page
        for h in range(Hk):
            got = []
            for x in "kv":
                c, e = s[x][at, h, slot].long(), s[x + "_scale"][at, h, slot].long()
                scale = torch.where(e // 8 == 0, (e % 8) / 512.0, (1 + (e % 8) / 8.0) * torch.exp2((e // 8 - 7).double()))
                code = torch.empty(L, D, dtype=torch.int64, device=out.device)
                code[:, 0::2], code[:, 1::2] = c % 16, c // 16
                w = mag[code % 8] * (1 - 2 * (code // 8)).double() * scale[:, torch.arange(D, device=out.device) // 16]
                got.append(w if s[x + "_amax"] is None else w * (s[x + "_amax"][h].double() / 2688))
            limit = (L - n) + torch.arange(n, device=out.device) if case["causal"] else torch.full((n,), L, device=out.device)
            for head in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                score = s["q"][mine, head].double() @ got[0].t() / math.sqrt(D)
                score.masked_fill_(j[None, :] > limit[:, None], -math.inf)
                lse[mine, head] = torch.logsumexp(score, 1)
                out[mine, head] = torch.softmax(score, 1) @ got[1]
                del score
    return dict(out=out, lse=lse)
