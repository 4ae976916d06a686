"""The operators of a layer whose weights are stored in NVFP4, as cases to be
measured: a root-mean-square norm that writes 8-bit activations, a gated
activation that keeps 8-bit checkpoints for its backward pass, matrix-vector
products for single tokens, and products grouped by expert with their
gradients.

`own` false: plain torch operations in 32 bits.  `own` true: this repository's
kernels.  Both take what `prepare` makes.

8-bit activations ("mx8"): e4m3 codes with one power-of-two scale (e8m0) for
each 32 consecutive elements of a row, the last group of a row possibly
shorter.  The scale is the smallest 2**s, s >= -117, with
max |finite value| <= 448 * 2**s; what is not finite is coded as NaN.

4-bit weights: e2m1 codes, two per byte, the even element in the low nibble;
one e4m3 scale for 16 elements of a row or for a 16x16 tile; a second-level
scale amax / (6 * 448) for a tensor (or expert) or for each row.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6
BOUND = 448.0


def listed():
    return [
        # one new token enters a layer while serving: latency counts
        dict(name="norm, one token", op="norm", T=1, H=7168, dtype="bf16", train=False),
        # a training step's activations, with the backward pass
        dict(name="norm, training", op="norm", T=8192, H=7168, dtype="bf16", train=True),
        # a residual stream in 32 bits, an odd width (the last group is half a group)
        dict(name="norm, odd, 32 bits", op="norm", T=1021, H=2064, dtype="f32", train=True),
        # a batch of tokens being decoded, nothing kept for a backward pass
        dict(name="swiglu, decoding", op="swiglu", T=16, F=2048, dtype="bf16", train=False),
        # a training step: the checkpoint is written, then the backward pass reads it
        dict(name="swiglu, training", op="swiglu", T=8192, F=8192, dtype="bf16", train=True),
        # one token times a square projection
        dict(name="matvec, one token", op="matvec", T=1, N=4096, K=4096, act="bf16", blocks="1x16", amax="tensor", out="bf16"),
        # a full decoding batch times the widest weight, 8-bit activations, 16x16 scale tiles
        dict(name="matvec, 16 tokens", op="matvec", T=16, N=18432, K=7168, act="mx8", blocks="16x16", amax="tensor", out="bf16"),
        # ragged sizes, a scale for each row, logits kept in 32 bits
        dict(name="matvec, odd", op="matvec", T=5, N=1001, K=2064, act="bf16", blocks="1x16", amax="row", out="f32"),
        # decoding with many experts: a row or two for each of them
        dict(name="experts, decoding", op="experts", T=64, E=32, N=4096, K=2048, act="bf16", blocks="1x16", amax="tensor", out="bf16", grad="", train=False),
        # a long prompt through eight experts, 8-bit activations
        dict(name="experts, prompt", op="experts", T=8192, E=8, N=4096, K=7168, act="mx8", blocks="1x16", amax="tensor", out="bf16", grad="", train=False),
        # a training step: forward, gradient of the input, gradient of the weights from the 8-bit checkpoint
        dict(name="experts, training", op="experts", T=16384, E=16, N=4096, K=2048, act="mx8", blocks="16x16", amax="tensor", out="bf16", grad="f32", train=True),
        # ragged sizes, some experts with no row at all
        dict(name="experts, odd, training", op="experts", T=1777, E=5, N=1040, K=528, act="bf16", blocks="1x16", amax="tensor", out="bf16", grad="bf16", train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "swiglu", "matvec", "experts", "experts"))
    if op == "norm":
        H = 16 * _log(rng, 8, 512)
        T = _log(rng, 1, min(16384, (8192 * 7168) // H))
        return dict(op=op, T=T, H=H, dtype=rng.choice(("bf16", "f32")) if T * H < 1 << 25 else "bf16", train=rng.random() < 0.5)
    if op == "swiglu":
        F = 16 * _log(rng, 8, 512)
        T = _log(rng, 1, min(16384, (8192 * 8192) // F))
        return dict(op=op, T=T, F=F, dtype=rng.choice(("bf16", "f32")) if T * F < 1 << 25 else "bf16", train=rng.random() < 0.5)
    act, blocks = rng.choice(("bf16", "mx8")), rng.choice(("1x16", "16x16"))
    if op == "matvec":
        T = rng.randint(1, 16)
        K = 16 * _log(rng, 16, 1024)
        N = _log(rng, 100, 18432)
        N = N - N % 16 if blocks == "16x16" else N
        amax = "tensor" if blocks == "16x16" else rng.choice(("none", "tensor", "row"))
        return dict(op=op, T=T, N=N, K=K, act=act, blocks=blocks, amax=amax, out=rng.choice(("bf16", "f32")))
    E = _log(rng, 1, 32)
    N, K = 16 * _log(rng, 16, 256), 16 * _log(rng, 16, 256)
    while E * N * K > 1 << 28:
        E = (E + 1) // 2
    T = _log(rng, 1, max(2, min(16384, (16384 * 4096 * 2048) // (N * K))))
    train = rng.random() < 0.6
    return dict(op=op, T=T, E=E, N=N, K=K, act=act, blocks=blocks, amax="tensor", out=rng.choice(("bf16", "f32")),
                grad=rng.choice(("bf16", "f32")) if train else "", train=train)


DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ inputs


def _quantize_weight(w, tile, rows):
    """4-bit codes of w [E, N, K]: (packed, scales, amax [E] or [E * N])."""
    E, N, K = w.shape
    amax = w.abs().amax(-1) if rows else w.abs().amax((1, 2)).unsqueeze(1)  # [E, N or 1]
    dec = (amax / (6 * BOUND)).unsqueeze(-1)
    b = w.abs().view(E, N, K // 16, 16).amax(-1)
    if tile:
        b = b.view(E, N // 16, 16, K // 16).amax(2)
    s = (b / 6 / dec).clamp(max=BOUND).to(F8)
    wide = (s.float().repeat_interleave(16, 1) if tile else s.float()) * dec
    v = (w.view(E, N, K // 16, 16) / wide.unsqueeze(-1).clamp(min=1e-30)).view(E, N, K)
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(v.abs(), borders).to(torch.uint8) | ((v < 0).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8), amax.reshape(-1).contiguous()


def _weight(g, E, N, K, case):
    w = torch.randn(E, N, K, device="cuda", generator=g) * 0.02
    tile, rows = case["blocks"] == "16x16", case["amax"] == "row"
    packed, scale, amax = _quantize_weight(w, tile, rows)
    got = dict(packed=packed.contiguous(), scale=scale.contiguous(), amax=None if case["amax"] == "none" else amax)
    if case.get("train"):  # the operand of the input's gradient: the same codes transposed (tiles), or a quantization of its own
        if tile:
            code = torch.stack((packed & 15, packed >> 4), -1).view(E, N, K).transpose(1, 2).contiguous()
            got["packed_t"], got["scale_t"] = code[..., 0::2] | (code[..., 1::2] << 4), got["scale"]
        else:
            got["packed_t"], got["scale_t"], _ = _quantize_weight(w.transpose(1, 2).contiguous(), False, False)
    return got


def _activations(g, T, K, case):
    x = torch.randn(T, K, device="cuda", generator=g) * (0.5 + 1.5 * torch.rand(T, 1, device="cuda", generator=g))
    return _mx8(x) if case["act"] == "mx8" else (x.bfloat16(), None)


def _ends(seed, T, E):
    """Cumulative row counts of E experts: uneven, and with four or more experts one has no row."""
    c = torch.Generator().manual_seed(seed * 7 + 3)
    share = torch.rand(E, generator=c) ** 2 + 0.05
    if E >= 4:
        share[int(torch.randint(E, (1,), generator=c))] = 0
    cut = (torch.cumsum(share, 0) / share.sum() * T).round().to(torch.int32)
    cut[-1] = T
    return cut


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 13 + 1)
    s = dict(case)

    def rand(*shape, dtype="bf16", by=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * by).to(DTYPE[dtype])

    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        s["x"] = rand(T, H, dtype=case["dtype"])
        s["residual"] = rand(T, H, dtype=case["dtype"], by=3.0)
        s["weight"] = 1 + 0.2 * rand(H, dtype="f32")
        if case["train"]:
            s["dy"], s["dhidden"] = rand(T, H, dtype=case["dtype"]), rand(T, H, dtype=case["dtype"])
    elif case["op"] == "swiglu":
        s["gate_up"] = rand(case["T"], 2 * case["F"], dtype=case["dtype"], by=2.0)
        if case["train"]:
            s["dout"] = rand(case["T"], case["F"], dtype=case["dtype"])
    else:
        E = case.get("E", 1)
        s.update(_weight(g, E, case["N"], case["K"], case))
        s["x"], s["x_scale"] = _activations(g, case["T"], case["K"], case)
        if case["op"] == "matvec":
            s["packed"], s["scale"] = s["packed"][0], s["scale"][0]
        else:
            ends = _ends(seed, case["T"], E)
            s["ends"], s["cuts"] = ends.cuda(), [0] + ends.tolist()
            if case["train"]:
                s["dy"] = rand(case["T"], case["N"], by=0.5)
    return s


# -------------------------------------------------------------- plain forms


def _mx8(v):
    """32-bit values -> (e4m3 codes, e8m0 scales)."""
    T, K = v.shape
    p = torch.nn.functional.pad(v, (0, -K % 32)).view(T, -1, 32)
    a = torch.where(torch.isfinite(p), p.abs(), 0.0).amax(-1)
    m, e = torch.frexp(a)
    s = torch.where(a == 0, -117, torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-117))
    q = torch.ldexp(p, -s.unsqueeze(-1))
    q = torch.where(torch.isfinite(q), q, float("nan")).to(F8).view(T, -1)[:, :K].contiguous()
    return q, (s + 127).to(torch.uint8).view(E8)


def _values(codes, scales):
    """32-bit values of mx8 codes."""
    K = codes.shape[1]
    return codes.float() * torch.exp2(scales.view(torch.uint8).float() - 127).repeat_interleave(32, 1)[:, :K]


def _dense(packed, scale, amax, tile):
    """32-bit values of 4-bit weights [..., N, K]; tile: False, True, or "t" for tiles of the transposed weight."""
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    v = grid[torch.stack((packed & 15, packed >> 4), -1).long()].flatten(-2)
    s = scale.view(F8).float()
    s = s.transpose(-1, -2) if tile == "t" else s
    s = s.repeat_interleave(16, -2) if tile else s
    v = v * s.repeat_interleave(16, -1)
    if amax is None:
        return v
    return v * (amax / (6 * BOUND)).view(v.shape[:-2] + (-1, 1))


def _plain_norm(s):
    dt = DTYPE[s["dtype"]]
    h = s["x"].float() + s["residual"].float()
    rstd = torch.rsqrt((h * h).mean(-1) + EPS)
    codes, scales = _mx8(h * rstd.unsqueeze(1) * s["weight"])
    out = dict(codes=codes, scales=scales, hidden=h.to(dt), rstd=rstd)
    if s["train"]:
        n = out["hidden"].float() * rstd.unsqueeze(1)
        dy = s["dy"].float()
        d = dy * s["weight"]
        dx = rstd.unsqueeze(1) * (d - n * (d * n).mean(-1, keepdim=True)) + s["dhidden"].float()
        out.update(dx=dx.to(dt), dweight=(dy * n).sum(0))
    return out


def _plain_swiglu(s):
    F = s["F"]
    gate, up = s["gate_up"].float().split(F, 1)
    codes, scales = _mx8(gate * torch.sigmoid(gate) * up)
    out = dict(codes=codes, scales=scales)
    if s["train"]:
        gc, gs = _mx8(gate)
        uc, us = _mx8(up)
        out.update(kept=torch.cat((gc, uc), 1), kept_scales=torch.cat((gs, us), 1))
        gate, up, d = _values(gc, gs), _values(uc, us), s["dout"].float()
        sig = torch.sigmoid(gate)
        dgate = d * up * sig * (1 + gate * (1 - sig))
        out["dgate_up"] = torch.cat((dgate, d * gate * sig), 1).to(DTYPE[s["dtype"]])
    return out


def _plain_matvec(s):
    x = s["x"].float() if s["x_scale"] is None else _values(s["x"], s["x_scale"])
    w = _dense(s["packed"], s["scale"], s["amax"], s["blocks"] == "16x16")
    return (x @ w.t()).to(DTYPE[s["out"]])


def _plain_experts(s):
    x = s["x"].float() if s["x_scale"] is None else _values(s["x"], s["x_scale"])
    tile, cuts, E = s["blocks"] == "16x16", s["cuts"], s["E"]
    w = _dense(s["packed"], s["scale"], s["amax"], tile)
    out = dict(y=torch.cat([x[cuts[e]:cuts[e + 1]] @ w[e].t() for e in range(E)]).to(DTYPE[s["out"]]))
    if s["train"]:
        dy = s["dy"].float()
        w = _dense(s["packed_t"], s["scale_t"], s["amax"], "t" if tile else False)
        out["dx"] = torch.cat([dy[cuts[e]:cuts[e + 1]] @ w[e].t() for e in range(E)]).bfloat16()
        out["dw"] = torch.stack([dy[cuts[e]:cuts[e + 1]].t() @ x[cuts[e]:cuts[e + 1]] for e in range(E)]).to(DTYPE[s["grad"]])
    return out


# ------------------------------------------------------------ the framework


def _own(s):
    import fp4_block_quantization_nvfp4_amd as nv

    if s["op"] == "norm":
        codes, scales, hidden, rstd = nv.add_rms_norm(s["x"], s["weight"], s["residual"], eps=EPS)
        out = dict(codes=codes, scales=scales, hidden=hidden, rstd=rstd)
        if s["train"]:
            out["dx"], out["dweight"] = nv.add_rms_norm_backward(s["dy"], hidden, s["weight"], rstd, s["dhidden"])
        return out
    if s["op"] == "swiglu":
        codes, scales, kept, kept_scales = nv.swiglu_checkpoint(s["gate_up"], keep=s["train"])
        out = dict(codes=codes, scales=scales)
        if s["train"]:
            out.update(kept=kept, kept_scales=kept_scales)
            out["dgate_up"] = nv.swiglu_backward(s["dout"], kept, kept_scales)
        return out
    tile, more = s["blocks"] == "16x16", dict(global_amax=s["amax"], bound=BOUND)
    if s["op"] == "matvec":
        return nv.matvec(s["x"], s["packed"], s["scale"], x_scale=s["x_scale"], tile16=tile, row_scaled=s["amax"] is not None and s["amax"].numel() > 1,
                         out_dtype=DTYPE[s["out"]], **more)
    out = dict(y=nv.grouped_matmul(s["x"], s["ends"], s["packed"], s["scale"], x_scale=s["x_scale"], tile16=tile, out_dtype=DTYPE[s["out"]], **more))
    if s["train"]:
        out["dx"] = nv.grouped_matmul(s["dy"], s["ends"], s["packed_t"], s["scale_t"], tile16=tile, transposed_tiles=tile, **more)
        out["dw"] = nv.grouped_wgrad(s["dy"], s["x"], s["ends"], x_scale=s["x_scale"], out_dtype=DTYPE[s["grad"]])
    return out


def run(state):
    if own:
        return _own(state)
    return {"norm": _plain_norm, "swiglu": _plain_swiglu, "matvec": _plain_matvec, "experts": _plain_experts}[state["op"]](state)


def work(case):
    """Inputs read once and outputs written once, whatever stays on the way between a case's calls; a multiply-add is two operations."""
    size = {"bf16": 2, "f32": 4}

    def mx8(T, K):
        return T * K + T * ((K + 31) // 32)

    if case["op"] == "norm":
        T, H, b = case["T"], case["H"], size[case["dtype"]]
        n = 3 * T * H * b + 4 * H + mx8(T, H) + 4 * T
        return dict(bytes=n + (3 * T * H * b + 4 * H if case["train"] else 0), flops=T * H * (16 if case["train"] else 6))
    if case["op"] == "swiglu":
        T, F, b = case["T"], case["F"], size[case["dtype"]]
        n = 2 * T * F * b + mx8(T, F)
        return dict(bytes=n + (2 * mx8(T, F) + 3 * T * F * b if case["train"] else 0), flops=T * F * (24 if case["train"] else 8))
    T, E, N, K = case["T"], case.get("E", 1), case["N"], case["K"]
    E = min(E, T)  # an expert without rows is not read
    x = mx8(T, K) if case["act"] == "mx8" else 2 * T * K
    w = E * (N * K // 2 + N * K // (256 if case["blocks"] == "16x16" else 16))
    n, f = x + w + T * N * size[case["out"]], 2 * T * N * K
    if case.get("train"):
        n += 2 * T * N + (0 if case["blocks"] == "16x16" else w) + 2 * T * K + case["E"] * N * K * size[case["grad"]]
        f *= 3
    return dict(bytes=n, flops=f)


# -------------------------------------------------------------- in 64 bits


def _round_e4m3(q):
    """Nearest value of the e4m3 grid, ties to the even one, for |q| <= 448."""
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(q / step) * step


def _exact_mx8(v):
    """Codes' values and scales' values of 64-bit v (finite), and the values that both stand for."""
    T, K = v.shape
    groups = torch.arange(K, device=v.device) // 32
    a = torch.zeros(T, (K + 31) // 32, dtype=v.dtype, device=v.device).scatter_reduce(1, groups.expand(T, K), v.abs(), "amax")
    s = torch.ceil(torch.log2((a / 448).clamp(min=2.0 ** -117)))
    s = torch.where(a > 448 * torch.exp2(s), s + 1, s)
    s = torch.where((s > -117) & (a <= 448 * torch.exp2(s - 1)), s - 1, s)
    wide = torch.exp2(s)[:, groups]
    codes = _round_e4m3(v / wide)
    return codes.to(F8), torch.exp2(s).to(E8), codes * wide


def _exact_weight(packed, scale, amax, tile, transposed=False):
    """[E, N, K] in 64 bits, from the bits of the codes and scales."""
    E, N, K = packed.shape[0], packed.shape[1], 2 * packed.shape[2]
    c = torch.empty(E, N, K, dtype=torch.int64, device=packed.device)
    c[..., 0::2], c[..., 1::2] = packed.long() % 16, packed.long() // 16
    exp, man = (c // 2) % 4, (c % 2).double()
    v = torch.where(exp == 0, man / 2, (1 + man / 2) * torch.exp2(exp.double() - 1)) * (1 - 2 * (c // 8)).double()
    b = scale.long()
    s = torch.where(b // 8 == 0, (b % 8).double() / 512, (1 + (b % 8).double() / 8) * torch.exp2((b // 8).double() - 7))
    n, k = torch.arange(N, device=c.device), torch.arange(K, device=c.device) // 16
    if tile and transposed:
        s = s[:, k][:, :, n // 16].transpose(1, 2)
    elif tile:
        s = s[:, n // 16][:, :, k]
    else:
        s = s[:, :, k]
    v = v * s
    if amax is not None:
        v = v * (amax.double() / (6 * BOUND)).reshape(E, -1, 1)
    return v


def _exact_x(s):
    if s["x_scale"] is None:
        return s["x"].double()
    g = torch.arange(s["K"], device=s["x"].device) // 32
    return s["x"].double() * torch.exp2(s["x_scale"].view(torch.uint8).double() - 127)[:, g]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        dt, w = DTYPE[case["dtype"]], s["weight"].double()
        h = s["x"].double() + s["residual"].double()
        rstd = 1 / torch.sqrt(h.square().sum(1) / case["H"] + EPS)
        codes, scales, _ = _exact_mx8(torch.einsum("th,t,h->th", h, rstd, w))
        out = dict(codes=codes, scales=scales, hidden=h.to(dt), rstd=rstd)
        if case["train"]:
            h, dy = h.to(dt).double(), s["dy"].double()
            c = torch.einsum("th,th,h->t", dy, h, w) * rstd ** 3 / case["H"]
            out["dx"] = torch.einsum("th,t,h->th", dy, rstd, w) - h * c[:, None] + s["dhidden"].double()
            out["dweight"] = torch.einsum("th,th,t->h", dy, h, rstd)
        return out
    if case["op"] == "swiglu":
        F = case["F"]
        gate, up = s["gate_up"].double()[:, :F], s["gate_up"].double()[:, F:]
        codes, scales, _ = _exact_mx8(gate / (1 + torch.exp(-gate)) * up)
        out = dict(codes=codes, scales=scales)
        if case["train"]:
            gc, gs, gate = _exact_mx8(gate)
            uc, us, up = _exact_mx8(up)
            out["kept"], out["kept_scales"] = torch.cat((gc, uc), 1), torch.cat((gs, us), 1)
            d, t = s["dout"].double(), torch.tanh(gate / 2)  # the logistic function is (1 + t) / 2, its derivative (1 - t^2) / 4
            out["dgate_up"] = torch.cat((d * up * ((1 + t) / 2 + gate * (1 - t * t) / 4), d * gate * (1 + t) / 2), 1)
        return out
    x, tile = _exact_x(s), case["blocks"] == "16x16"
    if case["op"] == "matvec":
        w = _exact_weight(s["packed"][None], s["scale"][None], s["amax"], tile)[0]
        return torch.stack([w @ row for row in x])
    w = _exact_weight(s["packed"], s["scale"], s["amax"], tile)
    which = torch.bucketize(torch.arange(case["T"], device=x.device), s["ends"], right=True)  # each row's expert
    out = dict(y=torch.zeros(case["T"], case["N"], dtype=torch.float64, device=x.device))
    for e in range(case["E"]):
        out["y"][which == e] = x[which == e] @ w[e].t()
    if case["train"]:
        del w
        w, dy = _exact_weight(s["packed_t"], s["scale_t"], s["amax"], tile, True), s["dy"].double()
        out["dx"] = torch.zeros_like(x)
        out["dw"] = torch.zeros(case["E"], case["N"], case["K"], dtype=torch.float64, device=x.device)
        for e in range(case["E"]):
            out["dx"][which == e] = dy[which == e] @ w[e].t()
            out["dw"][e] = dy[which == e].t() @ x[which == e]
    return out
