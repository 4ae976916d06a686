"""A layer of experts with weights stored in NVFP4: one training step, then
single tokens.

    python examples/expert_layer.py

norm with 8-bit output -> products grouped by expert -> gated activation that
keeps 8-bit checkpoints -> products back, and the whole backward pass: the
gradients of the input, of the norm's weight and of both expert weights.  The
weights are quantized on 16x16 tiles, so the backward products read the
columnwise codes of the same quantization.  Serving reads the same weights for
a few tokens, grouped by expert and through a single projection.

Rows are taken as sorted by expert; the choice of experts is not part of it.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import fp4_block_quantization_nvfp4_amd as nv


class Experts:
    """E weights [N, K] on 16x16 tiles: rowwise codes for x W^T, columnwise
    codes for the gradient of x, one set of tile scales for both."""

    def __init__(self, weights):
        parts = []
        for w in weights:
            amax = nv.amax(w)
            parts.append(nv.quantize_2d(w, amax) + (amax,))
        self.rows, self.columns, self.tiles, amax = (torch.stack(t) for t in zip(*parts))
        self.amax = amax.view(-1)

    def forward(self, x, x_scale, ends):
        return nv.grouped_matmul(x, ends, self.rows, self.tiles, x_scale=x_scale, tile16=True, global_amax=self.amax)

    def input_gradient(self, dy, ends):
        return nv.grouped_matmul(dy, ends, self.columns, self.tiles, tile16=True, transposed_tiles=True,
                                 global_amax=self.amax)


class ExpertLayer:
    def __init__(self, experts, hidden, inner, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        make = lambda n, k: [(torch.randn(n, k, device="cuda", generator=g) * k ** -0.5).bfloat16() for _ in range(experts)]
        self.norm = torch.ones(hidden, device="cuda")
        self.up, self.down = Experts(make(2 * inner, hidden)), Experts(make(hidden, inner))

    def forward(self, x, residual, ends, keep=True):
        codes, scales, hidden, rstd = nv.add_rms_norm(x, self.norm, residual)
        gate_up = self.up.forward(codes, scales, ends)
        y, y_scale, kept, kept_scales = nv.swiglu_checkpoint(gate_up, keep=keep)
        out = self.down.forward(y, y_scale, ends)
        return out, hidden, (codes, scales, hidden, rstd, y, y_scale, kept, kept_scales, ends)

    def backward(self, dout, dhidden, saved):
        """Gradients of x (and residual alike), the norm's weight and both expert weights."""
        codes, scales, hidden, rstd, y, y_scale, kept, kept_scales, ends = saved
        d_down = nv.grouped_wgrad(dout, y, ends, x_scale=y_scale)
        dgate_up = nv.swiglu_backward(self.down.input_gradient(dout, ends), kept, kept_scales)
        d_up = nv.grouped_wgrad(dgate_up, codes, ends, x_scale=scales)
        dx, dnorm = nv.add_rms_norm_backward(self.up.input_gradient(dgate_up, ends), hidden, self.norm, rstd, dhidden)
        return dx, dnorm, d_up, d_down


def main(tokens=4096, experts=8, hidden=2048, inner=1024):
    layer = ExpertLayer(experts, hidden, inner)
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=g).bfloat16()
    counts = torch.full((experts,), tokens // experts)
    counts[0], counts[1] = 2 * counts[0], 0  # uneven on purpose: one expert has no row
    ends = torch.cumsum(counts, 0).int().cuda()
    x, residual, target = rand(tokens, hidden), rand(tokens, hidden), rand(tokens, hidden)
    out, h, saved = layer.forward(x, residual, ends)
    dout = ((out.float() + h.float() - target.float()) / tokens).bfloat16()  # of half the mean squared distance
    grads = layer.backward(dout, dout, saved)
    for name, t in zip(("input", "norm weight", "up weights", "down weights"), grads):
        print(f"gradient of the {name}: {tuple(t.shape)} {str(t.dtype)[6:]}, norm {t.float().norm().item():.4g}")

    # serving: four tokens, two of them with expert 0, one each with 3 and 5
    few = torch.tensor([2, 2, 2, 3, 3, 4, 4, 4], dtype=torch.int32, device="cuda")[:experts]
    out, h, _ = layer.forward(x[:4].contiguous(), residual[:4].contiguous(), few, keep=False)
    one = nv.matvec(h[:1].contiguous(), layer.up.rows[0], layer.up.tiles[0], tile16=True, global_amax=layer.up.amax[:1])
    print(f"tokens: {tuple(out.shape)}, norm {out.float().norm().item():.4g}; one projection {tuple(one.shape)}")
    return grads, out, one


if __name__ == "__main__":
    main()
