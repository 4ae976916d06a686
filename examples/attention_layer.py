"""A decoder's attention with keys and values stored in NVFP4: prompts, then
single tokens, then the same queries over an encoder's states.

    python examples/attention_layer.py

norm of queries and keys for each head, rotation by position and quantization
into the cache in one pass -> attention over the cache.  Prompts of all sequences
lie one after the other in one call; tokens follow, one a sequence.  The last
step is the gradient of the norms and the rotation, as a training step has it.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import fp4_block_quantization_nvfp4_amd as nv


class Attention:
    """Pages are handed out in order; a sequence's row of the table names its own."""

    def __init__(self, heads, kv_heads, dim, sequences, most, page_size=64):
        self.heads, self.kv, self.page = heads, kv_heads, page_size
        width = -(-most // page_size)
        self.table = torch.arange(sequences * width, dtype=torch.int32, device="cuda").view(sequences, width)
        scale = lambda v: torch.full((kv_heads,), v, device="cuda")
        self.cache = nv.PagedCache.empty(sequences * width, page_size, kv_heads, dim, k_amax=scale(16.0), v_amax=scale(8.0))
        self.freqs, self.multiplier = nv.rotary_frequencies(dim, factor=4.0, scaling="parts", original_length=4096)
        self.q_weight, self.k_weight = torch.ones(dim, device="cuda"), torch.ones(dim, device="cuda")
        self.lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")

    def split(self, qkv):
        return qkv[:, :self.heads], qkv[:, self.heads:self.heads + self.kv], qkv[:, self.heads + self.kv:]

    def step(self, qkv, owner, place, ends):
        """qkv [T, heads + 2 kv_heads, D]; token t is number place[t] of sequence owner[t]."""
        q, k, v = self.split(qkv)
        slots = self.table[owner, place // self.page] * self.page + place % self.page
        q = nv.norm_rope_write(q, k, v, place.int(), self.freqs, self.cache, slots.int(), q_weight=self.q_weight,
                               k_weight=self.k_weight, multiplier=self.multiplier)
        self.lens.index_add_(0, owner, torch.ones_like(owner, dtype=torch.int32))
        return nv.cache_attention(q, self.cache, self.table, self.lens, ends)[0]

    def gradient(self, dq, dk, qkv, positions):
        q, k, _ = self.split(qkv)
        return nv.norm_rope_backward(dq, dk, q, k, positions, self.freqs, q_weight=self.q_weight, k_weight=self.k_weight,
                                     multiplier=self.multiplier)


def main(prompts=(700, 64, 1), heads=32, kv_heads=8, dim=128, tokens=4):
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda n: torch.randn(n, heads + 2 * kv_heads, dim, device="cuda", generator=g).bfloat16()
    B = len(prompts)
    layer = Attention(heads, kv_heads, dim, B, max(prompts) + tokens)
    counts = torch.tensor(prompts, device="cuda")
    owner = torch.repeat_interleave(torch.arange(B, device="cuda"), counts)
    place = torch.cat([torch.arange(n, device="cuda") for n in prompts])
    qkv = rand(len(owner))
    out = layer.step(qkv, owner, place, torch.cumsum(counts, 0).int())
    print(f"prompts of {tuple(prompts)}: {tuple(out.shape)}, norm {out.float().norm().item():.4g}")
    everyone = torch.arange(B, device="cuda")
    for i in range(tokens):
        last = layer.step(rand(B), everyone, layer.lens.long(), None)
    print(f"{tokens} tokens each: {tuple(last.shape)}, norm {last.float().norm().item():.4g}; keys now {layer.lens.tolist()}")
    # all queries see all keys of their sequence: what a decoder has over an encoder's states
    cross = nv.cache_attention(last, layer.cache, layer.table, layer.lens, causal=False)[0]
    grads = layer.gradient(qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv, place.int())
    for name, t in zip(("queries", "keys", "queries' weight", "keys' weight"), grads):
        print(f"gradient of the {name}: {tuple(t.shape)} {str(t.dtype)[6:]}, norm {t.float().norm().item():.4g}")
    return out, last, cross, grads, layer


if __name__ == "__main__":
    main()
