"""Angles of one step that are scaled for long contexts, on the CPU."""
import math

import pytest
import torch

import fp4_block_quantization_nvfp4_amd as nv


@pytest.mark.parametrize("dim,base,length,low,high", [
    # dim ln(length / (2 pi r)) / (2 ln base), for r = 32 down and for r = 1 up:
    (64, 10000.0, 4096, 10, 23),   # 10.47, 22.51
    (128, 500000.0, 8192, 18, 35),  # 18.08, 34.99
    (32, 10000.0, 512, 1, 8),      # 1.62, 7.64
])
def test_ramp_of_parts(dim, base, length, low, high):
    f, _ = nv.rotary_frequencies(dim, base=base, device="cpu")
    for factor in (1.0, 4.0, 32.0):
        g, m = nv.rotary_frequencies(dim, base=base, factor=factor, scaling="parts", original_length=length, device="cpu")
        assert math.isclose(m, 0.1 * math.log(factor) + 1, rel_tol=1e-15)
        for i in range(dim // 2):
            r = min(max((i - low) / (high - low), 0.0), 1.0)
            assert math.isclose(g[i], f[i] * (1 - r + r / factor), rel_tol=1e-14), (i, factor)


def test_frequencies_of_no_use_are_refused():
    inf, nan = math.inf, math.nan
    for bad in (dict(base=1.0, scaling="parts", original_length=4096), dict(base=0.5, scaling="parts", original_length=4096),
                dict(scaling="parts", original_length=-1), dict(scaling="parts", original_length=0), dict(scaling="parts", original_length=nan),
                dict(scaling="parts", original_length=inf), dict(base=inf), dict(base=nan), dict(factor=inf), dict(factor=nan), dict(base=-1.0)):
        with pytest.raises(ValueError):
            nv.rotary_frequencies(64, **{"factor": 2.0, **bad}, device="cpu")
    assert torch.equal(nv.rotary_frequencies(8, base=1.0, device="cpu")[0], torch.ones(4, dtype=torch.float64))
