"""Rules of the launches of attention on an NVFP4 cache that the kernels share with the host,
compiled for the CPU from the same header, and the launches of both types of rows."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from fp4_block_quantization_nvfp4_amd import _lib as L

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp4_block_quantization_nvfp4_amd", "csrc")


def test_pieces_cover_all_tiles(tmp_path):
    """Up to the largest total of a call, 2^31 - 1, where 32 bits do not hold total + pieces."""
    cxx = shutil.which("g++") or shutil.which("clang++", path="/opt/rocm/llvm/bin")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "piece_cuts")
    subprocess.run([cxx, "-O1", "-std=c++17", "-w", "-I", CSRC, "-o", exe, os.path.join(HERE, "c", "piece_cuts.cpp")], check=True)
    done = subprocess.run([exe], capture_output=True, text=True)
    assert done.returncode == 0, done.stdout
    assert int(done.stdout.split()[0]) > 10000


def plan(entry, T, Hq, Hk, D):
    out = (ctypes.c_int64 * 16)()
    return L.lib().nvfp4_selftest_attention_plan(entry, T, Hq, Hk, D, 1, 16, out), [list(out[4 * i:4 * i + 4]) for i in range(4)]


def test_launches_of_both_types():
    """32-bit rows have grids of their own, inside the dispatch limits, and the gradient's partial sums fit the workspace,
    which does not know the type."""
    rng = random.Random(4)
    own = 0
    for _ in range(3000):
        entry, D = rng.randrange(4), 16 * rng.randint(1, 32)
        T, Hq, Hk = int(2 ** rng.uniform(0, 31)), int(2 ** rng.uniform(0, 12)), int(2 ** rng.uniform(0, 8))
        (a, bf16), (b, f32) = plan(entry, T, Hq, Hk, D), plan(16 + entry, T, Hq, Hk, D)
        assert a == b and a in (L.OK, L.E_RANGE)
        if a != L.OK:
            continue
        own += bf16 != f32
        for launches in (bf16, f32):
            assert launches[0][0] == bf16[0][0]
            for _, x, y, lanes in launches:
                assert x == 0 or (1 <= x and x * lanes < 1 << 32 and y == 1 and lanes == 256)
            assert launches[0][1] * 4 <= max(T * 4096, 4)
            if entry == 1:
                assert launches[0][1] * 2 * D * 4 <= L.lib().nvfp4_norm_rope_backward_workspace_bytes(T, D)
    assert own > 300


def test_entries_of_the_plan():
    for entry in (7, 15, 20, 16 + 5, -1):
        assert plan(entry, 4, 4, 2, 64)[0] == L.E_ARG
