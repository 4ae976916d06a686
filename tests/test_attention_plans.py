"""Rules of the launches of attention on an NVFP4 cache that the kernels share with the host,
compiled for the CPU from the same header."""
import os
import shutil
import subprocess

import pytest

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
