"""No operand load of the matrix products relies on what a range check does with
a scalar offset past its buffer: the products' load code, compiled for the CPU
with the documented check in the builtins' place (tests/c/operand_loads.cpp),
reads inside its buffers and its callers' arrays on every walk, and gives zeros
past K."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp4_block_quantization_nvfp4_amd", "csrc")

# what nvfp4_weight.hpp takes of the device helpers, apart from the loads
HELPERS = """#pragma once
#include "nvfp4_buffer.hpp"
namespace nvfp4 {
typedef short nv_bf8 __attribute__((ext_vector_type(8)));
typedef float nv_f4 __attribute__((ext_vector_type(4)));
constexpr int kMxGroup = 32;
NV_DEV float e8m0_scale(uint32_t) { return 0.0f; }
NV_DEV nv_u2 mx8_to_bf16(uint32_t, float) { return nv_u2{0, 0}; }
NV_DEV nv_bf8 fp4_to_bf16(uint32_t, float) { return nv_bf8{}; }
NV_DEV float e4m3_byte(uint32_t, int) { return 0.0f; }
NV_DEV uint32_t pack_bf16(float, float) { return 0; }
}
"""


def test_operand_loads_stay_inside(tmp_path):
    clang = shutil.which("clang++", path="/opt/rocm/llvm/bin") or shutil.which("clang++")
    if clang is None:
        pytest.skip("clang++ not available")
    for name in ("nvfp4_weight.hpp", "nvfp4_buffer.hpp", "nvfp4_launch.hpp"):
        shutil.copy(os.path.join(CSRC, name), tmp_path)
    (tmp_path / "nvfp4_mx8.hpp").write_text(HELPERS)
    exe = str(tmp_path / "operand_loads")
    subprocess.run([clang, "-O2", "-std=c++17", "-w", "-I", str(tmp_path), "-o", exe,
                    os.path.join(HERE, "c", "operand_loads.cpp")], check=True)
    res = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stdout + res.stderr
    assert ", 0 faults" in res.stdout
