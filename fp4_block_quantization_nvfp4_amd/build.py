"""Build libnvfp4.so (the HIP kernels and the C ABI) and _layer.so (the torch
binding of the layer operators) in-tree for gfx950.

    python -m fp4_block_quantization_nvfp4_amd.build

Flags that matter for bit-exactness: -ffp-contract=off (no implicit fused
multiply-add), no fast-math (IEEE division, NaN-aware min/max, denormals
kept).  Packed-fp32 VALU instructions are disabled.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libnvfp4.so")
BIND = os.path.join(HERE, "_layer.so")
ARCH = os.environ.get("NVFP4_OFFLOAD_ARCH", "gfx950")

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-ffp-contract=off",
    "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-command-line-argument",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip"))) + sorted(glob.glob(os.path.join(CSRC, "*.cpp")))


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 feature name; that warning is expected
    err = "\n".join(l for l in res.stderr.splitlines() if "packed-fp32-ops" not in l and l.strip())
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({res.returncode}): {' '.join(cmd)}\n{res.stderr}")
    if err and verbose:
        print(err, file=sys.stderr)


def bind_commands(obj: str, out: str):
    """Compile and link commands of the binding: host code against torch's
    headers and libnvfp4.so beside it."""
    import torch
    from torch.utils import cpp_extension

    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], os.path.join(os.path.dirname(HERE), "include")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cxx = os.environ.get("CXX", "g++")
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", abi, *[a for p in inc for a in ("-I", p)],
             "-c", "-o", obj, os.path.join(HERE, "bind", "layer.cpp")],
            [cxx, "-shared", "-o", out, obj, "-L", HERE, "-l:libnvfp4.so", "-Wl,-rpath,$ORIGIN", "-L", libs, "-lc10",
             "-ltorch_cpu", "-ltorch_hip", "-ltorch_python"])


def _compile_bind(obj: str, out: str, verbose: bool):
    """Compiles the binding; the command that links it."""
    compile_bind, link_bind = bind_commands(obj, out)
    _run(compile_bind, verbose)
    return link_bind


def build(verbose: bool = False, jobs: int = 8) -> str:
    """Compile every source to an object in parallel, then link the shared
    library and the binding; each result replaces its file atomically.  The
    library is made whether or not the binding can be: what fails there is raised
    afterwards, and a binding of an older library is taken away."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    inc = ["-I", os.path.join(os.path.dirname(HERE), "include")]
    compile_flags = [f for f in FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory(prefix="nvfp4_build_") as tmpd:
        objs, cmds = [], []
        for src in sources():
            obj = os.path.join(tmpd, os.path.basename(src) + ".o")
            objs.append(obj)
            cmds.append([hipcc, *compile_flags, *inc, "-c", "-o", obj, src])
        bind_tmp = BIND + ".tmp"
        with ThreadPoolExecutor(max_workers=max(1, min(jobs, len(cmds) + 1))) as ex:
            bind = ex.submit(_compile_bind, os.path.join(tmpd, "layer.o"), bind_tmp, verbose)
            for f in [ex.submit(_run, c, verbose) for c in cmds]:
                f.result()
        tmp = LIB + ".tmp"
        _run([hipcc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs], verbose)
        os.replace(tmp, LIB)
        try:
            _run(bind.result(), verbose)
            os.replace(bind_tmp, BIND)
        except BaseException:
            if os.path.exists(BIND):
                os.remove(BIND)
            raise
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
