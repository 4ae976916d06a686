"""The build's order without a compiler: the C library needs hipcc alone, so a
binding that cannot be built (no torch headers, no g++) does not keep the
library from being made, and no binding of an older library stays beside it."""
import os

import pytest

from fp4_block_quantization_nvfp4_amd import build as B


@pytest.fixture
def made(tmp_path, monkeypatch):
    """Runs of the build with commands that write their output file, or fail."""
    state = {"fail": "", "commands": []}

    def run(cmd, verbose):
        out = cmd[cmd.index("-o") + 1]
        state["commands"].append(os.path.basename(out))
        if state["fail"] and any(state["fail"] in c for c in cmd):
            raise RuntimeError(f"{cmd[0]} failed")
        with open(out, "w") as f:
            f.write("new")

    monkeypatch.setattr(B, "_run", run)
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libnvfp4.so"))
    monkeypatch.setattr(B, "BIND", str(tmp_path / "_layer.so"))
    for p in (B.LIB, B.BIND):
        with open(p, "w") as f:
            f.write("old")
    return state


def content(p):
    return open(p).read() if os.path.exists(p) else None


def test_both_are_replaced(made):
    assert B.build() == B.LIB
    assert content(B.LIB) == "new" and content(B.BIND) == "new"
    assert made["commands"][-1] == "_layer.so.tmp" and made["commands"].count("libnvfp4.so.tmp") == 1


@pytest.mark.parametrize("what", [os.path.join("bind", "layer.cpp"), "-ltorch_python"], ids=["compile", "link"])
def test_a_binding_that_fails_leaves_the_library(made, what):
    made["fail"] = what
    with pytest.raises(RuntimeError):
        B.build()
    assert content(B.LIB) == "new" and content(B.BIND) is None


def test_a_torch_without_headers_leaves_the_library(made, monkeypatch):
    def commands(obj, out):
        raise ImportError("no torch")

    monkeypatch.setattr(B, "bind_commands", commands)
    with pytest.raises(ImportError):
        B.build()
    assert content(B.LIB) == "new" and content(B.BIND) is None


def test_a_kernel_that_fails_leaves_both_as_they_were(made):
    made["fail"] = "k_norm.hip"
    with pytest.raises(RuntimeError):
        B.build()
    assert content(B.LIB) == "old" and content(B.BIND) == "old"
