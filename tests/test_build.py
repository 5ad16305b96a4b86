"""The build's order and failures, on the CPU, with commands that only write their outputs."""
import os
import sys

import pytest

from mx_block_scaled_x128_amd import build


@pytest.fixture
def stub(monkeypatch, tmp_path):
    """Outputs go to tmp_path; `fail` names a part of an output's name whose command fails."""
    state = {"fail": None}

    def run(cmd):
        out = cmd[cmd.index("-o") + 1]
        if state["fail"] and state["fail"] in os.path.basename(out):
            with open(out, "w") as f:
                f.write("half of it")
            raise RuntimeError("hipcc failed: " + out)
        with open(out, "w") as f:
            f.write("built")
        return ""
    monkeypatch.setattr(build, "hipcc", lambda: "hipcc")
    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmxfp8.so"))
    monkeypatch.setattr(build, "TENSORS", str(tmp_path / "_mx_tensors.so"))
    state["dir"] = tmp_path
    return state


def files(stub):
    return sorted(p.name for p in stub["dir"].iterdir())


def test_both_are_built(stub):
    assert build.build() == build.LIB
    assert files(stub) == ["_mx_tensors.so", "libmxfp8.so"]


def test_the_library_is_built_without_torch(stub, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    with pytest.raises(ImportError):
        build.build()
    assert files(stub) == ["libmxfp8.so"]


def test_the_library_is_built_if_the_extension_fails(stub):
    stub["fail"] = "_mx_tensors"
    with pytest.raises(RuntimeError, match="_mx_tensors"):
        build.build()
    assert files(stub) == ["libmxfp8.so"]


@pytest.mark.parametrize("fail", ["libmxfp8", "mx_act.o"])
def test_a_failed_library_leaves_nothing_half_written(stub, fail):
    stub["fail"] = fail
    with pytest.raises(RuntimeError, match="hipcc failed"):
        build.build()
    assert files(stub) == ["_mx_tensors.so"]
