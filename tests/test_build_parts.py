"""What build() makes of the library and of the marshalling module, each by itself (compilers are stood in for)."""
import os
import subprocess

import pytest
import torch

from attention_backward_bwd_gb300 import build as b


@pytest.fixture
def calls(tmp_path, monkeypatch):
    """build()'s outputs below tmp_path; the compilers' commands, of which those in `broken` fail."""
    for name in ("LIB", "NATIVE", "BUILD"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name))))
    made, broken = [], set()

    def run(cmd, **kw):
        of = "native" if any(str(a).endswith("native.cpp") for a in cmd) else "link" if "-shared" in cmd else "unit"
        made.append(of)
        if of not in broken:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write(of)
        return subprocess.CompletedProcess(cmd, int(of in broken), "", f"{of} is broken")

    monkeypatch.setattr(b.subprocess, "run", run)
    run.made, run.broken = made, broken
    return run


def test_both_are_built_once(calls):
    assert b.build() == b.LIB and os.path.exists(b.LIB) and os.path.exists(b.NATIVE)
    assert calls.made.count("native") == 1 and calls.made.count("link") == 1
    calls.made.clear()
    assert b.build() == b.LIB and not calls.made


def test_the_library_does_not_wait_for_the_module(calls):
    calls.broken.add("native")
    with pytest.raises(RuntimeError, match="native"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.NATIVE)
    calls.broken.clear()
    calls.made.clear()
    b.build()
    assert calls.made == ["native"] and os.path.exists(b.NATIVE)


def test_a_torch_without_cuda_gets_the_library(calls, monkeypatch):
    monkeypatch.setattr(torch.version, "cuda", None)
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert "native" not in calls.made and not os.path.exists(b.NATIVE)
    calls.made.clear()
    assert b.build() == b.LIB and not calls.made


def test_another_torch_gets_another_module(calls, monkeypatch):
    b.build()
    calls.made.clear()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    b.build()
    assert calls.made == ["native"]
    calls.made.clear()
    b.build()
    assert not calls.made


def test_a_broken_unit_is_an_error(calls):
    calls.broken.add("unit")
    with pytest.raises(RuntimeError, match="unit"):
        b.build()
    assert not os.path.exists(b.LIB)
