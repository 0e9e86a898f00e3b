"""What build() makes: the C library needs neither torch nor the Python module."""

import os

import pytest

from wavelet_guided_sparse_gb300 import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """Runs nothing: every command writes its output, and is listed."""
    ran = []

    def run(what, cmd, verbose):
        ran.append(what)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libwavefilter.so"))
    monkeypatch.setattr(build, "MODULE", str(tmp_path / "_wf_torch.so"))
    return ran


def test_library_and_module(commands, tmp_path):
    assert build.build() == str(tmp_path / "libwavefilter.so")
    assert sorted(x for x in os.listdir(tmp_path) if x.endswith(".so")) == \
        ["_wf_torch.so", "libwavefilter.so"]
    assert len(commands) == len(build.sources()) + 3


def test_without_torch_the_library_is_built(commands, monkeypatch, tmp_path):
    real = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else real(name, *a))
    assert build.build() == str(tmp_path / "libwavefilter.so")
    assert os.path.exists(tmp_path / "libwavefilter.so")
    assert not os.path.exists(tmp_path / "_wf_torch.so")
    assert not any("wf_torch" in x or "module" in x for x in commands)


def test_a_module_that_does_not_compile_leaves_the_library(commands, monkeypatch, tmp_path):
    run = build._run

    def fails(what, cmd, verbose):
        if "wf_torch" in what:
            raise RuntimeError("g++ on wf_torch.cpp failed")
        run(what, cmd, verbose)

    monkeypatch.setattr(build, "_run", fails)
    with pytest.raises(RuntimeError, match="wf_torch"):
        build.build()
    assert os.path.exists(tmp_path / "libwavefilter.so")
