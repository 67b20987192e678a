"""What is rebuilt when: the CUDA library and the marshalling module stand on their own."""
import os
import shutil

import pytest
import torch

from fp8_fine_grained_amax_gb300 import build


@pytest.fixture
def built(monkeypatch, tmp_path):
    """An up-to-date build whose module is a copy, and the list of build steps that are taken."""
    build.build_library()
    steps = []
    ext = str(tmp_path / "_torch_calls.so")
    shutil.copy2(build.EXT, ext)
    monkeypatch.setattr(build, "EXT", ext)
    monkeypatch.setattr(build, "_compile", lambda src: steps.append(src) or pytest.fail("recompiled " + src))
    monkeypatch.setattr(build, "_compile_ext", lambda: steps.append("module") or "module.o")
    monkeypatch.setattr(build, "_link_ext", lambda obj: steps.append("link"))
    return steps


def test_nothing_is_rebuilt_without_need(built):
    assert build.build_library() == build.LIB and built == []


def test_a_module_that_does_not_build_leaves_the_library(built, monkeypatch):
    def fails():
        built.append("module")
        raise RuntimeError("g++ failed")

    os.remove(build.EXT)
    monkeypatch.setattr(build, "_compile_ext", fails)
    for _ in range(3):
        with pytest.warns(RuntimeWarning, match="g\\+\\+ failed"):
            assert build.build_library() == build.LIB
    assert set(built) == {"module"}


def test_an_older_module_does_not_stay_where_the_new_one_fails(built, monkeypatch):
    def fails():
        raise RuntimeError("g++ failed")

    os.utime(build.EXT, (0, 0))
    monkeypatch.setattr(build, "_compile_ext", fails)
    with pytest.warns(RuntimeWarning):
        build.build_library()
    assert not os.path.exists(build.EXT)


def test_the_module_is_rebuilt_for_another_torch(built, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    build.build_library()
    assert built == ["module", "link"]
