"""build(): libm3.so does not depend on what the serving operators' binding needs (no GPU needed)."""
import os

import pytest


@pytest.fixture
def builder(tmp_path, monkeypatch):
    from autoregressive_audio_token_b200 import build
    build.build()  # whatever is missing here is built once
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_ops.so"))
    return build


def _hide_torch(monkeypatch, build):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)


def _hide_headers(monkeypatch, build):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": "/nowhere"})


def _hide_compiler(monkeypatch, build):
    monkeypatch.setenv("CXX", "/nowhere/c++")


@pytest.mark.parametrize("hide,what", [(_hide_torch, "torch"), (_hide_headers, "Python.h"), (_hide_compiler, "/nowhere/c++")])
def test_the_library_without_the_binding(builder, monkeypatch, capfd, hide, what):
    hide(monkeypatch, builder)
    assert builder.build() == builder.LIB
    assert f"{what} is missing" in capfd.readouterr().err
    assert not os.path.exists(builder.BINDING)


def test_a_module_older_than_its_sources_does_not_stay(builder, monkeypatch):
    _hide_compiler(monkeypatch, builder)
    with open(builder.BINDING, "w"):
        pass
    builder.build()
    assert os.path.exists(builder.BINDING)  # newer: nothing to build
    os.utime(builder.BINDING, (1, 1))
    builder.build()
    assert not os.path.exists(builder.BINDING)
