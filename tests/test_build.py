"""The library's build without what only the binding module needs, and the errors of
a build that has it."""
import os

import pytest

from gemm_swiglu_mlp_gb300 import build, cache


@pytest.fixture
def library(monkeypatch, tmp_path):
    """A build whose library is there and whose binding is not."""
    build.build()
    path = str(tmp_path / "_cache_binding_test.so")
    monkeypatch.setattr(build, "BINDING_PATH", path)
    monkeypatch.setattr(cache, "BINDING_PATH", path)
    monkeypatch.setattr(cache, "_binding", None)
    return path


def no_python_headers(monkeypatch, tmp_path):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})


def no_torch(monkeypatch, tmp_path):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)


@pytest.mark.parametrize("without,named", [(no_python_headers, "Python's headers"),
                                           (no_torch, "PyTorch")])
def test_library_is_built_without_the_bindings_headers(library, monkeypatch, tmp_path, capsys,
                                                       without, named):
    with monkeypatch.context() as m:
        without(m, tmp_path)
        assert build.build() == build.LIB_PATH
        assert named in capsys.readouterr().err and not os.path.exists(library)
        with pytest.raises(RuntimeError, match=named):      # the calls say what is missing
            cache._native()
    assert build.binding_needs() == []


def test_torch_need_not_be_installed(monkeypatch):
    def nothing(name):
        raise build.importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(build.importlib.metadata, "version", nothing)
    assert build._torch_version() == "none"


def test_an_error_in_the_binding_is_raised(library, monkeypatch, tmp_path):
    source = tmp_path / "bad.cpp"
    source.write_text("#error no\n")
    monkeypatch.setattr(build, "BINDING_SOURCE", str(source))
    with pytest.raises(RuntimeError):
        build.build()
    assert not os.path.exists(library)
