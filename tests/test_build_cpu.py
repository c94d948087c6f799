"""The build's decisions, with compilers replaced by stubs that write text files."""
import os
import shutil
import sys
import time

import pytest

from depthwise_convolution_nhwc_gb300 import _build

HOST_OBJECT = _build._host_object


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package folder with a finished library, one host source and stub compilers; `use(version)` is the
    PyTorch version of the next build."""
    csrc, objs = tmp_path / "csrc", tmp_path / "_build"
    csrc.mkdir()
    (csrc / "dwc_norm_py.cpp").write_text("source")
    (tmp_path / "lib.so").write_text("library")
    past = time.time() - 1000
    os.utime(csrc / "dwc_norm_py.cpp", (past, past))
    monkeypatch.setattr(_build, "CSRC", str(csrc))
    monkeypatch.setattr(_build, "ROOT", str(tmp_path))
    monkeypatch.setattr(_build, "OBJ_DIR", str(objs))
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_build, "HOST_SRC", str(csrc / "dwc_norm_py.cpp"))
    monkeypatch.setattr(_build, "HOST_PATH", str(tmp_path / "host.so"))
    monkeypatch.setattr(_build, "nvcc_path", lambda: "nvcc")
    clock = [past + 10]

    def stamped(path):
        clock[0] += 10
        os.utime(path, (clock[0], clock[0]))

    def compile_host(obj):
        with open(obj, "w") as f:
            f.write(os.path.basename(obj))
        stamped(obj)
        calls.append("compile")

    def link_host(obj):
        shutil.copyfile(obj, _build.HOST_PATH)
        stamped(_build.HOST_PATH)
        calls.append("link")

    calls = []
    monkeypatch.setattr(_build, "_compile_host", compile_host)
    monkeypatch.setattr(_build, "_link_host", link_host)

    def use(version):
        monkeypatch.setattr(_build, "_host_object", lambda: str(objs / f"host-{version}.o"))

    return use, calls


def linked():
    with open(_build.HOST_PATH) as f:
        return f.read()


def test_the_host_module_is_that_of_the_version_in_use(tree):
    use, calls = tree
    for version in ("a", "b", "a", "b", "a"):
        use(version)
        _build.build()
        assert linked() == f"host-{version}.o", version
    assert calls.count("compile") == 2


def test_nothing_is_done_twice(tree):
    use, calls = tree
    use("a")
    for _ in range(3):
        _build.build()
    assert calls == ["compile", "link"]
    os.remove(_build.HOST_PATH)
    _build.build()
    assert calls == ["compile", "link", "link"]
    now = time.time()
    os.utime(_build.HOST_SRC, (now, now))
    _build.build()
    assert calls[3:] == ["compile", "link"]


def test_the_library_is_built_without_pytorch(tree, monkeypatch):
    """The C ABI needs no PyTorch, nor does its build, which then leaves out the host module."""
    _, calls = tree
    monkeypatch.setattr(_build, "_host_object", HOST_OBJECT)
    monkeypatch.setitem(sys.modules, "torch", None)     # `import torch` raises ImportError
    assert _build.build() == _build.LIB_PATH and calls == []
