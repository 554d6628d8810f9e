"""The extension with the plain f4 calls beside libw4.so: the library is built and
the binding works without it (no GPU needed)."""
import importlib.util
import os
import subprocess

import pytest

from w4_quant_matmul_b200 import build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """An extension file of the test's own, older than its sources."""
    path = tmp_path / "_f4call.so"
    path.write_bytes(b"an older build")
    os.utime(path, (1, 1))
    monkeypatch.setattr(build, "CALLS", str(path))
    return path


def no_torch(monkeypatch):
    real = importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else real(name, *a))


def no_compiler(monkeypatch):
    real = subprocess.run

    def run(cmd, *a, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        return real(cmd, *a, **kw)
    monkeypatch.setattr(build.subprocess, "run", run)


def no_cuda_torch(monkeypatch):
    real = subprocess.run

    def run(cmd, *a, **kw):
        if cmd[0] == "g++":
            return subprocess.CompletedProcess(cmd, 1, "", "cannot find -ltorch_cuda")
        return real(cmd, *a, **kw)
    monkeypatch.setattr(build.subprocess, "run", run)


@pytest.mark.parametrize("without", [no_torch, no_compiler, no_cuda_torch])
def test_the_library_is_built_without_the_extension(monkeypatch, elsewhere, without):
    without(monkeypatch)
    with pytest.warns(UserWarning, match="_f4call.so is not built"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB)
    assert not elsewhere.exists()  # no older one in its place
