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


def test_the_extension_is_built_for_this_torch(monkeypatch, tmp_path):
    torch = pytest.importorskip("torch")
    if not os.path.exists(build.CALLS):
        pytest.skip("the extension cannot be built here")
    tag = build.calls_tag(torch.__version__)
    spec = importlib.util.find_spec("torch")
    assert build._torch_version(os.path.dirname(spec.origin)) == torch.__version__
    assert build._built_for(build.CALLS, tag)
    assert not build._built_for(build.CALLS, build.calls_tag("1.0"))
    # newer than its sources, but of another torch: built again
    path = tmp_path / "_f4call.so"
    path.write_bytes(b"\x7fELF ... " + build.calls_tag("1.0").encode())
    monkeypatch.setattr(build, "CALLS", str(path))
    assert build.build_calls() == str(path)
    assert build._built_for(str(path), tag)
    # and left alone where it fits
    before = path.stat().st_mtime_ns
    build.build_calls()
    assert path.stat().st_mtime_ns == before


def test_an_extension_of_another_torch_is_not_called(monkeypatch):
    torch = pytest.importorskip("torch")
    import w4_quant_matmul_b200 as w4
    monkeypatch.setattr(w4, "_ext", None)
    monkeypatch.setattr(torch, "__version__", "1.0")
    with pytest.warns(UserWarning, match="built for another torch"):
        assert w4._calls() is False
    with pytest.raises(ValueError, match="must be a CUDA tensor"):  # the other way, as ever
        w4.f4_dequantize(torch.zeros((4, 32), dtype=torch.uint8),
                         torch.zeros((1, 1, 512), dtype=torch.uint8), None)
