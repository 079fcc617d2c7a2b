"""The C library is built where the Python binding of the layer operators cannot be: with a small
source in the library's place."""
import ctypes
import os
import shutil

import pytest

from moe_grouped_gemm_fp32_amd import build

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs hipcc")


@pytest.fixture
def small(tmp_path, monkeypatch):
    src = tmp_path / "small.hip"
    src.write_text('extern "C" int answer() { return 42; }\n')
    monkeypatch.setattr(build, "SRCS", [str(src)])
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(build, "CALL", str(tmp_path / "call.so"))
    return tmp_path


def made(folder):
    assert ctypes.CDLL(str(folder / "lib.so")).answer() == 42
    return sorted(p.name for p in folder.iterdir()) == ["lib.so", "small.hip"]  # and nothing half done


def test_no_host_compiler(small, monkeypatch):
    monkeypatch.setenv("CXX", str(small / "no-such-compiler"))
    with pytest.raises(RuntimeError, match="call.so"):
        build.build(verbose=False)
    assert made(small)


def test_no_headers(small, monkeypatch):
    def missing():
        raise ImportError("no torch")
    monkeypatch.setattr(build, "_call_command", missing)
    with pytest.raises(RuntimeError, match="no torch"):
        build.build(verbose=False)
    assert made(small)


def test_a_binding_that_does_not_compile(small, monkeypatch, tmp_path_factory):
    bad = tmp_path_factory.mktemp("bad") / "bad.cpp"
    bad.write_text("int f( {\n")
    monkeypatch.setattr(build, "CALL_SRC", str(bad))
    with pytest.raises(RuntimeError, match="call.so"):
        build.build(verbose=False)
    assert made(small)


def test_a_library_that_does_not_compile_is_raised(small):
    (small / "small.hip").write_text("int f( {\n")
    with pytest.raises(RuntimeError, match="lib.so"):
        build.build(verbose=False)
    assert not (small / "lib.so").exists()


def test_the_library_alone(small):
    assert build.build_library(verbose=False) == str(small / "lib.so")
    assert made(small)
