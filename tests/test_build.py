"""The in-tree build's bookkeeping, with stand-ins for the compilers: the library is
linked whether or not the Python binding builds, and each is rebuilt for its own inputs."""
import importlib.util
import os
import stat

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def bmod(tmp_path, monkeypatch):
    """The build module in a folder of its own, nvcc and g++ writing their outputs' names."""
    spec = importlib.util.spec_from_file_location("_kvq_build_t", os.path.join(ROOT, "fp8_quantized_paged_gb300", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    bin_dir = tmp_path / "bin"
    bin_dir.mkdir()
    for tool in ("nvcc", "g++"):
        f = bin_dir / tool
        f.write_text(f'#!/bin/sh\necho x >> {tmp_path}/calls.{tool}\n[ -e {tmp_path}/broken.{tool} ] && exit 1\n'
                     'while [ $# -gt 0 ]; do [ "$1" = -o ] && echo built > "$2"; shift; done\nexit 0\n')
        f.chmod(f.stat().st_mode | stat.S_IEXEC)
    monkeypatch.setenv("PATH", f"{bin_dir}:{os.environ['PATH']}")
    build = tmp_path / "_build"
    for name, value in (("BUILD", build), ("LIB", build / "libkvq.so"), ("BINDING_LIB", build / "_kvq_fp4.so")):
        monkeypatch.setattr(m, name, str(value))
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "version.py").write_text("__version__ = '1'\n")
    monkeypatch.setattr(m, "_torch_root", lambda: str(torch))
    m.tmp, m.torch = tmp_path, torch
    m.calls = lambda tool: len((tmp_path / f"calls.{tool}").read_text().split()) if (tmp_path / f"calls.{tool}").exists() else 0
    return m


def test_both_are_built_once(bmod):
    for _ in range(2):
        assert bmod.build(lib=bmod.LIB) == bmod.LIB
        assert os.path.exists(bmod.LIB) and os.path.exists(bmod.BINDING_LIB)
        assert bmod.calls("nvcc") == len(bmod.UNITS) + 1 and bmod.calls("g++") == 1


def test_library_without_torch(bmod, monkeypatch, capsys):
    def none():
        raise RuntimeError("torch not found")
    monkeypatch.setattr(bmod, "_torch_root", none)
    assert bmod.build(lib=bmod.LIB) == bmod.LIB
    assert os.path.exists(bmod.LIB) and not os.path.exists(bmod.BINDING_LIB)
    assert "torch not found" in capsys.readouterr().err


def test_library_with_a_binding_that_does_not_compile(bmod, capsys):
    bmod.build(lib=bmod.LIB)
    (bmod.tmp / "broken.g++").write_text("")
    bmod.build(lib=bmod.LIB, force=True)
    assert os.path.exists(bmod.LIB) and "not built" in capsys.readouterr().err
    assert not os.path.exists(bmod.BINDING_LIB)  # nor an old one


def test_binding_follows_torch_and_its_own_source(bmod, monkeypatch):
    bmod.build(lib=bmod.LIB)
    cuda = bmod.calls("nvcc")
    (bmod.torch / "version.py").write_text("__version__ = '2'\n")
    bmod.build(lib=bmod.LIB)
    assert bmod.calls("g++") == 2 and bmod.calls("nvcc") == cuda
    os.utime(bmod.BINDING_LIB, (1, 1))  # older than its source
    bmod.build(lib=bmod.LIB)
    assert bmod.calls("g++") == 3 and bmod.calls("nvcc") == cuda
    os.utime(bmod.LIB, (1, 1))
    bmod.build(lib=bmod.LIB)
    assert bmod.calls("g++") == 3 and bmod.calls("nvcc") == 2 * cuda
