"""The library without the binding's compiled host side: a machine without a C++
compiler still gets libfp8blk.so, and a host side that does not load costs speed,
not the library."""
import os
import subprocess

import pytest
import torch

from blockwise_fp8_pretraining_b200 import _abi, build


@pytest.fixture
def fresh(monkeypatch):
    """The binding before its first load."""
    build.build()
    monkeypatch.setattr(_abi, "_lib", None)
    monkeypatch.setattr(_abi, "_host", None)


@pytest.mark.parametrize("error", [FileNotFoundError("g++"), subprocess.CalledProcessError(1, ["g++"])])
def test_no_compiler(monkeypatch, tmp_path, capsys, error):
    """build() compiles the library first, and without a host side says so."""
    ran = []

    def run(cmd, **kwargs):
        ran.append(cmd[0])
        if cmd[0].endswith("nvcc"):
            open(cmd[cmd.index("-o") + 1], "w").close()
        else:
            raise error

    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfp8blk.so"))
    monkeypatch.setattr(build, "HOST_LIB", str(tmp_path / "host.so"))
    monkeypatch.setattr(build.subprocess, "check_call", run)
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    (tmp_path / "host.so").write_bytes(b"of an older header")
    os.utime(tmp_path / "host.so", (1, 1))
    assert build.build() == str(tmp_path / "libfp8blk.so")
    assert os.path.exists(build.LIB) and not os.path.exists(build.HOST_LIB)
    assert ran[0].endswith("nvcc") and len(ran) == 2
    assert "host side was not built" in capsys.readouterr().err


def test_a_failed_library_build_is_an_error(monkeypatch, tmp_path):
    def run(cmd, **kwargs):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfp8blk.so"))
    monkeypatch.setattr(build.subprocess, "check_call", run)
    with pytest.raises(subprocess.CalledProcessError):
        build.build()


def test_a_host_side_that_does_not_load(fresh, monkeypatch, tmp_path):
    broken = tmp_path / "host.so"
    broken.write_bytes(b"not a shared object")
    monkeypatch.setattr(build, "HOST_LIB", str(broken))
    with pytest.warns(RuntimeWarning, match="does not load"):
        lib = _abi.load()
    assert _abi._host is None
    assert lib.fp8_status_string(0) is not None
    with pytest.raises(ValueError):                  # the Python checks are at work
        _abi.fp8_token_logprobs(torch.zeros(4, 100))


def test_no_host_side(fresh, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "HOST_LIB", str(tmp_path / "none.so"))
    _abi.load()
    assert _abi._host is None
