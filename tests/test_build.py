"""What a build needs: hipcc for the C libraries, and PyTorch for the binding only."""
import os
import subprocess

import pytest

from hadamard_rotated_w4a4_amd import build as hip


@pytest.fixture
def commands(monkeypatch):
    """The compilers' command lines of a build that runs none of them."""
    run = []
    monkeypatch.setattr(hip, "_run", lambda cmd, tool, verbose: run.append(cmd))
    monkeypatch.setattr(hip.os, "replace", lambda a, b: None)
    return run


def test_the_c_libraries_are_built_without_pytorch(commands, monkeypatch, capsys):
    real = hip.importlib.util.find_spec
    monkeypatch.setattr(hip.importlib.util, "find_spec", lambda name: None if name == "torch" else real(name))
    monkeypatch.setitem(hip.sys.modules, "torch", None)  # importing it fails
    assert hip.build() == hip.LIB
    assert [cmd[cmd.index("-o") + 1] for cmd in commands] == [hip.LIB + ".tmp", hip.CEILINGS_LIB + ".tmp"]
    assert "_native.so is not" in capsys.readouterr().out


def test_the_binding_takes_the_headers_of_its_hipcc(commands, monkeypatch, tmp_path):
    pytest.importorskip("torch")
    for made in ("bin/hipcc", "include/hip/hip_runtime.h"):
        path = tmp_path / "rocm" / made
        path.parent.mkdir(parents=True)
        path.write_text("")
        path.chmod(0o755)
    monkeypatch.setattr(hip, "HIPCC", str(tmp_path / "rocm" / "bin" / "hipcc"))
    hip.build()
    native = commands[-1]
    assert len(commands) == 3 and native[-1].startswith("-Wl,-rpath")
    assert f"-isystem{tmp_path / 'rocm' / 'include'}" in native and "-isystem/opt/rocm/include" not in native
    os.symlink(tmp_path / "rocm" / "bin" / "hipcc", tmp_path / "hipcc")  # a link on PATH, say
    monkeypatch.setattr(hip, "HIPCC", str(tmp_path / "hipcc"))
    assert hip._rocm_include() == str(tmp_path / "rocm" / "include")


def test_a_compiler_that_fails_is_reported(monkeypatch):
    monkeypatch.setattr(hip.subprocess, "run",
                        lambda cmd, **kw: subprocess.CompletedProcess(cmd, 1, "", "no such header"))
    with pytest.raises(RuntimeError, match="no such header"):
        hip.build()
