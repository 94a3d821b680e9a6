"""The library is linked without torch and without a host compiler; only the Python binding needs them (CPU only,
the compilers are stood in for)."""
import os
import subprocess
import sys

import pytest

sys.path.insert(0, os.path.join(os.path.dirname(__file__), "..", "bitwise_reproducible_amd", "csrc"))
import build as lib_build  # noqa: E402


@pytest.fixture
def run(monkeypatch, tmp_path):
    """Runs build() in an empty folder; the commands that it ran, by the program."""
    def call(host_fails):
        commands = []

        def stand_in(cmd, **kw):
            commands.append(cmd)
            fails = host_fails and cmd[0] != lib_build.HIPCC
            if not fails:
                with open(cmd[cmd.index("-o") + 1], "w"):
                    pass
            return subprocess.CompletedProcess(cmd, int(fails), "", "no host compiler" if fails else "")

        for name in ("LIB", "RATES_LIB", "BINDING_LIB"):
            monkeypatch.setattr(lib_build, name, str(tmp_path / os.path.basename(getattr(lib_build, name))))
        monkeypatch.setattr(lib_build, "BUILD_DIR", str(tmp_path / "objects"))
        monkeypatch.setattr(lib_build.subprocess, "run", stand_in)
        try:
            return lib_build.build()
        finally:
            monkeypatch.undo()
    return call


def test_library_without_torch(run, monkeypatch, tmp_path, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    assert run(host_fails=False) == str(tmp_path / "librepro.so")
    assert (tmp_path / "librepro.so").exists() and (tmp_path / "libvalu_rates.so").exists()
    assert not (tmp_path / "_layer.so").exists()
    assert "torch" in capsys.readouterr().out


def test_library_without_a_host_compiler(run, tmp_path):
    # The binding's failure is an error, but the library is there by then.
    with pytest.raises(RuntimeError, match="no host compiler"):
        run(host_fails=True)
    assert (tmp_path / "librepro.so").exists() and not (tmp_path / "_layer.so").exists()


def test_all_is_built(run, tmp_path):
    run(host_fails=False)
    assert {"librepro.so", "libvalu_rates.so", "_layer.so"} <= set(os.listdir(tmp_path))
