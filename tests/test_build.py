"""What build() makes where something is missing or has changed (no compiler is run)."""

import os
import shutil
import types

import pytest

from mixture_experts_ffn_infer_gb300 import build


@pytest.fixture
def ran(tmp_path, monkeypatch):
    """build.build() into an empty folder, with compilers that write a file and are noted."""
    log = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        log.append(os.path.basename(out).split(".tmp")[0])
        with open(out, "w") as f:
            f.write(" ".join(cmd))
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libmoe_ffn.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_mx_torch.so"))
    return log


def made(log):
    """What was linked since the last time."""
    got = {f for f in log if not f.endswith(".o")}
    log.clear()
    return got


def test_everything_once(ran):
    build.build()
    assert made(ran) == {"libmoe_ffn.so", "_mx_torch.so"} and build.up_to_date()
    build.build()
    assert made(ran) == set()


@pytest.mark.parametrize("lacking", ["g++", "torch's headers", "Python's headers", "torch"])
def test_the_library_needs_neither_torch_nor_a_host_compiler_of_its_own(ran, monkeypatch, tmp_path, capsys, lacking):
    if lacking == "g++":
        monkeypatch.setattr(shutil, "which", lambda name: None if name == "g++" else "/usr/bin/" + name)
    elif lacking == "torch's headers":
        monkeypatch.setattr(build, "_torch_paths", lambda: ([str(tmp_path)] * 2, str(tmp_path)))
    elif lacking == "Python's headers":
        monkeypatch.setattr(build, "sysconfig", types.SimpleNamespace(get_paths=lambda: {"include": str(tmp_path)}))
    else:
        find = build.importlib.util.find_spec
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None if name == "torch" else find(name))
    monkeypatch.setattr(build, "nvcc", lambda: "nvcc")
    build.build()
    assert made(ran) == {"libmoe_ffn.so"} and lacking in capsys.readouterr().err
    assert build.up_to_date()
    build.build()
    assert made(ran) == set()


def test_another_torch_means_another_module(ran, monkeypatch):
    build.build()
    made(ran)
    monkeypatch.setattr(build, "_torch_version", lambda: "0.0.1")
    assert not build.up_to_date() and build.library_up_to_date()
    build.build()
    assert made(ran) == {"_mx_torch.so"} and build.up_to_date()


def test_a_changed_source_means_both(ran, monkeypatch):
    build.build()
    made(ran)
    later = os.path.getmtime(build.BINDING) + 10
    sources = build.sources()
    real = os.path.getmtime
    monkeypatch.setattr(os.path, "getmtime", lambda p: later if p == sources[0] and os.path.exists(build.LIB) else real(p))
    assert not build.up_to_date()
    build.build()
    assert made(ran) == {"libmoe_ffn.so", "_mx_torch.so"}


def test_a_failed_module_leaves_the_library(ran, monkeypatch):
    monkeypatch.setattr(build, "compile_binding", lambda: (_ for _ in ()).throw(RuntimeError("g++ failed")))
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
