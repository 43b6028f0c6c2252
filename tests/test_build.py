"""The build's two products: the C library does not depend on what only the Python binding
needs, and each is made again when its own inputs are newer. The compilers are stand-ins."""
import os
import sysconfig
import types

import pytest

from structured_sparse_matmul_gb300 import build


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Build into an empty folder with compilers that only write their output; the outputs made."""
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libvnm.so"))
    monkeypatch.setattr(build, "BINDING_PATH", str(tmp_path / os.path.basename(build.BINDING_PATH)))
    outputs, broken = [], []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        if any(b in cmd[0] for b in broken):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="no such compiler")
        open(out, "w").close()
        outputs.append(os.path.basename(out))
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build.subprocess, "run", run)
    return types.SimpleNamespace(outputs=outputs, broken=broken)


def test_both_are_built_once(made):
    build.build()
    assert os.path.exists(build.LIB_PATH) and os.path.exists(build.BINDING_PATH) and build.up_to_date()
    n = len(made.outputs)
    build.build()
    assert len(made.outputs) == n


def test_the_library_without_a_host_compiler_for_the_binding(made, monkeypatch):
    monkeypatch.setenv("CC", "absent-compiler")
    made.broken.append("absent-compiler")
    with pytest.raises(RuntimeError):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)
    made.broken.clear()
    n = len(made.outputs)
    build.build()  # the binding alone
    assert len(made.outputs) == n + 1 and build.up_to_date()


def test_the_library_without_pythons_headers(made, monkeypatch, tmp_path, capsys):
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.BINDING_PATH)
    assert "Python.h" in capsys.readouterr().err


def test_the_binding_is_for_this_python():
    assert build.BINDING_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
