"""The optional part of the build: the binding's checks in C.  The library is complete without them."""
import os
import sysconfig

import pytest

from deepseek_v4_compressed_csa_gb300 import build


@pytest.fixture
def target(tmp_path, monkeypatch):
    path = str(tmp_path / os.path.basename(build.CHECKS))
    monkeypatch.setattr(build, "CHECKS", path)
    return path


@pytest.mark.parametrize("cc", [None, "", "gcc -pipe", "env LC_ALL=C gcc"])
def test_compilers_with_and_without_arguments(target, cc, monkeypatch):
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("no Python headers here")
    monkeypatch.delenv("CC", raising=False)
    if cc is not None:
        monkeypatch.setenv("CC", cc)
    assert build.build_checks() == target and os.path.exists(target)


@pytest.mark.parametrize("cc", ["/nonexistent/cc", "false", "gcc --no-such-option", "'unbalanced"])
def test_a_compiler_that_does_not_work_leaves_the_checks_out(target, cc, monkeypatch, capsys):
    """... and an older build's, which may not be this source's, with them."""
    open(target, "w").close()
    monkeypatch.setenv("CC", cc)
    assert build.build_checks() is None and not os.path.exists(target)
    assert "checks" in capsys.readouterr().err


def test_without_python_headers(target, monkeypatch, capsys):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": "/nonexistent"})
    open(target, "w").close()
    assert build.build_checks() is None and not os.path.exists(target)
