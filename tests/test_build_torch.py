"""The part of the build that has torch's tensor layout compiled in is used under the torch that it was built for, and under no
other."""
import ctypes
import os

import pytest
import torch

import deepseek_v4_compressed_csa_gb300 as csa
from deepseek_v4_compressed_csa_gb300 import _binding as B
from deepseek_v4_compressed_csa_gb300 import build


@pytest.fixture(scope="module")
def built():
    if not os.path.exists(B.LIB_PATH):
        build.build()
    csa.load_library()
    if not os.path.exists(build.TENSORS):
        pytest.skip("not built here (no headers of torch)")
    return build.TENSORS


def test_it_says_which_torch(built):
    f = ctypes.CDLL(built).csa_tensors_torch
    f.restype = ctypes.c_char_p
    assert f().decode() == f"{torch.__version__} {torch.version.git_version}"
    assert B._tensors() == ctypes.cast(ctypes.CDLL(built).csa_tensor, ctypes.c_void_p).value


@pytest.mark.parametrize("version,commit", [("2.99.0", None), (None, "0" * 40), (None, "")])
def test_another_torch_asks_by_attributes(built, version, commit, monkeypatch):
    """Another release, or another commit that goes by the same version: its symbols may all be there."""
    if version is not None:
        monkeypatch.setattr(torch, "__version__", version)
    if commit is not None:
        monkeypatch.setattr(torch.version, "git_version", commit)
    assert B._tensors() == 0


@pytest.mark.parametrize("text", ["", "int csa_other(void) { return 1; }", "const char* csa_tensors_torch(void) { return \"\"; }",
                                  "int csa_tensor(void) { return 1; }"])
def test_a_library_that_does_not_say(text, tmp_path):
    """One without the functions, or that is no library: as if it were not there."""
    import shutil
    import subprocess
    path = str(tmp_path / "libcsa_tensors.so")
    assert B._tensors(path) == 0
    if not text:
        open(path, "w").write("no library")
    else:
        if shutil.which("gcc") is None:
            pytest.skip("no C compiler")
        (tmp_path / "t.c").write_text(text)
        subprocess.run(["gcc", "-shared", "-fPIC", "-o", path, str(tmp_path / "t.c")], check=True)
    assert B._tensors(path) == 0


def test_without_it_calls_ask_by_attributes(built):
    """The checks in C take 0 for 'not there', and the address again."""
    if B._plain is None:
        pytest.skip("the checks in C are not built here (no Python headers)")
    try:
        B._plain.tensors(0)
        assert B._plain.add_norm(0, b"", torch.bfloat16, *([None] * 9)) is None
    finally:
        B._plain.tensors(B._tensors())
