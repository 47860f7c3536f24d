"""The optional part of the build that reads torch's tensors directly: the checks in C work without it, and it says no more
of a tensor than its attributes do."""
import ctypes
import os

import pytest
import torch

import deepseek_v4_compressed_csa_gb300 as csa
from deepseek_v4_compressed_csa_gb300 import _binding as B
from deepseek_v4_compressed_csa_gb300 import build


@pytest.fixture
def target(tmp_path, monkeypatch):
    path = str(tmp_path / os.path.basename(build.TENSORS))
    monkeypatch.setattr(build, "TENSORS", path)
    return path


@pytest.mark.parametrize("cxx", ["/nonexistent/c++", "false", "g++ --no-such-option", "'unbalanced"])
def test_a_compiler_that_does_not_work_leaves_it_out(target, cxx, monkeypatch, capsys):
    """... and an older build's with it."""
    open(target, "w").close()
    monkeypatch.setenv("CXX", cxx)
    assert build.build_tensors() is None and not os.path.exists(target)
    assert "attributes" in capsys.readouterr().err


@pytest.fixture(scope="module")
def look():
    csa.load_library()
    if not os.path.exists(build.TENSORS):
        pytest.skip("not built here (no headers of torch)")
    f = ctypes.PyDLL(build.TENSORS).csa_tensor
    f.argtypes = [ctypes.py_object, ctypes.py_object, ctypes.c_int] + [ctypes.c_void_p] * 4
    f.restype = ctypes.c_int

    def call(t, dtype, most=8):
        n, dims, dev, p = ctypes.c_int(), (ctypes.c_longlong * 8)(), ctypes.c_longlong(), ctypes.c_void_p()
        r = f(t, dtype, most, ctypes.addressof(n), ctypes.addressof(dims), ctypes.addressof(dev), ctypes.addressof(p))
        return (r, tuple(dims[: n.value]), dev.value, p.value) if r == 1 else r
    return call


def test_what_is_no_plain_tensor(look):
    class Sub(torch.Tensor):
        pass
    t = torch.zeros(2, 3)
    for o in (None, 5, "t", [t], t.as_subclass(Sub), type("T", (), dict(dtype=torch.float32))()):
        assert look(o, torch.float32) == -1
    assert look(t, "float32") == -1 and look(t, None) == -1
    # tensors that are not on a GPU, or have no address
    for o in (t, torch.nn.Parameter(t), torch.empty(2, device="meta"), t.to_sparse(), torch.zeros(())):
        assert look(o, torch.float32) == 0


@pytest.mark.gpu
def test_tensors_on_the_gpu(look):
    t = torch.zeros(2, 3, 4, device="cuda", dtype=torch.bfloat16)
    want = (1, (2, 3, 4), 0, t.data_ptr())
    assert look(t, torch.bfloat16) == want and look(torch.nn.Parameter(t), torch.bfloat16) == want
    assert look(t[1], torch.bfloat16) == (1, (3, 4), 0, t[1].data_ptr())
    assert look(t[:0], torch.bfloat16)[:2] == (1, (0, 3, 4))
    assert look(t, torch.float16) == 0 and look(t, torch.bfloat16, 2) == 0
    assert look(t[:, :2], torch.bfloat16) == 0 and look(t.transpose(0, 1), torch.bfloat16) == 0
    assert look(t.to_sparse(), torch.bfloat16) == 0


@pytest.mark.gpu
def test_calls_with_and_without(look):
    """The same outputs, and the same refusals, whichever way the checks look at the tensors."""
    if B._plain is None:
        pytest.skip("the checks in C are not built here (no Python headers)")
    L = csa.Layer(dtype=torch.bfloat16, H=64, D=512, R=64, W=128, ratio=4, Hi=64, Di=128, topk=512, X=4096)
    x, w = torch.randn(5, 4096, device="cuda").bfloat16(), torch.randn(4096, device="cuda")
    outs = []
    address = ctypes.cast(ctypes.CDLL(build.TENSORS).csa_tensor, ctypes.c_void_p).value
    try:
        for at in (address, 0):
            B._plain.tensors(at)
            kept = dict(out=torch.empty_like(x), residual_out=torch.empty_like(x), codes=torch.empty(5, 4096, dtype=torch.uint8, device="cuda"),
                        scales=torch.empty(5, 32, device="cuda"))
            csa.add_norm(L, x, x, w, group=128, **kept)
            outs.append(kept)
            for bad in (dict(out=kept["out"][:4]), dict(codes=kept["scales"]), dict(scales=kept["scales"].cpu())):
                with pytest.raises((TypeError, ValueError)):
                    csa.add_norm(L, x, x, w, group=128, **{**kept, **bad})
    finally:
        B._plain.tensors(address)
    assert all(torch.equal(outs[0][k], outs[1][k]) for k in outs[0])
