"""The tree calls without a GPU: what the binding and the C ABI refuse on the host, before anything is enqueued."""
import ctypes
import os

import numpy as np
import pytest
import torch

import deepseek_v4_compressed_csa_gb300 as csa
from deepseek_v4_compressed_csa_gb300 import _binding as B
from tests import _tree as TR

FAKE = 0x7f0000000000  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from deepseek_v4_compressed_csa_gb300 import build
        build.build()
    return csa.load_library()


def _layer(**kw):
    base = dict(dtype=B.CSA_BF16, H=64, D=512, R=64, W=128, ratio=4, Hi=64, Di=128, topk=512, X=4096, scale=0.0,
                rms_eps=1e-6, rollback=0, index_fp8=0)
    base.update(kw)
    return B._Layer(*[base[f] for f, _ in B._Layer._fields_])


def _nr(lib, n=1, B_=1, T=1, parent=None, pos=FAKE, invf=FAKE, err=FAKE, layer=None, **row):
    base = dict(x=FAKE, out=FAKE + 4096, weight=None, heads=64, dim=512, norm=1, x_stride=0)
    base.update(row)
    rows = (B._Rows * 4)(*[B._Rows(*[base[f] for f, _ in B._Rows._fields_])] * 4)
    return lib.csa_norm_rope(ctypes.byref(layer or _layer()), rows, n, B_, T, parent, pos, invf, err, None)


def test_norm_rope_refusals(lib):
    for bad in (dict(n=0), dict(n=5), dict(B_=0), dict(T=0), dict(B_=1 << 12, T=1 << 13), dict(parent=FAKE, T=65),
                dict(parent=FAKE + 2), dict(pos=None), dict(invf=FAKE + 4), dict(err=None), dict(x=FAKE + 8),
                dict(out=None), dict(weight=FAKE + 4), dict(heads=0), dict(heads=4097), dict(dim=0), dict(dim=1032),
                dict(dim=516), dict(dim=56), dict(norm=2), dict(x_stride=64 * 512 - 8), dict(x_stride=64 * 512 + 4),
                dict(x_stride=-8), dict(out=FAKE, x_stride=64 * 512 + 8), dict(layer=_layer(R=60))):
        assert _nr(lib, **bad) == B.CSA_ERR_ARG, bad


def _comp(d):
    return ctypes.byref(B._Comp(FAKE, FAKE, FAKE, FAKE, d))


def _compress(lib, layer=None, ca=True, ci=True, ws_bytes=1 << 34, ws=FAKE, B_=2, T=8, **over):
    a = dict(x=FAKE, parent=FAKE, pos=FAKE, fa=FAKE, pa=FAKE, ra=FAKE, fi=FAKE, pi=FAKE, ri=FAKE, invf=FAKE, err=FAKE)
    a.update(over)
    return lib.csa_compress_tree(ctypes.byref(layer or _layer()), _comp(512) if ca is True else ca,
                                 _comp(128) if ci is True else ci, a["x"], B_, T, a["parent"], a["pos"], a["fa"], a["pa"],
                                 a["ra"], a["fi"], a["pi"], a["ri"], a["invf"], ws, ws_bytes, a["err"], None)


def test_compress_tree_refusals(lib):
    for k in ("x", "parent", "pos", "fa", "pa", "ra", "fi", "pi", "ri", "invf", "err"):
        assert _compress(lib, **{k: None}) == B.CSA_ERR_ARG, k
        assert _compress(lib, **{k: FAKE + 2}) == B.CSA_ERR_ARG, k
    assert _compress(lib, T=65) == B.CSA_ERR_ARG and _compress(lib, T=0) == B.CSA_ERR_ARG
    assert _compress(lib, B_=0) == B.CSA_ERR_ARG and _compress(lib, B_=65535, T=64) == B.CSA_ERR_ARG
    assert _compress(lib, ca=None) == B.CSA_ERR_ARG
    assert _compress(lib, ca=_comp(128)) == B.CSA_ERR_ARG and _compress(lib, ci=_comp(512)) == B.CSA_ERR_ARG
    assert _compress(lib, layer=_layer(ratio=128)) == B.CSA_ERR_UNSUPPORTED
    f32 = dict(layer=_layer(dtype=B.CSA_F32))  # (the tensor-core projection of the bf16 layer needs no workspace)
    assert _compress(lib, ws_bytes=1024, **f32) == B.CSA_ERR_WORKSPACE
    assert _compress(lib, ws=None, **f32) == B.CSA_ERR_WORKSPACE


def test_index_scores_tree_refusals(lib):
    def call(layer=None, B_=2, T=8, cap=100, ws=None, ws_bytes=0, **over):
        a = dict(iq=FAKE, iw=FAKE, parent=FAKE, ikeys=FAKE, rows=FAKE, n_rows=FAKE, pos=FAKE, scores=FAKE, err=FAKE)
        a.update(over)
        return lib.csa_index_scores_tree(ctypes.byref(layer or _layer()), a["iq"], a["iw"], B_, T, a["parent"],
                                         a["ikeys"], cap, a["rows"], a["n_rows"], a["pos"], a["scores"], ws, ws_bytes,
                                         a["err"], None)
    for k in ("iq", "iw", "parent", "ikeys", "rows", "n_rows", "pos", "scores", "err"):
        assert call(**{k: None}) == B.CSA_ERR_ARG, k
        assert call(**{k: FAKE + 1}) == B.CSA_ERR_ARG, k
    for k in ("iq", "iw", "ikeys", "rows"):  # rows that are read 16 bytes at a time
        assert call(**{k: FAKE + 8}) == B.CSA_ERR_ARG, k
    assert call(T=65) == B.CSA_ERR_ARG and call(cap=0) == B.CSA_ERR_ARG and call(B_=0) == B.CSA_ERR_ARG
    assert call(cap=2 ** 31 - 256) == B.CSA_ERR_ARG
    assert call(layer=_layer(ratio=128)) == B.CSA_ERR_UNSUPPORTED
    # fp8 rows: the queries' codes and weights go into the workspace
    fp8, need = _layer(index_fp8=1), 2 * 8 * 64 * 132
    for kw in (dict(), dict(ws=FAKE, ws_bytes=need - 1), dict(ws_bytes=need), dict(ws=FAKE + 8, ws_bytes=need)):
        assert call(layer=fp8, **kw) == B.CSA_ERR_WORKSPACE, kw
    n = ctypes.c_size_t()
    assert lib.csa_workspace_size(ctypes.byref(fp8), B.OP_INDEX_SCORES_TREE, 2, 8, 1, ctypes.byref(n)) == 0
    assert n.value == need
    assert lib.csa_workspace_size(ctypes.byref(_layer()), B.OP_INDEX_SCORES_TREE, 2, 8, 1, ctypes.byref(n)) == 0
    assert n.value == 0


def test_attend_tree_refusals(lib):
    def call(layer=None, B_=2, T=8, cap=100, ws=FAKE, ws_bytes=1 << 34, **over):
        a = dict(q=FAKE, kv=FAKE, sink=FAKE, parent=FAKE, window=FAKE, pool=FAKE, rows=FAKE, scores=FAKE, n_rows=FAKE,
                 pos=FAKE, invf=FAKE, out=FAKE, sel=None, err=FAKE)
        a.update(over)
        return lib.csa_attend_tree(ctypes.byref(layer or _layer()), a["q"], a["kv"], a["sink"], B_, T, a["parent"],
                                   a["window"], a["pool"], cap, a["rows"], a["scores"], a["n_rows"], a["pos"], a["invf"],
                                   a["out"], a["sel"], ws, ws_bytes, a["err"], None)
    for k in ("q", "kv", "sink", "parent", "window", "pool", "rows", "n_rows", "pos", "invf", "out", "err"):
        assert call(**{k: None}) == B.CSA_ERR_ARG, k
        assert call(**{k: FAKE + 2}) == B.CSA_ERR_ARG, k
    assert call(T=65) == B.CSA_ERR_ARG and call(cap=0) == B.CSA_ERR_ARG
    assert call(cap=2 ** 31 - 256) == B.CSA_ERR_ARG
    assert call(layer=_layer(ratio=128)) == B.CSA_ERR_ARG          # scores on a layer without an indexer
    assert call(scores=None, sel=FAKE) == B.CSA_ERR_ARG            # a selection without scores
    assert call(sel=FAKE + 2) == B.CSA_ERR_ARG
    assert call(ws_bytes=64) == B.CSA_ERR_WORKSPACE


def test_commit_tree_refusals(lib):
    names = ("parent", "leaf", "pos", "pos_out", "kv", "window", "pa", "fa", "ra", "pla", "na", "nao", "pi", "fi", "ri",
             "pli", "ni", "nio", "err")

    def call(layer=None, B_=2, T=8, cap_a=100, cap_i=100, **over):
        a = dict.fromkeys(names, FAKE)
        a.update(over)
        return lib.csa_commit_tree(ctypes.byref(layer or _layer()), B_, T, a["parent"], a["leaf"], a["pos"],
                                   a["pos_out"], a["kv"], a["window"], a["pa"], a["fa"], a["ra"], a["pla"], cap_a,
                                   a["na"], a["nao"], a["pi"], a["fi"], a["ri"], a["pli"], cap_i, a["ni"], a["nio"],
                                   a["err"], None)
    for k in names:
        if k != "pli":  # without an index pool, its other arguments are not looked at
            assert call(**{k: None}) == B.CSA_ERR_ARG, k
        assert call(**{k: FAKE + 2}) == B.CSA_ERR_ARG, k
    assert call(cap_a=0) == B.CSA_ERR_ARG and call(cap_i=0) == B.CSA_ERR_ARG and call(T=65) == B.CSA_ERR_ARG
    assert call(layer=_layer(ratio=128)) == B.CSA_ERR_UNSUPPORTED


def test_workspace_sizes(lib):
    n = ctypes.c_size_t()
    for op in (B.OP_COMPRESS_TREE, B.OP_ATTEND_TREE):
        for bad in ((0, 8), (2, 0), (2, 65), (65536, 1), (65535, 64)):
            assert lib.csa_workspace_size(ctypes.byref(_layer()), op, *bad, 100, ctypes.byref(n)) == B.CSA_ERR_ARG
        assert lib.csa_workspace_size(ctypes.byref(_layer(dtype=B.CSA_F32)), op, 2, 64, 100, ctypes.byref(n)) == 0
        assert n.value > 0


# ------------------------------------------------------------------------------------------------ the binding

LAYER = csa.Layer(dtype=torch.bfloat16, H=64, D=512, R=64, W=128, ratio=4, Hi=64, Di=128, topk=512, X=64)


def z(*s, dt=torch.bfloat16):
    return torch.zeros(*s, dtype=dt)


def test_binding_names_the_wrong_tensor(lib):
    """CPU tensors: dtypes and shapes are refused first, by name, and the device last."""
    i32, f32 = torch.int32, torch.float32
    good = dict(q=z(2, 3, 64, 512), kv=z(2, 3, 512), sink=z(64, dt=f32), window=z(2, 128, 512), pool=z(2, 40, 512),
                rows_a=z(2, 3, 512), scores=z(2, 3, 43, dt=f32), parent=z(2, 3, dt=i32), n_rows=z(2, dt=i32),
                pos=z(2, dt=i32), inv_freq=z(32, dt=f32), out=z(2, 3, 64, 512))
    with pytest.raises(ValueError, match="CUDA"):
        csa.attend_tree(LAYER, **good)
    with pytest.raises(ValueError, match="q"):
        csa.attend_tree(LAYER, **{**good, "q": z(2, 3, 64, 256)})
    with pytest.raises(ValueError, match="pool"):
        csa.attend_tree(LAYER, **{**good, "q": _cuda_like(good["q"]), "pool": z(40, 512)})
    fake = {k: _cuda_like(t) for k, t in good.items()}
    for name in ("kv", "sink", "parent", "window", "rows_a", "scores", "n_rows", "pos", "inv_freq", "out"):
        wrong = torch.float64 if good[name].dtype != torch.float64 else f32
        with pytest.raises(TypeError, match=name):
            csa.attend_tree(LAYER, **{**fake, name: _cuda_like(good[name].to(wrong))})
        with pytest.raises(ValueError, match=name):
            csa.attend_tree(LAYER, **{**fake, name: _cuda_like(z(*good[name].shape, 1, dt=good[name].dtype))})
    with pytest.raises(ValueError, match="xs"):
        csa.norm_rope(LAYER, [z(2, 3)])
    with pytest.raises(TypeError, match="xs"):
        csa.norm_rope(LAYER, [z(2, 3, 64, 512, dt=f32)])
    with pytest.raises(ValueError, match="CUDA"):
        csa.norm_rope(LAYER, [z(2, 3, 64, 512)])
    with pytest.raises(ValueError, match="1 to 4"):
        csa.norm_rope(LAYER, [])
    with pytest.raises(ValueError, match="one entry"):
        csa.norm_rope(LAYER, [z(2, 3, 64, 512)], norm=[True, False])


def _cuda_like(t):
    """A CPU tensor that says it is on the GPU, for checks that come before any use of its address."""
    class Fake(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0
    return t.as_subclass(Fake)


def test_tree_helpers():
    """The test helpers themselves: paths, visible columns, selections (ties to the lower column, -0 equal to 0)."""
    assert TR.paths([-1, 0, 0, 1, -2]) == [[0], [0, 1], [0, 2], [0, 1, 3], None]
    layer = type("L", (), dict(ratio=4, topk=3))
    assert TR.columns(layer, [0, 1, 3], 6, 5) == [0, 2]  # one committed row, node 1's at position 7
    s = np.array([0.0, 5.0, -0.0, 5.0, 1.0])
    layer = type("L", (), dict(ratio=1, topk=3))
    assert TR.select(layer, s, [], 5, 0).tolist() == [1, 3, 4]
    assert TR.select(layer, np.array([0.0, -0.0, 0.0, -1.0]), [], 4, 0).tolist() == [0, 1, 2]


def test_packed_structures_are_the_c_layouts(lib):
    """The binding packs the C structures as bytes: sizes and fields are those of their ctypes declarations."""
    import struct
    assert struct.calcsize(B._COMP_FMT) == ctypes.sizeof(B._Comp)
    assert struct.calcsize(B._ROWS_FMT) == ctypes.sizeof(B._Rows)
    c = B._Comp.from_buffer_copy(struct.pack(B._COMP_FMT, 16, 32, 48, 64, 7))
    assert (c.wkv, c.wgate, c.ape, c.norm_w, c.d) == (16, 32, 48, 64, 7)
    r = B._Rows.from_buffer_copy(struct.pack(B._ROWS_FMT, 16, 32, 0, 5, 6, 1, 1 << 40))
    assert (r.x, r.out, r.weight, r.heads, r.dim, r.norm, r.x_stride) == (16, 32, None, 5, 6, 1, 1 << 40)
    assert LAYER._packed() == bytes(LAYER._c()) and LAYER._packed() is LAYER._packed()
    import dataclasses
    other = dataclasses.replace(LAYER, topk=7)
    assert other._packed() == bytes(other._c()) != LAYER._packed() and other != LAYER


@pytest.mark.parametrize("native", [True, False])
def test_checks_of_tensors(lib, native, monkeypatch):
    """The checks in C and those in Python: the same addresses, the same refusals (device -1: CPU tensors)."""
    if native and B._addresses is None:
        pytest.skip("the checks in C are not built here (no Python headers)")
    if not native:
        monkeypatch.setattr(B, "_addresses", None)
    t, v = z(2, 3, 4), z(5, dt=torch.int32)
    good = [("t", t, torch.bfloat16, (2, 3, 4)), ("v", v, torch.int32, (5,)), ("s", z(0, 7), torch.bfloat16, (0, 7))]
    assert B._ptrs(-1, *good)[:2] == [t.data_ptr(), v.data_ptr()] and B._ptrs(-1) == []
    for bad, error in ((("t", t, torch.float16, (2, 3, 4)), TypeError), (("t", None, torch.bfloat16, (2,)), ValueError),
                       (("t", t, torch.bfloat16, (2, 3, 5)), ValueError), (("t", t, torch.bfloat16, (2, 12)), ValueError),
                       (("t", t[:, :2], torch.bfloat16, (2, 2, 4)), ValueError), (("t", 5, torch.int32, ()), TypeError),
                       (("t", t.transpose(0, 1), torch.bfloat16, (3, 2, 4)), ValueError)):
        with pytest.raises(error, match="t"):
            B._ptrs(-1, good[1], bad)
    with pytest.raises(ValueError, match="t"):
        B._ptrs(0, good[0])


def test_checks_hold_no_references(lib):
    import sys
    if B._addresses is None:
        pytest.skip("the checks in C are not built here (no Python headers)")
    t = z(2, 3)
    spec, wrong = ("t", t, torch.bfloat16, (2, 3)), ("t", t, torch.bfloat16, (3, 2))
    before = [sys.getrefcount(x) for x in (t, spec, wrong, spec[3], torch.bfloat16)]
    for _ in range(1000):
        assert B._addresses(-1, spec, spec) == [t.data_ptr()] * 2
        assert B._addresses(-1, spec, wrong) is wrong
    after = [sys.getrefcount(x) for x in (t, spec, wrong, spec[3], torch.bfloat16)]
    assert after == before
    with pytest.raises(TypeError):
        B._addresses()
    with pytest.raises(TypeError):
        B._addresses(-1, ("t", t))
    with pytest.raises(TypeError):
        B._addresses("x", spec)


# ------------------------------------------------------------------------------------------------ tokens of norm_rope


@pytest.fixture
def calls(monkeypatch):
    """What the binding would hand to the library; nothing is launched."""
    got = []
    monkeypatch.setattr(B, "_tree_call", lambda fn, dev, stream, *args: got.append((fn, args)))
    return got


def _rows_of(args):
    return B._Rows.from_buffer_copy(args[1])


def _norm_rope(x):
    return csa.norm_rope(LAYER, [_cuda_like(x)], outs=[_cuda_like(z(*x.shape))], err=_cuda_like(z(1, dt=torch.int32)))


@pytest.mark.parametrize("shape, src", [
    ((2, 3, 8, 128), (1, 1, 8, 128)), ((1, 3, 8, 128), (1, 1, 8, 128)), ((4, 1, 8, 128), (1, 1, 8, 128)),
    ((4, 1, 128), (1, 1, 128)), ((1, 5, 128), (1, 1, 128)), ((2, 3, 128), (1, 1, 128)), ((2, 3, 8, 128), (2, 1, 8, 128)),
    ((2, 3, 8, 128), (1, 3, 8, 128))])
def test_norm_rope_refuses_broadcast_tokens(lib, calls, shape, src):
    """An expanded tensor holds fewer tokens than its shape says: a token stride of 0 must not be taken for 'dense'."""
    with pytest.raises(ValueError, match=r"xs\[0\]: strides"):
        _norm_rope(z(*src).expand(*shape))
    assert not calls


def test_norm_rope_refuses_overlapping_tokens(lib, calls):
    """Tokens one value or one head apart lie over one another."""
    buf = z(4096)
    for shape, strides in (((1, 3, 8, 128), (0, 128, 128, 1)), ((3, 1, 8, 128), (512, 512, 128, 1)),
                           ((1, 4, 128), (0, 8, 1)), ((2, 2, 8, 128), (1024, 512, 128, 1))):
        with pytest.raises(ValueError, match=r"xs\[0\]: strides"):
            _norm_rope(buf.as_strided(shape, strides))
    assert not calls


def test_norm_rope_takes_slices_of_wider_tensors(lib, calls):
    """What the call documents: heads contiguous, one real stride from token to token; a single token has none."""
    wide = z(2, 3, 1160)
    for x, stride in ((wide[..., :1024].unflatten(-1, (8, 128)), 1160), (wide[..., 1024:1152], 1160),
                      (wide[:1, :, :128], 1160), (wide[:, :1, :128], 3 * 1160), (wide[:1, :1, :128], 0),
                      (z(2, 3, 8, 128), 0)):
        _norm_rope(x)
        fn, args = calls.pop()
        row = _rows_of(args)
        assert fn == "csa_norm_rope" and row.x_stride == stride and row.x == x.data_ptr(), (x.shape, x.stride())


def test_norm_rope_returns_its_error_word(lib, calls, monkeypatch):
    """Without err= the call makes the word: it lives with the outputs, where the caller can read it."""
    monkeypatch.setattr(B, "_new", lambda device, stream, new, *size, dtype: _cuda_like(new(*size, dtype=dtype)))
    x = _cuda_like(z(2, 3, 8, 128))
    got = csa.norm_rope(LAYER, [x], outs=[_cuda_like(z(2, 3, 8, 128))])
    assert isinstance(got, list) and len(got) == 1
    assert got.err.dtype == torch.int32 and got.err.tolist() == [0] and calls[0][1][-1] == got.err.data_ptr()
    own = _cuda_like(z(1, dt=torch.int32))
    assert csa.norm_rope(LAYER, [x], outs=[x], err=own).err is own and calls[1][1][-1] == own.data_ptr()


def test_attend_tree_key_counts_fit(lib):
    """A node's keys are counted in 32 bits: capacity, nodes and window together are bounded."""
    def call(W, cap):
        return lib.csa_attend_tree(ctypes.byref(_layer(W=W)), FAKE, FAKE, FAKE, 2, 8, FAKE, FAKE, FAKE, cap, FAKE, FAKE, FAKE,
                                   FAKE, FAKE, FAKE, None, None, 0, FAKE, None)
    assert call(1 << 30, 1 << 30) == B.CSA_ERR_ARG and call(128, 2 ** 31 - 257 - 135) == B.CSA_ERR_ARG
    assert call(128, 2 ** 31 - 257 - 136) == B.CSA_ERR_WORKSPACE  # (sizes accepted, no workspace given)
