"""add_norm, append_pages and attend_pages without a GPU: what the binding and the C ABI refuse on the host, before anything
is enqueued, and that the binding's two ways of making a call hand the library the same."""
import ctypes
import os
import struct

import pytest
import torch

import deepseek_v4_compressed_csa_gb300 as csa
from deepseek_v4_compressed_csa_gb300 import _binding as B
from tests.test_tree_host import FAKE, _cuda_like, _layer, z

GAP = 1 << 32  # tensors far apart
I32, F32, U8, BF16 = torch.int32, torch.float32, torch.uint8, torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from deepseek_v4_compressed_csa_gb300 import build
        build.build()
    return csa.load_library()


# ------------------------------------------------------------------------------------------------ the C ABI


def _norm(lib, layer=None, N=4, X=4096, group=128, xs=0, rs=0, **over):
    a = dict(x=FAKE, residual=FAKE + GAP, weight=FAKE + 2 * GAP, out=FAKE + 3 * GAP, residual_out=FAKE + 4 * GAP,
             codes=FAKE + 5 * GAP, scales=FAKE + 6 * GAP)
    a.update(over)
    return lib.csa_add_norm(ctypes.byref(layer or _layer()), a["x"], xs, a["residual"], rs, a["weight"], N, X, a["out"],
                            a["residual_out"], a["codes"], a["scales"], group, None)


def test_add_norm_refusals(lib):
    for bad in (dict(N=-1), dict(N=1 << 31), dict(X=0), dict(X=4), dict(X=4100), dict(X=16392), dict(group=0), dict(group=4),
                dict(group=96), dict(group=512), dict(X=264, group=16), dict(xs=4088), dict(xs=4100), dict(xs=-4096),
                dict(rs=4088), dict(rs=4100), dict(rs=(1 << 31) + 8), dict(x=None), dict(x=FAKE + 8), dict(residual=FAKE + 8),
                dict(weight=FAKE + 4), dict(out=FAKE + 3 * GAP + 8), dict(residual_out=FAKE + 4 * GAP + 2), dict(codes=None),
                dict(scales=None), dict(codes=FAKE + 5 * GAP + 8), dict(scales=FAKE + 6 * GAP + 2),
                dict(out=None, residual_out=None, codes=None, scales=None), dict(layer=_layer(D=4))):
        assert _norm(lib, **bad) == B.CSA_ERR_ARG, bad
    # no rows: nothing to do, whatever the addresses
    assert _norm(lib, N=0, x=None, out=None, residual=None, codes=None, scales=None) == 0
    assert _norm(lib, N=0, X=4100) == B.CSA_ERR_ARG


def test_add_norm_overlaps(lib):
    """An output may be a dense input itself, and lie over nothing else."""
    row = 4096 * 2
    for bad in (dict(out=FAKE + 16), dict(out=FAKE + 3 * row), dict(out=FAKE - 3 * row - 16), dict(residual_out=FAKE + GAP + 16),
                dict(codes=FAKE), dict(scales=FAKE + GAP + 4), dict(out=FAKE, xs=4104), dict(residual_out=FAKE + GAP, rs=8192),
                dict(out=FAKE, residual_out=FAKE), dict(residual_out=FAKE + 3 * GAP + 64), dict(codes=FAKE + 3 * GAP),
                dict(scales=FAKE + 5 * GAP + 4096), dict(weight=FAKE + 3 * GAP), dict(out=FAKE + 2 * GAP + 4 * 4096 - 16),
                dict(xs=1 << 20, out=FAKE + (3 << 21))):
        assert _norm(lib, **bad) == B.CSA_ERR_ARG, bad


def _pages(n=10, rows=64, codes=FAKE + 8 * GAP, scales=FAKE + 9 * GAP):
    return struct.pack(B._PAGES_FMT, codes or 0, scales or 0, n, rows)


POOLS = (dict(n=0), dict(rows=0), dict(n=-1), dict(n=1 << 20, rows=2048), dict(n=2 ** 31 - 256, rows=1), dict(codes=None),
         dict(scales=None), dict(codes=FAKE + 8), dict(scales=FAKE + 2))


def _append(lib, layer=None, pages=_pages(), B_=2, T=3, width=5, sb=0, st=0, norm=1, **over):
    a = dict(rows=FAKE, table=FAKE + GAP, pos=FAKE + 2 * GAP, n_new=FAKE + 3 * GAP, weight=FAKE + 4 * GAP, invf=FAKE + 5 * GAP,
             err=FAKE + 6 * GAP)
    a.update(over)
    return lib.csa_append_pages(ctypes.byref(layer or _layer()), pages, a["rows"], sb, st, B_, T, a["table"], width, a["pos"],
                                a["n_new"], a["weight"], norm, a["invf"], a["err"], None)


def test_append_pages_refusals(lib):
    for bad in POOLS:
        assert _append(lib, pages=_pages(**bad)) == B.CSA_ERR_ARG, bad
    for bad in (dict(pages=None), dict(B_=0), dict(T=0), dict(B_=1 << 12, T=(1 << 12) + 1), dict(width=0), dict(width=-1),
                dict(width=(1 << 24) + 1), dict(norm=2), dict(norm=-1), dict(rows=None), dict(rows=FAKE + 8), dict(table=None),
                dict(table=FAKE + 2), dict(pos=None), dict(pos=FAKE + 1), dict(n_new=FAKE + 2), dict(weight=FAKE + 4),
                dict(invf=FAKE + 4), dict(err=None), dict(err=FAKE + 2), dict(st=504), dict(st=516), dict(st=-512),
                dict(sb=4), dict(sb=-8), dict(sb=(1 << 40) + 8), dict(layer=_layer(R=60))):
        assert _append(lib, **bad) == B.CSA_ERR_ARG, bad


def _attend(lib, layer=None, pages=_pages(), B_=2, T=3, tw=5, first=4, rw=6, ws=FAKE + 15 * GAP, ws_bytes=1 << 34, **over):
    a = {k: FAKE + i * GAP for i, k in enumerate(("q", "sink", "pos", "n_new", "tok", "row", "n_rows", "sel", "x", "y", "n_sel",
                                                  "invf", "out", "err"))}
    a.update(over)
    return lib.csa_attend_pages(ctypes.byref(layer or _layer()), pages, a["q"], B_, T, a["sink"], a["pos"], a["n_new"],
                                a["tok"], tw, first, a["row"], rw, a["n_rows"], a["sel"], a["n_sel"], a["invf"], a["out"], ws,
                                ws_bytes, a["err"], None)


def test_attend_pages_refusals(lib):
    for bad in POOLS:
        assert _attend(lib, pages=_pages(**bad)) == B.CSA_ERR_ARG, bad
    for k in ("q", "pos", "out", "err", "n_rows", "n_sel"):
        assert _attend(lib, **{k: None}) == B.CSA_ERR_ARG, k
    for k in ("q", "sink", "pos", "n_new", "tok", "row", "n_rows", "sel", "n_sel", "invf", "out", "err"):
        assert _attend(lib, **{k: FAKE + 2}) == B.CSA_ERR_ARG, k
    for k in ("q", "invf", "out"):  # rows that are read 16 bytes at a time
        assert _attend(lib, **{k: FAKE + 40 * GAP + 8}) == B.CSA_ERR_ARG, k
    for bad in (dict(pages=None), dict(B_=0), dict(T=0), dict(B_=257, T=256), dict(first=-1), dict(tw=0), dict(rw=0),
                dict(tw=(1 << 24) + 1), dict(rw=(1 << 24) + 1), dict(tok=None, row=None), dict(row=None),
                dict(layer=_layer(ratio=128)), dict(layer=_layer(R=60)),
                # queries and outputs over one another: 6 x 64 x 512 x 2 bytes
                dict(out=FAKE), dict(out=FAKE + 6 * 65536 - 16), dict(q=FAKE + 12 * GAP + 5 * 65536)):
        assert _attend(lib, **bad) == B.CSA_ERR_ARG, bad
    # tables that could hold more tiles than an int counts: 2^14 queries of 2^24 pages of 64 rows each
    wide = dict(B_=1 << 7, T=1 << 7, rw=1 << 24, sel=None, n_sel=None)
    assert _attend(lib, **wide) == B.CSA_ERR_ARG
    assert _attend(lib, B_=1 << 7, T=1 << 7, tw=1 << 24) == B.CSA_ERR_ARG
    # ... or one query more keys than an int counts
    assert _attend(lib, B_=1, T=1, tw=1 << 24, rw=1 << 24, sel=None, n_sel=None) == B.CSA_ERR_ARG
    for ws in (dict(ws=None), dict(ws=FAKE + 8), dict(ws_bytes=0)):
        assert _attend(lib, **ws) == B.CSA_ERR_WORKSPACE, ws


def test_workspace_of_attend_pages(lib):
    """Enough for two parts a block and the table of queries; one byte less is refused, also in the smallest call."""
    n = ctypes.c_size_t()
    for layer in (_layer(), _layer(dtype=B.CSA_F32, H=5, D=72, R=24, W=9, Hi=3, Di=40, topk=7, X=64)):
        sizes = []
        for b, t in ((1, 1), (3, 5), (1 << 8, 1 << 8)):
            assert lib.csa_workspace_size(ctypes.byref(layer), B.OP_ATTEND_PAGES, b, t, 1, ctypes.byref(n)) == 0
            assert n.value >= 2 * 152 * layer.H * (4 * layer.D + 8) + 8 * b * t
            sizes.append(n.value)
            assert _attend(lib, layer=layer, B_=b, T=t, ws_bytes=n.value - 1, out=FAKE + 80 * GAP) == B.CSA_ERR_WORKSPACE
        assert sizes == sorted(sizes)
    for b, t in ((0, 1), (1, 0), (257, 256), (-1, 1)):
        assert lib.csa_workspace_size(ctypes.byref(_layer()), B.OP_ATTEND_PAGES, b, t, 1, ctypes.byref(n)) == B.CSA_ERR_ARG


# ------------------------------------------------------------------------------------------------ the binding

LAYER = csa.Layer(dtype=BF16, H=64, D=512, R=64, W=128, ratio=4, Hi=64, Di=128, topk=512, X=4096)


def _good(which):
    if which == "add_norm":
        return dict(x=z(3, 2, 256), residual=z(3, 2, 256), weight=z(256, dt=F32), out=z(3, 2, 256), residual_out=z(3, 2, 256),
                    codes=z(3, 2, 256, dt=U8), scales=z(3, 2, 8, dt=F32)), dict(group=32)
    if which == "append_pages":
        return dict(rows=z(2, 3, 512), codes=z(5, 16, 512, dt=U8), scales=z(5, 16, dt=F32), table=z(2, 4, dt=I32),
                    pos=z(2, dt=I32), n_new=z(2, dt=I32), weight=z(512, dt=F32), inv_freq=z(32, dt=F32), err=z(1, dt=I32)), dict(norm=True)
    return dict(q=z(2, 3, 64, 512), codes=z(5, 16, 512, dt=U8), scales=z(5, 16, dt=F32), sink=z(64, dt=F32), pos=z(2, dt=I32),
                out=z(2, 3, 64, 512), token_table=z(2, 4, dt=I32), row_table=z(2, 7, dt=I32), n_rows=z(2, dt=I32),
                sel=z(2, 3, 512, dt=I32), n_sel=z(2, 3, dt=I32), n_new=z(2, dt=I32), inv_freq=z(32, dt=F32),
                ws=z(1 << 10, dt=U8), err=z(1, dt=I32)), dict(first=4)


def _run(which, tensors, rest, fake=True):
    t = {k: _cuda_like(v) if fake and isinstance(v, torch.Tensor) else v for k, v in tensors.items()}
    if which != "add_norm":
        t["pages"] = csa.Pages(t.pop("codes"), t.pop("scales"))
    return getattr(csa, which)(LAYER, **t, **rest)


@pytest.fixture
def calls(monkeypatch):
    """What the binding would hand to the library; nothing is launched (nor by the calls made in C, where a GPU is)."""
    got = []
    monkeypatch.setattr(B, "_plain", None)
    monkeypatch.setattr(B, "_tree_call", lambda fn, dev, stream, *args: got.append((fn, args)))
    return got


@pytest.mark.parametrize("which", ["add_norm", "append_pages", "attend_pages"])
def test_binding_names_the_wrong_tensor(lib, calls, which):
    tensors, rest = _good(which)
    _run(which, tensors, rest)
    assert calls.pop()[0] == "csa_" + which
    with pytest.raises(ValueError, match="CUDA"):
        _run(which, tensors, rest, fake=False)
    for name, t in tensors.items():
        if name != "ws":  # (of any type: its bytes count)
            with pytest.raises((TypeError, ValueError), match=name):
                _run(which, {**tensors, name: t.to(torch.float64)}, rest)
        if name not in ("ws", "err"):
            if (which, name) != ("add_norm", "x"):
                with pytest.raises(ValueError, match=name):
                    _run(which, {**tensors, name: z(*t.shape, 1, dt=t.dtype)}, rest)
            if name not in ("table", "token_table", "row_table", "codes") or which == "add_norm":
                short = z(*(n - 1 if n > 1 else n for n in t.shape), dt=t.dtype)
                with pytest.raises(ValueError):
                    _run(which, {**tensors, name: short}, rest)
        if name not in ("x", "residual", "rows", "weight", "pos", "n_new", "n_rows", "sink", "inv_freq", "ws", "err"):
            with pytest.raises(ValueError, match=name):  # every other value of a wider tensor
                _run(which, {**tensors, name: t.repeat_interleave(2, -1)[..., ::2]}, rest)
        with pytest.raises((TypeError, ValueError)):
            _run(which, {**tensors, name: "no tensor"}, rest)
    assert not calls


def test_binding_refuses_what_does_not_fit_together(lib, calls):
    tensors, rest = _good("add_norm")
    for bad, more in ((dict(residual=None), {}), (dict(), dict(group=None)), (dict(), dict(group=96)), (dict(), dict(group=0))):
        with pytest.raises(ValueError):
            _run("add_norm", {**tensors, **bad}, {**rest, **more})
    wide = z(3, 5, 256)
    for x in (wide[:, 1:3], z(2, 3, 256).transpose(0, 1), z(1, 1, 256).expand(3, 2, 256), z(3, 1, 256).expand(3, 2, 256),
              z(600).as_strided((3, 2, 256), (16, 8, 1))):  # rows more than one stride apart, or over one another
        with pytest.raises(ValueError, match="strides"):
            _run("add_norm", {**tensors, "x": x}, rest)
    tensors, rest = _good("append_pages")
    with pytest.raises(ValueError, match="norm"):
        _run("append_pages", tensors, dict(norm=False))
    for rows in (z(1, 3, 512).expand(2, 3, 512), z(2, 1, 512).expand(2, 3, 512), z(2, 3, 1024)[..., ::2],
                 z(4096).as_strided((2, 3, 512), (1536, 256, 1))):
        with pytest.raises(ValueError, match="strides"):
            _run("append_pages", {**tensors, "rows": rows}, rest)
    tensors, rest = _good("attend_pages")
    for bad in (dict(token_table=None, row_table=None, n_rows=None, sel=None, n_sel=None), dict(row_table=None), dict(n_rows=None),
                dict(n_sel=None), dict(sel=None)):
        with pytest.raises(ValueError):
            _run("attend_pages", {**tensors, **bad}, rest)
    assert not calls


def test_binding_refuses_what_an_int_does_not_hold(lib, calls):
    """Sizes and counts that the C ABI's ints would cut off (tensors that are one value, expanded)."""
    tensors, rest = _good("add_norm")
    with pytest.raises(ValueError, match="16384"):
        _run("add_norm", dict(x=z(1, 1).expand(1, (1 << 32) + 8)), {})
    tensors, rest = _good("append_pages")
    with pytest.raises(ValueError, match="2.24"):
        _run("append_pages", {**tensors, "rows": z(1, 512).expand(1 << 25, 1, 512)}, rest)
    with pytest.raises(ValueError, match="table"):
        _run("append_pages", {**tensors, "table": z(2, 1, dt=I32).expand(2, (1 << 32) + 4)}, rest)
    tensors, rest = _good("attend_pages")
    for first in (-1, 1 << 31, (1 << 32) + 4):
        with pytest.raises(ValueError, match="first"):
            _run("attend_pages", tensors, dict(first=first))
    with pytest.raises(ValueError, match="2.16"):
        _run("attend_pages", {**tensors, "q": z(64, 512).expand(1 << 17, 1, 64, 512)}, rest)
    assert not calls


def test_binding_passes_strides(lib, calls):
    tensors, rest = _good("add_norm")
    wide = z(6, 512 + 8)
    _run("add_norm", {**tensors, "x": wide[:, 8:264].unflatten(0, (3, 2)), "residual": wide.view(6, 520)[:, :256].unflatten(0, (3, 2))}, rest)
    args = calls.pop()[1]
    assert args[1:5] == (wide[:, 8:].data_ptr(), 520, wide.data_ptr(), 520) and args[6:8] == (6, 256)
    tensors, rest = _good("append_pages")
    wide = z(2, 5, 2048)
    for rows, strides in ((wide[:, 1:4, 512:1024], (5 * 2048, 2048)), (wide[:, :3, :512], (5 * 2048, 2048)),
                          (wide[:, :1, :512], (5 * 2048, 0)), (wide[:1, :3, :512], (0, 2048)), (z(2, 3, 512), (0, 0))):
        few = dict(tensors, rows=rows, table=z(rows.shape[0], 4, dt=I32), pos=z(rows.shape[0], dt=I32), n_new=None)
        _run("append_pages", few, rest)
        args = calls.pop()[1]
        assert args[2:7] == (rows.data_ptr(), *strides, *rows.shape[:2]), rows.shape


FORMS = {
    "add_norm": [{}, dict(residual=None, residual_out=None), dict(weight=None), dict(out=False), dict(residual_out=False),
                 dict(group=None, codes=None, scales=None), dict(group=256, scales=z(3, 2, 1, dt=F32))],
    "append_pages": [{}, dict(n_new=None), dict(weight=None), dict(norm=False, weight=None), dict(inv_freq=None)],
    "attend_pages": [{}, dict(sink=None), dict(n_new=None), dict(inv_freq=None), dict(token_table=None), dict(sel=None, n_sel=None),
                     dict(row_table=None, n_rows=None, sel=None, n_sel=None), dict(first=0)],
}


@pytest.mark.parametrize("which", list(FORMS))
def test_both_ways_of_a_call_hand_over_the_same(lib, which, monkeypatch):
    """Calls made whole in C, and by the binding's own code: the same arguments to the library."""
    if B._plain is None:
        pytest.skip("the checks in C are not built here (no Python headers)")
    holds = ((0, len(LAYER._packed())), (1, struct.calcsize(B._PAGES_FMT)))[: 1 if which == "add_norm" else 2]
    got, contents = [], []

    def record(*args):  # addresses as the library would see them; structures by what they hold
        contents.append([ctypes.string_at(args[i], n) for i, n in holds])
        got.append(args)
        return 0

    stub = ctypes.CFUNCTYPE(ctypes.c_int, *getattr(lib, "csa_" + which).argtypes)(record)
    monkeypatch.setitem(B._at, which, ctypes.cast(stub, ctypes.c_void_p).value)
    real = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    tensors, rest = _good(which)
    try:
        B._plain.setup(F32, U8, I32, lambda dev: 4242 + dev, lambda: 0)
        for form in FORMS[which]:
            both = {**tensors, **rest, **form}
            t = {k: v for k, v in both.items() if k not in ("group", "norm", "first")}
            r = {k: v for k, v in both.items() if k in ("group", "norm", "first")}
            _run(which, t, r)
            in_c = got.pop()
            packed = contents.pop()
            assert not got
            made = []
            with monkeypatch.context() as m:
                m.setattr(B, "_plain", None)
                m.setattr(B, "_tree_call", lambda name, dev, stream, *args: made.append(args))
                _run(which, t, r)
            own = made.pop()
            assert [own[i] for i, _ in holds] == packed, form
            n = len(holds)
            assert [a or 0 for a in in_c[n:-1]] == [a or 0 for a in own[n:]] and in_c[-1] == 4242, form
    finally:
        B._plain.setup(F32, U8, I32, *real)


def test_calls_in_c_hold_no_references(lib, monkeypatch):
    import sys
    if B._plain is None:
        pytest.skip("the checks in C are not built here (no Python headers)")
    real = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    stubs = []
    try:
        B._plain.setup(F32, U8, I32, lambda dev: 1, lambda: 0)
        for which in FORMS:
            fn = getattr(lib, "csa_" + which)
            stubs.append(ctypes.CFUNCTYPE(ctypes.c_int, *fn.argtypes)(lambda *a: 0))
            monkeypatch.setitem(B._at, which, ctypes.cast(stubs[-1], ctypes.c_void_p).value)
            tensors, rest = _good(which)
            fake = {k: _cuda_like(v) for k, v in tensors.items()}
            if which != "add_norm":
                fake["pages"] = csa.Pages(fake.pop("codes"), fake.pop("scales"))
            watch = [*[v for v in fake.values()], F32, U8, I32, BF16, LAYER._packed()]
            call = getattr(csa, which)
            call(LAYER, **fake, **rest)
            before = [sys.getrefcount(x) for x in watch]
            for _ in range(300):
                call(LAYER, **fake, **rest)
            assert [sys.getrefcount(x) for x in watch] == before, which
    finally:
        B._plain.setup(F32, U8, I32, *real)


def test_packed_pages_are_the_c_layout():
    class C(ctypes.Structure):
        _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("n", ctypes.c_int), ("rows", ctypes.c_int)]
    c = C.from_buffer_copy(_pages(n=7, rows=9))
    assert (c.codes, c.scales, c.n, c.rows) == (FAKE + 8 * GAP, FAKE + 9 * GAP, 7, 9)
