"""append_pages and attend_pages: what they write may lie over nothing that they read, nor over what else they write."""
import pytest
import torch

import deepseek_v4_compressed_csa_gb300 as csa
from deepseek_v4_compressed_csa_gb300 import _binding as B
from tests.test_pages_host import FAKE, GAP, _append, _attend, _norm, _pages, lib  # noqa: F401 (lib: a fixture)

ROWS, D = 10 * 64, 512  # of the pool that _pages describes
CODES, SCALES = FAKE + 8 * GAP, FAKE + 9 * GAP
APPEND = dict(rows=6 * D * 2, table=2 * 5 * 4, pos=8, n_new=8, weight=D * 4, invf=64 * 2)
ATTEND = dict(q=6 * 64 * D * 2, sink=64 * 4, pos=8, n_new=8, tok=2 * 5 * 4, row=2 * 6 * 4, n_rows=8, sel=6 * 512 * 4, n_sel=6 * 4,
              invf=64 * 2)


def over(at, size, of):
    """Addresses of a tensor of `of` bytes (a multiple of 16 apart) that just meet [at, at + size): its last and first 16 bytes,
    and itself."""
    return {at, at + (size - 1) // 16 * 16, at - (of - 1) // 16 * 16}


def test_append_pages(lib):  # noqa: F811
    for name, size in APPEND.items():
        for at in over(CODES, ROWS * D, size) | over(SCALES, ROWS * 4, size):
            assert _append(lib, **{name: at}) == B.CSA_ERR_ARG, (name, at - CODES)
    here = dict(zip(("rows", "table", "pos", "n_new", "weight", "invf"), (FAKE + i * GAP for i in range(6))))
    for name, size in APPEND.items():
        assert _append(lib, err=here[name] + (size - 1) // 4 * 4) == B.CSA_ERR_ARG, name
    # rows strides apart, up to the last one's end
    assert _append(lib, sb=1 << 20, st=1 << 16, rows=CODES - 2 * ((1 << 20) + 2 * (1 << 16)) - D * 2 + 16) == B.CSA_ERR_ARG
    assert _append(lib, pages=_pages(scales=CODES + ROWS * D - 4)) == B.CSA_ERR_ARG
    assert _append(lib, err=CODES + 64) == B.CSA_ERR_ARG and _append(lib, err=SCALES + ROWS * 4 - 4) == B.CSA_ERR_ARG


def test_attend_pages(lib):  # noqa: F811
    names = ("q", "sink", "pos", "n_new", "tok", "row", "n_rows", "sel", "x", "y", "n_sel", "invf", "out", "err")
    here = {k: FAKE + i * GAP for i, k in enumerate(names)}
    sizes = dict(ATTEND, codes=ROWS * D, scales=ROWS * 4)
    here |= dict(codes=CODES, scales=SCALES)
    out, ws = ATTEND["q"], 2 * 152 * 64 * (4 * D + 8)  # (the least that the workspace takes)
    for name, size in sizes.items():
        for at in over(here[name], size, out):
            assert _attend(lib, out=at) == B.CSA_ERR_ARG, (name, at - here[name])
        for at in over(here[name], size, ws):
            assert _attend(lib, ws=at) == B.CSA_ERR_ARG, (name, at - here[name])
        assert _attend(lib, err=here[name] + (size - 1) // 4 * 4) == B.CSA_ERR_ARG, name
    for at in over(here["out"], out, ws):
        assert _attend(lib, ws=at) == B.CSA_ERR_ARG
    assert _attend(lib, err=here["out"] + out - 4) == B.CSA_ERR_ARG and _attend(lib, err=FAKE + 15 * GAP + ws - 4) == B.CSA_ERR_ARG


def test_strides_past_the_address_space(lib):  # noqa: F811
    """Rows whose strides span more than an address counts: refused, not compared by a span that wrapped."""
    assert _append(lib, B_=1 << 24, T=1, sb=1 << 40) == B.CSA_ERR_ARG
    assert _append(lib, B_=1 << 20, T=16, sb=(1 << 36) + 8) == B.CSA_ERR_ARG
    assert _norm(lib, N=(1 << 31) - 1, xs=1 << 31) == B.CSA_ERR_ARG and _norm(lib, N=(1 << 31) - 1, rs=1 << 31) == B.CSA_ERR_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("small", [False, True])
def test_neighbours_are_no_overlap(small):
    """Every tensor of both calls behind the other in one buffer, with nothing in between: taken, and the same results."""
    from tests import _pages as P
    from tests.test_gpu_pages import build, call, i32, normal, gen
    L = P.layer(small)
    cache, q, out, h, host = build(L, 3, 2, [2000, 40, 700], 16, "select", 3, [2, 2, 2], seed=9)
    assert call(L, cache, q, out, h, host).item() == 0
    x, w = normal(gen(1), 3, 2, L.D, dtype=L.dtype), 1 + 0.1 * normal(gen(2), L.D)
    codes, scales = cache.codes.clone(), cache.scales.clone()
    assert csa.append_pages(L, x, csa.Pages(codes, scales), host["token_table"].cuda(), i32(h["pos"]), weight=w, norm=True,
                            inv_freq=host["freq"]).item() == 0
    size = csa.workspace_size(L, csa.OP_ATTEND_PAGES, 3, 2, 1)
    t = dict(codes=cache.codes, out=torch.full_like(out, 7.0), q=q, scales=cache.scales, sink=host["sink"], pos=i32(h["pos"]),
             tok=host["token_table"], ws=torch.zeros(size, dtype=torch.uint8), row=host["row_table"], n_rows=i32(host["n_rows"]),
             sel=host["sel"], n_sel=host["n_sel"], err=torch.zeros(1, dtype=torch.int32), freq=host["freq"], w=w, x=x)
    slab = torch.empty(sum(-(-v.numel() * v.element_size() // 16) * 16 for v in t.values()), dtype=torch.uint8, device="cuda")
    at = 0
    for k, v in t.items():  # (each starts on 16 bytes: the next one behind its last)
        n = v.numel() * v.element_size()
        t[k] = slab[at : at + n].view(v.dtype).view(v.shape)
        t[k].copy_(v)
        at += -(-n // 16) * 16
    pages = csa.Pages(t["codes"], t["scales"])
    csa.attend_pages(L, t["q"], pages, t["sink"], t["pos"], t["out"], token_table=t["tok"], first=3, row_table=t["row"],
                     n_rows=t["n_rows"], sel=t["sel"], n_sel=t["n_sel"], inv_freq=t["freq"], ws=t["ws"], err=t["err"])
    assert t["err"].item() == 0 and torch.equal(t["out"], out)
    csa.append_pages(L, t["x"], pages, t["tok"], t["pos"], weight=t["w"], norm=True, inv_freq=t["freq"], err=t["err"])
    assert t["err"].item() == 0 and torch.equal(t["codes"], codes)
    assert torch.equal(t["scales"].view(torch.int32), scales.view(torch.int32))
