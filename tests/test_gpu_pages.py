"""add_norm, append_pages and attend_pages on the GPU, each against its definition in 64 bits, and as they are used."""
import math

import pytest
import torch

import deepseek_v4_compressed_csa_gb300 as csa
from tests import _pages as P

pytestmark = pytest.mark.gpu
F64, U32 = P.F64, P.U32


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------------------------------- add_norm


def norm_ref(L, x, r, w):
    """(h, y, error of y): the square sum of X terms by a tree of about 16 + 9 roundings, the root and three products."""
    h = x.to(F64) + (0 if r is None else r.to(F64))
    y = h / (h.pow(2).mean(-1, keepdim=True) + L.rms_eps).sqrt()
    y = y if w is None else y * w.to(F64)
    return h, y, y.abs() * 64 * U32


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("N,X,group", [(1, 4096, 128), (3, 8, 8), (7, 128, 32), (5, 248, 8), (9, 256, 256), (2, 264, 264),
                                       (33, 512, 64), (2, 520, 8), (4, 1024, 1024), (3, 4104, 8), (5, 7168, 128), (2, 8192, 256),
                                       (3, 16384, 16), (2, 16384, 16384), (1030, 4096, 128)])
def test_add_norm(small, N, X, group):
    L = P.layer(small)
    g = gen(N * X)
    x, r, w = normal(g, N, X, dtype=L.dtype), normal(g, N, X, scale=4.0, dtype=L.dtype), 1 + 0.1 * normal(g, X)
    out, res, codes, scales = csa.add_norm(L, x, r, w, group=group)
    h, y, err = norm_ref(L, x, r, w)
    half = P.HALF[L.dtype]
    P.check(res, h, h.abs() * (half + U32), "residual")
    P.check(out, y, err + y.abs() * half, "out")
    P.check_codes(codes.view(N, -1, group), scales, y.view(N, -1, group), err.view(N, -1, group))


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("X", [128, 4096])
def test_add_norm_forms(small, X):
    """Without a residual, a weight, an output; in place; rows a stride apart; leading dimensions."""
    L = P.layer(small)
    g = gen(5)
    x, r, w = normal(g, 2, 3, X, dtype=L.dtype), normal(g, 2, 3, X, dtype=L.dtype), 1 + 0.1 * normal(g, X)
    full = csa.add_norm(L, x, r, w, group=32)
    assert full.out.shape == x.shape and full.scales.shape == (2, 3, X // 32)
    plain = csa.add_norm(L, x)
    assert plain.residual is None and plain.codes is None and plain.scales is None
    _, y, err = norm_ref(L, x, None, None)
    P.check(plain.out, y, err + y.abs() * P.HALF[L.dtype])
    only = csa.add_norm(L, x, r, w, group=32, out=False, residual_out=False)
    assert only.out is None and only.residual is None
    assert torch.equal(only.codes, full.codes) and torch.equal(only.scales, full.scales)
    for target in ("x", "r"):
        a, b = x.clone(), r.clone()
        got = csa.add_norm(L, a, b, w, group=32, residual_out=a if target == "x" else b)
        assert got.residual is (a if target == "x" else b)
        assert torch.equal(got.residual, full.residual) and torch.equal(got.out, full.out)
        assert torch.equal(a if target == "r" else b, x if target == "r" else r)
    a = x.clone()
    got = csa.add_norm(L, a, r, w, out=a)
    assert got.out is a and torch.equal(a, full.out) and torch.equal(got.residual, full.residual)
    wide, wide_r = normal(g, 6, 2 * X + 8, dtype=L.dtype), normal(g, 6, X + 16, dtype=L.dtype)
    xs, rs = wide[:, 8:X + 8], wide_r[:, :X]
    got = csa.add_norm(L, xs, rs, w, group=64)
    want = csa.add_norm(L, xs.contiguous(), rs.contiguous(), w, group=64)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    empty = csa.add_norm(L, x[:0], r[:0], w, group=32)
    assert empty.out.shape == (0, 3, X)


def test_add_norm_odd_values():
    """Rows of zeros, a NaN, an infinity, values near the type's ends; a group of zeros beside others."""
    L = P.layer()
    g = gen(8)
    x = normal(g, 8, 512, dtype=L.dtype)
    x[0] = 0
    x[1, 5] = math.nan
    x[2, 300] = math.inf
    x[3] *= 1e-20
    x[4] *= 2.0 ** 60
    x[5, 64:128] = 0
    x[6] = 1e-38
    out, _, codes, scales = csa.add_norm(L, x, group=64)
    v = codes.view(P.F8).float() * scales.repeat_interleave(64, -1)
    assert (out[0] == 0).all() and (scales[0] == 0).all() and (codes[0] == 0).all()
    assert torch.isnan(out[1]).all() and torch.isnan(scales[1]).all() and torch.isnan(v[1]).all()
    # an infinity: its own value inf * 0 is NaN, the others are 0
    assert torch.isnan(out[2, 300]) and (out[2, :300] == 0).all() and torch.isnan(scales[2, 4]) and (scales[2, :4] == 0).all()
    assert (scales[5, 1] == 0) and (codes[5, 64:128] == 0).all()
    fine = [3, 4, 5, 6, 7]
    _, y, err = norm_ref(L, x[fine], None, None)
    P.check(out[fine], y, err + y.abs() * P.HALF[L.dtype] + 2.0 ** -133)
    P.check_codes(codes[fine].view(5, 8, 64), scales[fine], y.view(5, 8, 64), err.view(5, 8, 64))


# ---------------------------------------------------------------------------------------------------- append_pages


def append_ref(L, x, pos, freq, w, norm):
    """(y, error) of rows [n, D] at positions pos [n]."""
    y = x.to(F64)
    if norm:
        y = y / (y.pow(2).mean(-1, keepdim=True) + L.rms_eps).sqrt()
        y = y if w is None else y * w.to(F64)
    err = y.abs() * (64 * U32 if norm else 0)
    if freq is not None:  # sines and cosines within 2 units, two products and a sum
        err = P.pair_sum(err + 8 * U32 * y.abs(), L.R)
        y = P.turn(y, pos, freq, 1.0)
    return y, err


@pytest.mark.parametrize("kw", [dict(small=False), dict(small=True), dict(small=True, D=8, R=8, Di=8), dict(small=True, D=1024, R=128, Di=128),
                                dict(small=False, D=264, R=8, Di=128), dict(small=False, D=1024, R=1024, Di=1024)])
@pytest.mark.parametrize("B,T,page,pos", [(1, 1, 64, [0]), (3, 5, 16, [0, 13, 100]), (2, 130, 8, [63, 1]), (4, 3, 7, [5, 6, 7, 20])])
def test_append_pages(kw, B, T, page, pos):
    L = P.layer(**kw)
    freq, g = P.inv_freq(L), gen(B * T + page)
    for norm, weighted, rotated, counts in ((1, True, True, None), (1, False, False, [T - b % (T + 1) for b in range(B)]),
                                            (0, False, True, [max(0, T - 2 * b) for b in range(B)])):
        x, w = normal(g, B, T, L.D, scale=3.0, dtype=L.dtype), 1 + 0.1 * normal(g, L.D)
        cache = P.Cache(L, page, sum(-(-(p + T) // page) for p in pos) + 3, seed=T)
        width = max(-(-(p + T) // page) for p in pos)
        table = cache.table(B, width)
        n = counts or [T] * B
        at = [cache.place(table, b, range(pos[b], pos[b] + n[b])) for b in range(B)]
        before = (cache.codes.clone(), cache.scales.clone())
        err = csa.append_pages(L, x, cache.pages, table.cuda(), i32(pos), n_new=None if counts is None else i32(counts),
                               weight=w if weighted else None, norm=bool(norm), inv_freq=freq if rotated else None)
        assert err.item() == 0
        touched = torch.zeros(cache.n * page, dtype=torch.bool, device="cuda")
        for b in range(B):
            if not n[b]:
                continue
            rows = torch.tensor(at[b], device="cuda")
            touched[rows] = True
            y, e = append_ref(L, x[b, : n[b]], pos[b] + torch.arange(n[b], device="cuda"), freq if rotated else None,
                              w if weighted else None, norm)
            P.check_codes(cache.codes.view(-1, L.D)[rows], cache.scales.view(-1)[rows], y, e, f"b{b}")
        # every other row is as it was
        assert torch.equal(cache.codes.view(-1, L.D)[~touched], before[0].view(-1, L.D)[~touched])
        assert torch.equal(cache.scales.view(-1)[~touched].view(torch.int32), before[1].view(-1)[~touched].view(torch.int32))


def test_append_pages_strides_and_odd_values():
    L = P.layer()
    freq, g = P.inv_freq(L), gen(3)
    wide = normal(g, 3, 7, 3 * 512, dtype=L.dtype)
    x = wide[:, 1:5, 512:1024]
    pos = [0, 30, 64]
    outs = []
    for rows in (x, x.contiguous(), x[:, :1], x[:, :1].contiguous()):
        cache = P.Cache(L, 16, 40)
        table = cache.table(3, 8)
        for b in range(3):
            cache.place(table, b, range(pos[b], pos[b] + 4))
        assert csa.append_pages(L, rows, cache.pages, table.cuda(), i32(pos), norm=True, inv_freq=freq).item() == 0
        outs.append((cache.codes.clone(), cache.scales.clone().view(torch.int32)))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.equal(outs[2][0], outs[3][0]) and torch.equal(outs[2][1], outs[3][1])
    # zeros, a NaN, an infinity, tiny values
    x = normal(g, 1, 5, 512, dtype=L.dtype)
    x[0, 0] = 0
    x[0, 1, 3] = math.nan
    x[0, 2, 3] = math.inf
    x[0, 3] *= 1e-30
    cache = P.Cache(L, 8, 4)
    table = cache.table(1, 1)
    at = torch.tensor(cache.place(table, 0, range(5)), device="cuda")
    csa.append_pages(L, x, cache.pages, table.cuda(), i32([0]))
    c, s = cache.codes.view(-1, 512)[at], cache.scales.view(-1)[at]
    assert s[0] == 0 and (c[0] == 0).all() and torch.isnan(s[1]) and torch.isnan(c[1].view(P.F8).float()).all()
    assert s[2] == math.inf and torch.isnan(c[2].view(P.F8).float()[3])
    P.check_codes(c[3:], s[3:], x[0, 3:].to(F64), torch.zeros(2, 512, dtype=F64, device="cuda"))


def test_append_pages_errors():
    """What a table, a position or a count says wrongly is reported, and only those rows are left out."""
    L, g = P.layer(True), gen(4)
    x = normal(g, 6, 4, L.D)
    cache = P.Cache(L, 8, 20)
    table = cache.table(6, 2)
    pos = [0, -1, 13, 4, 6, 2 ** 31 - 4]
    for b in (0, 2, 4):
        cache.place(table, b, range(16))
    table[3] = torch.tensor([20, -5])       # pages that the pool has not
    table[4, 1] = 1 << 30
    n_new = [4, 4, 4, 4, 4, 4]
    err = csa.append_pages(L, x, cache.pages, table.cuda(), i32(pos), n_new=i32(n_new))
    assert err.item() == csa.DEV_STATE | csa.DEV_CAPACITY | csa.DEV_RANGE
    good = [(0, range(0, 4), range(4)), (2, range(13, 16), range(3)), (4, range(6, 8), range(2))]
    wrote = torch.zeros(160, dtype=torch.bool, device="cuda")
    for b, rows, i in good:
        at = torch.tensor(cache.place(table, b, rows), device="cuda")
        wrote[at] = True
        y = x[b, list(i)].to(F64)
        P.check_codes(cache.codes.view(-1, L.D)[at], cache.scales.view(-1)[at], y, torch.zeros_like(y))
    assert (cache.codes.view(-1, L.D)[~wrote] == 0x7F).all()
    for count in (-1, 5):
        cache = P.Cache(L, 8, 20)
        table = cache.table(6, 2)
        for b in range(6):
            cache.place(table, b, range(16))
        err = csa.append_pages(L, x, cache.pages, table.cuda(), i32([0] * 6), n_new=i32([count] * 6))
        assert err.item() == csa.DEV_STATE and (cache.codes == 0x7F).all()


# ---------------------------------------------------------------------------------------------------- attend_pages


def build(L, B, T, ctx, page, keys, first, counts, seed, junk=-1, spread=1.0, q_scale=2.0):
    """A call of attend_pages whose every unread row is poison: (arguments, host values)."""
    g = gen(seed)
    need_t = [sorted({t for i in range(counts[b]) for t in (set(range(max(0, ctx[b] + i - L.W + 1), ctx[b] + i + 1)) |
                                                            set(range(min(first, ctx[b] + i + 1))))}) for b in range(B)]
    n_rows = [(ctx[b] + T) // L.ratio for b in range(B)]
    per = lambda rows: len({j // page for j in rows})  # noqa: E731
    total = 3 + sum(per(need_t[b]) + (0 if keys == "window" else -(-n_rows[b] // page)) for b in range(B))
    cache = P.Cache(L, page, total, seed, junk)
    tok = cache.table(B, max(1, max(-(-(c + T) // page) for c in ctx)))
    row = cache.table(B, max(1, max(-(-n // page) for n in n_rows)))
    h = dict(pos=ctx, counts=counts, n_rows=n_rows)
    sel = n_sel = None
    if keys == "select":
        sel = torch.full((B, T, L.topk), -1, dtype=torch.int32)
        n_sel = torch.zeros(B, T, dtype=torch.int32)
        r = torch.Generator().manual_seed(seed)
        for b in range(B):
            for i in range(T):
                see = min(n_rows[b], (ctx[b] + i + 1) // L.ratio)
                k = min(see, L.topk)
                n_sel[b, i] = k
                sel[b, i, :k] = torch.randperm(see, generator=r)[:k].sort().values.int()
    for b in range(B):
        if keys == "all":
            rows = range(min(n_rows[b], (ctx[b] + max(1, counts[b])) // L.ratio))
        elif keys == "select":
            rows = sorted({int(j) for i in range(counts[b]) for j in sel[b, i, : int(n_sel[b, i])]})
        else:
            rows = []
        rows = list(rows)
        if rows:
            cache.put(row, b, rows, normal(g, len(rows), L.D) * torch.exp(spread * normal(g, len(rows), 1)))
        if keys != "rows" and need_t[b]:
            cache.put(tok, b, need_t[b], normal(g, len(need_t[b]), L.D) * torch.exp(spread * normal(g, len(need_t[b]), 1)))
    q, sink = normal(g, B, T, L.H, L.D, scale=q_scale, dtype=L.dtype), normal(g, L.H)
    out = torch.full((B, T, L.H, L.D), 7.0, dtype=L.dtype, device="cuda")
    host = dict(token_table=tok, first=first, sink=sink, freq=P.inv_freq(L))
    if keys != "window":
        host |= dict(row_table=row, n_rows=n_rows)
    if sel is not None:
        host |= dict(sel=sel, n_sel=n_sel)
    return cache, q, out, h, host


def call(L, cache, q, out, h, host, **kw):
    args = dict(token_table=host["token_table"].cuda(), first=host["first"], inv_freq=host["freq"])
    if "row_table" in host:
        args |= dict(row_table=host["row_table"].cuda(), n_rows=i32(host["n_rows"]))
    if "sel" in host:
        args |= dict(sel=host["sel"].cuda(), n_sel=host["n_sel"].cuda())
    args |= kw
    return csa.attend_pages(L, q, cache.pages, host["sink"], i32(h["pos"]), out, n_new=i32(h["counts"]), **args)


def verify(L, cache, q, out, h, host):
    want, allow = P.attend_all(L, q, cache, h["pos"], h["counts"], torch.full_like(out, 7.0), **host)
    P.check(out, want, allow)


CASES = [  # B, T, ctx, page, keys, first, counts
    (1, 1, [0], 8, "window", 0, [1]),
    (1, 1, [0], 8, "all", 3, [1]),
    (1, 1, [3], 64, "all", 0, [1]),
    (2, 3, [126, 127], 16, "window", 4, [3, 3]),
    (3, 2, [128, 500, 131], 24, "window", 70, [2, 1, 2]),
    (2, 1, [1000, 37], 128, "all", 0, [1, 1]),
    (3, 4, [777, 5, 300], 64, "all", 1, [4, 0, 3]),
    (2, 2, [2051, 1300], 32, "select", 0, [2, 2]),
    (4, 3, [2600, 90, 255, 2048], 8, "select", 7, [3, 2, 1, 0]),
    (1, 1, [9000], 64, "all", 0, [1]),
    (5, 8, [700, 33, 64, 65, 2100], 16, "all", 2, [8, 8, 1, 5, 8]),
]


@pytest.mark.parametrize("B,T,ctx,page,keys,first,counts", CASES)
@pytest.mark.parametrize("kind", ["small", "odd page", "flash"])
def test_attend_pages(kind, B, T, ctx, page, keys, first, counts):
    """The portable kernel (fp32; bf16 where a page is no whole group of rows) and the tensor cores."""
    L = P.layer(kind == "small")
    if kind == "odd page":
        page -= 3
    args = build(L, B, T, ctx, page, keys, first, counts, seed=B * 100 + T + page, junk=-1 if T % 2 else 1 << 29)
    err = call(L, *args)
    assert err.item() == 0
    verify(L, *args)
