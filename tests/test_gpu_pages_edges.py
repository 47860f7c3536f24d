"""append_pages and attend_pages where they can go wrong: what tables, counts and selections say wrongly, batches of every
plan, queries split over many blocks, far positions, large pools, odd values, streams, graphs, guard bands."""
import math
import random
import threading

import pytest
import torch

import csa_synth
import deepseek_v4_compressed_csa_gb300 as csa
from deepseek_v4_compressed_csa_gb300 import _binding as B
from tests import _pages as P
from tests.test_gpu_pages import append_ref, build, call, gen, i32, normal, norm_ref, verify

pytestmark = pytest.mark.gpu
F64 = P.F64

if torch.cuda.is_available():
    from tests import _gpu as G
    from tests.test_gpu_guard_bands import Guards

KINDS = {"small": (True, 8), "odd page": (False, 13), "flash": (False, 16)}  # layer, rows of a page


def tensor_cores(L, page):
    return L.dtype == torch.bfloat16 and (L.H, L.D, L.R) == (64, 512, 64) and page % 8 == 0


def expect(L, q, cache, keys, pos, sink, freq, out0=7.0):
    """Outputs and allowances where query (b, i) has the physical rows keys[b][i] (None: it is not there)."""
    want = torch.full(q.shape, out0, dtype=F64, device="cuda")
    allow = torch.zeros_like(want)
    for b, row in enumerate(keys):
        for i, at in enumerate(row):
            if at is None:
                continue
            at = torch.tensor(at, dtype=torch.long, device="cuda")
            codes = cache.codes.view(P.F8).view(-1, L.D)[at].to(F64)
            o, e = P.attend_ref(L, q[b, i], codes, cache.scales.view(-1)[at].to(F64), sink, tensor_cores(L, cache.page))
            if freq is not None:
                e = P.pair_sum(e + 8 * P.U32 * o.abs(), L.R)
                o = P.turn(o, torch.full((L.H,), pos[b] + i, device="cuda"), freq, -1.0)
            want[b, i], allow[b, i] = o, e + (o.abs() + e) * P.HALF[L.dtype] + P.LEAST[L.dtype]
    return want, allow


def phys(cache, table, b, rows):
    return [int(table[b, j // cache.page]) * cache.page + j % cache.page for j in rows]


def fill(cache, table, b, rows, seed, scale=1.0):
    rows = list(rows)
    cache.put(table, b, rows, normal(gen(seed), len(rows), cache.L.D, scale=scale))


# ------------------------------------------------------------------------------------------------ reported errors


@pytest.mark.parametrize("kind", list(KINDS))
def test_bad_tables_and_counts(kind):
    """Every wrong entry is reported, and only what it names is left out."""
    small, page = KINDS[kind]
    L = P.layer(small, W=32)
    nb, T = 7, 2
    cache = P.Cache(L, page, 100)
    pos = [70, 50, -3, 40, 2 ** 31 - 1, 33, 30]
    n_rows = [18, 9, 4, -2, 4, 400, 8]
    width_t, width_r = -(-72 // page), -(-18 // page)
    tok, row = cache.table(nb, width_t), cache.table(nb, width_r)
    for b in range(nb):
        fill(cache, tok, b, range(0, width_t * page), 10 + b)
        fill(cache, row, b, range(0, width_r * page), 30 + b)
    lost_t, lost_r = tok.clone(), row.clone()
    bad_t, bad_r = pos[0] // page - 1, 0
    tok[0, bad_t], row[0, bad_r] = cache.n, -1       # pages that the pool has not, in a window and among the rows
    counts = [2, 2, 2, 2, 2, 1, 3]                   # more than T: skipped; one sequence of one
    q, sink, freq = normal(gen(1), nb, T, L.H, L.D, dtype=L.dtype), normal(gen(2), L.H), P.inv_freq(L)
    out = torch.full_like(q, 7.0)

    def keys(b, i, rows):
        p = pos[b] + i
        toks = sorted(set(range(max(0, p - 31), p + 1)) | set(range(min(3, p + 1))))
        return ([x for j, x in zip(rows, phys(cache, lost_r, b, rows)) if row[b, j // page] >= 0] +
                [x for j, x in zip(toks, phys(cache, lost_t, b, toks)) if tok[b, j // page] < cache.n])

    see = lambda b, i: list(range(min(max(n_rows[b], 0), (pos[b] + i + 1) // L.ratio)))  # noqa: E731
    want = [[keys(b, i, see(b, i)) if b in (0, 1, 3) or (b == 5 and i == 0) else None for i in range(T)] for b in range(nb)]
    err = csa.attend_pages(L, q, cache.pages, sink, i32(pos), out, token_table=tok.cuda(), first=3, row_table=row.cuda(),
                           n_rows=i32(n_rows), n_new=i32(counts), inv_freq=freq)
    assert err.item() == csa.DEV_RANGE | csa.DEV_STATE
    P.check(out, *expect(L, q, cache, want, pos, sink, freq))


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("what", ["tokens", "rows"])
def test_rows_behind_a_table(kind, what):
    """A table too short for what a query sees: reported, and the rest of its keys counts."""
    small, page = KINDS[kind]
    L = P.layer(small, W=32, ratio=4 if what == "tokens" else 128)
    cache = P.Cache(L, page, 60)
    tok, row = cache.table(1, 3 if what == "tokens" else 500), cache.table(1, 2)
    pos, n_rows = (3 * page + 1, 1) if what == "tokens" else (128 * (2 * page + 1), 10 ** 9)
    last = 3 * page if what == "tokens" else pos + 1
    toks = sorted(set(range(max(0, pos - 31), min(pos + 1, last))) | {0, 1})
    fill(cache, tok, 0, toks, 1)
    fill(cache, row, 0, range(2 * page), 2)
    q, sink = normal(gen(3), 1, 1, L.H, L.D, dtype=L.dtype), normal(gen(4), L.H)
    out = torch.full_like(q, 7.0)
    err = csa.attend_pages(L, q, cache.pages, sink, i32([pos]), out, token_table=tok.cuda(), first=2, row_table=row.cuda(),
                           n_rows=i32([n_rows]))
    assert err.item() == csa.DEV_CAPACITY
    rows = range(min(n_rows, (pos + 1) // L.ratio, 2 * page))
    P.check(out, *expect(L, q, cache, [[phys(cache, row, 0, rows) + phys(cache, tok, 0, toks)]], [pos], sink, None))


@pytest.mark.parametrize("kind", list(KINDS))
def test_selections(kind):
    """Indices out of range are reported and left out, one listed twice counts twice, counts out of range are bounded; a
    selection of nothing, in and out of order, behind its count anything."""
    small, page = KINDS[kind]
    L = P.layer(small)
    nb, T, K = 6, 2, L.topk
    cache = P.Cache(L, page, 60)
    row = cache.table(nb, -(-40 // page))
    for b in range(nb):
        fill(cache, row, b, range(40), 50 + b)
    sel = torch.full((nb, T, K), 1 << 30, dtype=torch.int32)
    n_sel = torch.zeros(nb, T, dtype=torch.int32)
    lists = [[[0, 1, 39], []], [[5, 5, 5, 7], [39, 3, 17, 2]], [[40, 3], [-1, 4]], [[2 ** 31 - 1, -2 ** 31, 8], [41]],
             [list(range(K)) if K <= 40 else [j % 40 for j in range(K)], [1]], [[9, 30], [31, 10]]]
    n_rows = [40, 40, 40, 40, 40, 30]
    bad = [[0, 0], [0, 0], [1, 1], [1, 1], [1, 1], [1, 1]]
    for b in range(nb):
        for i in range(T):
            v = lists[b][i]
            sel[b, i, : len(v)] = torch.tensor(v, dtype=torch.int64).to(torch.int32)
            n_sel[b, i] = len(v)
    n_sel[4, 0], n_sel[4, 1] = K + 5, -1  # bounded to K, and to none
    lists[4][1] = []
    pos, sink, freq = [200] * nb, normal(gen(6), L.H), P.inv_freq(L)
    q = normal(gen(5), nb, T, L.H, L.D, dtype=L.dtype)
    for b in range(nb):
        one = torch.full_like(q[b:b + 1], 7.0)
        err = csa.attend_pages(L, q[b:b + 1], cache.pages, sink, i32(pos[:1]), one, row_table=row[b:b + 1].cuda(),
                               n_rows=i32(n_rows[b:b + 1]), sel=sel[b:b + 1].cuda(), n_sel=n_sel[b:b + 1].cuda(), inv_freq=freq)
        assert err.item() == (csa.DEV_RANGE if any(bad[b]) else 0), b
        keys = [[phys(cache, row, b, [j for j in v if 0 <= j < n_rows[b]]) for v in lists[b]]]
        P.check(one, *expect(L, q[b:b + 1], cache, keys, pos, sink, freq), f"b{b}")


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("sink", [True, False])
def test_no_keys(kind, sink):
    """Queries whose tables name nothing, whose rows are none yet: zeros, with a sink and without."""
    small, page = KINDS[kind]
    L = P.layer(small)
    cache = P.Cache(L, page, 4)
    row = cache.table(3, 2)
    q, z = normal(gen(7), 3, 1, L.H, L.D, dtype=L.dtype), normal(gen(8), L.H) if sink else None
    out = torch.full_like(q, 7.0)
    err = csa.attend_pages(L, q, cache.pages, z, i32([0, 500, 500]), out, row_table=row.cuda(), n_rows=i32([5, 0, 3]),
                           inv_freq=P.inv_freq(L))
    assert err.item() == csa.DEV_RANGE  # the last one's rows have no page
    assert (out == 0).all()
    out.fill_(7.0)
    err = csa.attend_pages(L, q, cache.pages, z, i32([3, 5, 6]), out, token_table=row.cuda(), n_new=i32([0, 0, 0]))
    assert err.item() == 0 and (out == 7.0).all()


# ------------------------------------------------------------------------------------------------ plans


BATCHES = {  # sequences, queries each, lengths, counts (sequence -> queries)
    "one each": (200, 1, lambda b: 37 * b % 900, lambda b: 1),
    "one long": (170, 1, lambda b: 40000 if b == 77 else 30 + b, lambda b: 1),
    "two a thread": (130, 4, lambda b: 61 * b % 500, lambda b: (b * 7) % 5),
    "few of many": (420, 1, lambda b: 2500 + b, lambda b: int(b % 70 == 3)),
    "none": (170, 2, lambda b: 9, lambda b: 0),
    "one of many": (1000, 1, lambda b: 9000, lambda b: int(b == 999)),
    "40": (40, 1, lambda b: 300 + 97 * b, lambda b: 1),
    "151": (151, 1, lambda b: 700 * (b % 3), lambda b: 1),
    "152": (152, 1, lambda b: 5 + 900 * (b % 2), lambda b: 1),
    "33 short": (33, 1, lambda b: b, lambda b: 1),
}


@pytest.mark.parametrize("kind", ["small", "flash"])
@pytest.mark.parametrize("name", list(BATCHES))
def test_batches(kind, name):
    nb, T, length, count = BATCHES[name]
    small, page = KINDS[kind]
    L = P.layer(small, topk=24)
    for keys, first in (("all", 2), ("select", 0), ("window", 5)):
        args = build(L, nb, T, [length(b) for b in range(nb)], page, keys, first, [count(b) for b in range(nb)], seed=nb + T)
        assert call(L, *args).item() == 0
        verify(L, *args)


@pytest.mark.parametrize("kind", ["small", "flash"])
def test_largest_batch(kind):
    """2^16 queries, few of them there; ratio 1."""
    small, page = KINDS[kind]
    L = P.layer(small, ratio=1)
    there = {0: 7, 100: 256, 255: 31}
    args = build(L, 256, 256, [300 * (b in there) for b in range(256)], page, "all", 3, [there.get(b, 0) for b in range(256)], seed=5)
    assert call(L, *args).item() == 0
    verify(L, *args)


@pytest.mark.parametrize("kind", ["small", "flash"])
@pytest.mark.parametrize("nb,T,ctx", [(1, 1, 90000), (2, 3, 30000), (5, 1, 20011)])
def test_long_queries(kind, nb, T, ctx):
    """Queries that every block has a part of, split unevenly among some: the merge."""
    small, page = KINDS[kind]
    L = P.layer(small)
    args = build(L, nb, T, [max(0, ctx - 7001 * b) for b in range(nb)], page * 4, "all", 1, [T] * nb, seed=T, q_scale=1.0)
    assert call(L, *args).item() == 0
    verify(L, *args)


@pytest.mark.parametrize("D,R,H,dtype", [(8, 8, 1, torch.float32), (16, 8, 3, torch.bfloat16), (24, 8, 9, torch.float32),
                                         (72, 24, 5, torch.bfloat16), (136, 16, 17, torch.float32), (256, 256, 2, torch.bfloat16),
                                         (264, 64, 8, torch.float32), (512, 64, 64, torch.float32), (520, 8, 7, torch.bfloat16),
                                         (1024, 64, 8, torch.float32), (1024, 1024, 1, torch.bfloat16), (512, 64, 32, torch.bfloat16)])
def test_layers(D, R, H, dtype):
    L = P.layer(True, D=D, R=R, H=H, dtype=dtype, Di=max(R, 8), Hi=2, W=20, topk=33)
    for keys, ctx in (("all", [3, 5000, 400]), ("select", [250, 90, 30]), ("window", [0, 19, 77])):
        args = build(L, 3, 2, ctx, 9, keys, 1, [2, 1, 2], seed=D + R)
        assert call(L, *args).item() == 0
        verify(L, *args)


@pytest.mark.parametrize("seed", range(6))
def test_shapes_at_random(seed):
    """Layers, batches, lengths, pages and counts drawn over their ranges, six calls a seed."""
    r = random.Random(seed)
    for n in range(6):
        kw = dict(ratio=r.choice([1, 4, 4, 128]), W=r.choice([1, 7, 32, 128, 300]), topk=r.choice([5, 64, 100, 512]))
        small, keys = r.random() < 0.4, r.choice(["window", "select", "all"])
        if small:
            kw |= dict(H=r.choice([1, 3, 8, 11]), D=r.choice([16, 64, 72, 264, 512, 640]), R=r.choice([8, 16]), Di=16,
                       dtype=r.choice([torch.float32, torch.bfloat16]))
        L = P.layer(small, **{**kw, "ratio": 4 if keys == "select" else kw["ratio"]})
        nb, T = int(200 ** r.random()), r.choice([1, 1, 2, 3, 8, 40])
        nb = min(nb, max(1, 300 // T))
        most = 60000 // (nb * T) * L.ratio if keys == "all" else 4000
        ctx = [r.randint(0, max(1, min(most, 20000))) for _ in range(nb)]
        counts = [r.choice([T, T, r.randint(0, T)]) for _ in range(nb)]
        args = build(L, nb, T, ctx, r.choice([8, 16, 24, 40, 64, 128, 13, 1, 7]), keys, r.choice([0, 1, 4, 70]), counts,
                     seed=100 * seed + n, junk=r.choice([-1, 1 << 29]), spread=r.choice([0.3, 1.0, 2.0]), q_scale=r.choice([0.5, 2.0, 6.0]))
        assert call(L, *args).item() == 0
        verify(L, *args)


# ------------------------------------------------------------------------------------------------ values


@pytest.mark.parametrize("kind", ["small", "flash"])
@pytest.mark.parametrize("growth", [1.0, 1.02, 0.98, 1.5])
def test_growing_and_falling_keys(kind, growth):
    """Maxima that rise all along the keys, or fall: logits from far below the largest to it, in both directions."""
    small, page = KINDS[kind]
    L = P.layer(small)
    n = 1200 if growth != 1.5 else 180
    cache = P.Cache(L, page, 400)
    row = cache.table(1, -(-n // page))
    base = normal(gen(3), 1, L.D)
    size = torch.tensor([growth ** (j if growth < 1.5 else j % 30) for j in range(n)], device="cuda", dtype=torch.float32)[:, None]
    cache.put(row, 0, list(range(n)), (base + 0.3 * normal(gen(4), n, L.D)) * size / size.amax())
    q = (base[None, None] * (1 + 0.1 * normal(gen(5), 1, 2, L.H, 1)) + normal(gen(6), 1, 2, L.H, L.D, scale=0.1)).to(L.dtype)
    q[:, :, 1] *= -1
    out = torch.full_like(q, 7.0)
    p = 4 * n + 3
    assert csa.attend_pages(L, q, cache.pages, None, i32([p]), out, row_table=row.cuda(), n_rows=i32([n])).item() == 0
    keys = [[phys(cache, row, 0, range(n))] * 2]
    P.check(out, *expect(L, q, cache, keys, [p], None, None))


@pytest.mark.parametrize("kind", ["small", "flash"])
def test_one_key_above_a_long_tail(kind):
    """One key beside tens of thousands that weigh 2^-14 of it each, and as much together."""
    small, page = KINDS[kind]
    L = P.layer(small)
    n = 30000
    cache = P.Cache(L, page * 4, n // page // 4 + 9)
    row = cache.table(1, -(-n // (4 * page)))
    x = normal(gen(3), n, L.D)
    x[:, 0] = 0
    q = torch.zeros(1, 1, L.H, L.D, device="cuda")
    q[..., 0] = 8.0
    x[777] = 0
    x[777, 0] = 14 * math.log(2) / (8.0 * L.D ** -0.5)
    cache.put(row, 0, list(range(n)), x)
    q, out = q.to(L.dtype), torch.full((1, 1, L.H, L.D), 7.0, dtype=L.dtype, device="cuda")
    p = 4 * n
    assert csa.attend_pages(L, q, cache.pages, None, i32([p]), out, row_table=row.cuda(), n_rows=i32([n])).item() == 0
    P.check(out, *expect(L, q, cache, [[phys(cache, row, 0, range(n))]], [p], None, None))


@pytest.mark.parametrize("kind", ["small", "flash"])
def test_scales_of_all_sizes(kind):
    """Rows of zeros, scales from 2^-112 to 2^20 and of both signs beside one another and by themselves; queries that are
    tiny, huge, zero."""
    small, page = KINDS[kind]
    L = P.layer(small)
    for group, powers in enumerate(([0, -3, -20, -60, -112], [-110] * 5, [20, 19, -5, 0, -100], [-130, -140, 0, -1, -2])):
        n = 200
        cache = P.Cache(L, page, 60)
        row = cache.table(1, -(-n // page))
        fill(cache, row, 0, range(n), 60 + group)
        at = torch.tensor(phys(cache, row, 0, range(n)), device="cuda")
        s = cache.scales.view(-1)
        s[at] *= torch.tensor([2.0 ** powers[j % 5] * (-1.0 if j % 7 == 3 else 1.0) for j in range(n)], device="cuda", dtype=F64).float()
        s[at[::11]] = 0.0
        q = normal(gen(9), 1, 4, L.H, L.D)
        q[0, 1] *= 2.0 ** -100
        q[0, 2] = 0
        q[0, 3, :, 5:] = 0
        if max(powers) < 10:
            q[0, 3] *= 8
        else:
            q *= 2.0 ** -20
        q, out = q.to(L.dtype), torch.full((1, 4, L.H, L.D), 7.0, dtype=L.dtype, device="cuda")
        p = 4 * n
        assert csa.attend_pages(L, q, cache.pages, None, i32([p]), out, row_table=row.cuda(), n_rows=i32([n])).item() == 0
        want, allow = expect(L, q, cache, [[phys(cache, row, 0, range(n))] * 4], [p], None, None)
        # (below the normal numbers a rounding is half a step of 2^-133 in bf16, of 2^-149 in fp32)
        P.check(out, want, allow + 2.0 ** -133, f"group {group}")


@pytest.mark.parametrize("kind", ["small", "flash"])
def test_nan_and_infinity(kind):
    """A NaN or an infinity in a row reaches the queries that see it, in a query its own head, in a sink its head: nothing
    else; also where the query is split."""
    small, page = KINDS[kind]
    L = P.layer(small)
    for ctx in (900, 12000):
        cache, q, out, h, host = build(L, 3, 2, [ctx, ctx, ctx], page, "all", 0, [2, 2, 2], seed=3)
        assert call(L, cache, q, out, h, host).item() == 0
        clean = out.clone()
        cache.codes[int(host["row_table"][1, 0]), 1, 5] = 0x7F
        q[0, 1, 2, 7] = math.nan
        q[2, 0, 3, 1] = math.inf
        host["sink"] = host["sink"].clone()
        host["sink"][4] = math.nan
        host["sink"][5] = -math.inf
        assert call(L, cache, q, out, h, host).item() == 0
        nan = torch.isnan(out.float())
        assert nan[1].all() and nan[:, :, 4].all()
        whole = torch.zeros(3, 2, L.H, dtype=torch.bool, device="cuda")
        whole[1], whole[:, :, 4], whole[0, 1, 2], whole[2, 0, 3] = True, True, True, True
        assert nan[whole].all() and not nan[~whole].any()
        other = ~whole
        other[:, :, 5] = False  # (without its sink)
        assert torch.equal(out[other], clean[other])


# ------------------------------------------------------------------------------------------------ places


@pytest.mark.parametrize("p", [99999, 123457, 1 << 24, (1 << 27) + 5, (1 << 29) - 2, (1 << 29) + 3, (1 << 30) + 11, 2 ** 31 - 3])
@pytest.mark.parametrize("kind", list(KINDS))
def test_far_positions(kind, p):
    """Angles of positions far out: split queries and whole ones, and rows appended there."""
    small, page = KINDS[kind]
    L = P.layer(small)
    n = 4000
    cache = P.Cache(L, page, n // page + 9)
    row = cache.table(2, -(-n // page))
    fill(cache, row, 0, range(n), 1)
    fill(cache, row, 1, range(30), 2)
    q, sink, freq = normal(gen(3), 2, 2, L.H, L.D, dtype=L.dtype), normal(gen(4), L.H), P.inv_freq(L)
    out = torch.full_like(q, 7.0)
    pos = [p, p]
    assert csa.attend_pages(L, q, cache.pages, sink, i32(pos), out, row_table=row.cuda(), n_rows=i32([n, 30]),
                            inv_freq=freq).item() == 0
    keys = [[phys(cache, row, 0, range(n))] * 2, [phys(cache, row, 1, range(30))] * 2]
    P.check(out, *expect(L, q, cache, keys, pos, sink, freq))
    if p + 1 < 1 << 30:
        big = 1 << 20  # rows of a page: few of them reach far
        L = P.layer(True, D=16, R=16, Di=16)
        freq = P.inv_freq(L)
        cache = P.Cache(L, big, 3)
        table = cache.table(1, (p + 2) // big + 1)
        at = torch.tensor(cache.place(table, 0, [p, p + 1]), device="cuda")
        x = normal(gen(5), 1, 2, L.D, dtype=L.dtype)
        assert csa.append_pages(L, x, cache.pages, table.cuda(), i32([p]), norm=True, inv_freq=freq).item() == 0
        y, e = append_ref(L, x[0], torch.tensor([p, p + 1], device="cuda"), freq, None, 1)
        P.check_codes(cache.codes.view(-1, L.D)[at], cache.scales.view(-1)[at], y, e)


@pytest.mark.parametrize("kind", ["small", "flash"])
def test_large_pools(kind):
    """Pools beyond 2^32 bytes (Flash), and of the most rows a pool may have, in pages of one."""
    L = P.layer(False) if kind == "flash" else P.layer(True, D=8, R=8, Di=8)
    page, n_pages = (8, 6_000_000) if kind == "flash" else (1, 2 ** 31 - 257)
    codes = torch.empty(n_pages, page, L.D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(n_pages, page, device="cuda")
    cache = P.Cache(L, page, 1)
    cache.codes, cache.scales, cache.n = codes, scales, n_pages
    n, T = 70, 3
    far = [n_pages - 1 - k for k in range(200)] + [0, 1, n_pages // 2, 2 ** 32 // (page * L.D), 2 ** 31 // (page * L.D) + 1]
    cache.free = far
    tok, row = cache.table(1, -(-n // page)), cache.table(1, -(-(n // 4) // page))
    x, rows, freq = normal(gen(1), 1, n, L.D, dtype=L.dtype), normal(gen(2), 1, n // 4, L.D, dtype=L.dtype), P.inv_freq(L)
    at, at_r = cache.place(tok, 0, range(n)), cache.place(row, 0, range(n // 4))
    assert csa.append_pages(L, x, cache.pages, tok.cuda(), i32([0]), norm=True, inv_freq=freq).item() == 0
    assert csa.append_pages(L, rows, cache.pages, row.cuda(), i32([0])).item() == 0
    y, e = append_ref(L, x[0], torch.arange(n, device="cuda"), freq, None, 1)
    where = torch.tensor(at, device="cuda")
    P.check_codes(codes.view(-1, L.D)[where], scales.view(-1)[where], y, e)
    q, sink = normal(gen(3), 1, T, L.H, L.D, dtype=L.dtype), normal(gen(4), L.H)
    out = torch.full_like(q, 7.0)
    p = n - T
    assert csa.attend_pages(L, q, cache.pages, sink, i32([p]), out, token_table=tok.cuda(), first=2, row_table=row.cuda(),
                            n_rows=i32([n // 4]), inv_freq=freq).item() == 0
    keys = [[at_r[: min(n // 4, (p + i + 1) // L.ratio)] + [at[t] for t in sorted(set(range(max(0, p + i - L.W + 1), p + i + 1)) | {0, 1})]
             for i in range(T)]]
    P.check(out, *expect(L, q, cache, keys, [p], sink, freq))


def test_a_page_in_two_tables_and_twice_in_one():
    """A prefix that sequences share, and a page that one table names twice, are read as often as they are named."""
    L = P.layer()
    cache = P.Cache(L, 64, 20)
    tok = cache.table(2, 4)
    fill(cache, tok, 0, range(200), 1)
    tok[1] = tok[0]
    tok[1, 2] = tok[1, 1]
    q, sink = normal(gen(2), 2, 1, L.H, L.D, dtype=L.dtype), normal(gen(3), L.H)
    out = torch.full_like(q, 7.0)
    assert csa.attend_pages(L, q, cache.pages, sink, i32([199, 199]), out, token_table=tok.cuda(), first=9).item() == 0
    toks = list(range(9)) + list(range(72, 200))
    P.check(out, *expect(L, q, cache, [[phys(cache, tok, b, toks)] for b in range(2)], [199, 199], sink, None))


# ------------------------------------------------------------------------------------------------ runs


def step(seed, small=False, kind="all", nb=3, T=2, ctx=4000):
    L = P.layer(small)
    args = build(L, nb, T, [ctx + 13 * b for b in range(nb)], 16, kind, 2, [T] * nb, seed=seed)
    return L, args


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("kind", ["all", "select", "window"])
def test_runs_repeat_exactly(small, kind):
    """The same call gives the same bits: by itself, behind others, from the binding's own code, captured and replayed on
    changed inputs, twice in one graph with a workspace that both share."""
    L, args = step(1, small, kind)
    cache, q, out, h, host = args
    first = q.new_full(q.shape, 0)
    assert call(L, *args).item() == 0
    first.copy_(out)
    ws = torch.full((max(256, csa.workspace_size(L, csa.OP_ATTEND_PAGES, 3, 2, 1)),),
                    0xFF, dtype=torch.uint8, device="cuda")
    fixed = dict(ws=ws, err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    for _ in range(3):
        out.fill_(7.0)
        call(L, *args, **fixed)
        assert torch.equal(out, first)
        ws.fill_(0xFF)
    kept, B._plain = B._plain, None
    try:
        out.fill_(7.0)
        call(L, *args, **fixed)
    finally:
        B._plain = kept
    assert torch.equal(out, first)
    tables = dict(token_table=host["token_table"].cuda())
    if "row_table" in host:
        tables |= dict(row_table=host["row_table"].cuda(), n_rows=i32(host["n_rows"]))
    if "sel" in host:
        tables |= dict(sel=host["sel"].cuda(), n_sel=host["n_sel"].cuda())
    pos, fresh, out2 = i32(h["pos"]), i32(h["counts"]), torch.empty_like(out)
    q2 = q.flip(0).contiguous()

    def both():
        for a, o in ((q, out), (q2, out2)):
            csa.attend_pages(L, a, cache.pages, host["sink"], pos, o, first=2, inv_freq=host["freq"], n_new=fresh, **tables, **fixed)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    out.fill_(7.0)
    want2 = out2.clone()
    out2.fill_(7.0)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(out2, want2)
    q.copy_(q2)  # other queries in the captured tensors
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want2) and fixed["err"].item() == 0


def test_streams_and_threads():
    """Calls at once from two threads, each on a stream of its own, eager and replayed: each as by itself."""
    jobs = [step(11, False, "all"), step(12, False, "select", ctx=3000), step(13, True, "all", ctx=9000), step(14, False, "window")]
    want = []
    for L, args in jobs:
        assert call(L, *args).item() == 0
        want.append(args[2].clone())
    torch.cuda.synchronize()
    got, errors = [None] * len(jobs), []

    def work(k):
        try:
            L, args = jobs[k]
            with torch.cuda.stream(torch.cuda.Stream()):
                outs = []
                for _ in range(20):
                    out = torch.full_like(args[2], 7.0)
                    err = call(L, args[0], args[1], out, *args[3:])
                    outs.append((out, err))
                torch.cuda.current_stream().synchronize()
                got[k] = outs
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not errors
    for k, outs in enumerate(got):
        assert all(torch.equal(o, want[k]) and e.item() == 0 for o, e in outs), k


def test_stream_argument():
    """stream=: the call runs there, behind what was enqueued there before, its own memory with it."""
    L, args = step(21)
    cache, q, out, h, host = args
    call(L, *args)
    want = out.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    later = torch.zeros_like(q)
    with torch.cuda.stream(side):
        a = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            a = a @ a * 1e-3
        later.copy_(q)
    o2 = torch.full_like(out, 7.0)
    side.wait_stream(torch.cuda.current_stream())
    err = call(L, cache, later, o2, h, host, stream=side)
    junk = [torch.full((1 << 22,), -1.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(o2, want)
    del junk
    x = normal(gen(1), 5, 512, dtype=L.dtype)
    ref = csa.add_norm(L, x, x, group=64)
    got = csa.add_norm(L, x, x, group=64, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("kind", list(KINDS))
def test_guard_bands(kind):
    """Nothing is written outside the buffers, and nothing that lies there is read for a result."""
    small, page = KINDS[kind]
    L = P.layer(small)
    for keys, ctx, T in (("all", [5, 3001, 64], 3), ("select", [2500, 40, 129], 2), ("window", [0, 131, 77], 1), ("all", [9000], 1)):
        cache, q, out, h, host = build(L, len(ctx), T, ctx, page, keys, 3, [T] * len(ctx), seed=T)
        nb = len(ctx)
        gd = Guards()
        x, r, w = normal(gen(2), nb, T, L.D, dtype=L.dtype), normal(gen(3), nb, T, L.D, dtype=L.dtype), normal(gen(4), L.D)
        names = dict(q=q, out=out, sink=host["sink"], pos=i32(h["pos"]), tok=host["token_table"], freq=host["freq"],
                     codes=cache.codes, scales=cache.scales, x=x, r=r, w=w, n=i32(h["counts"]))
        t = {k: gd.wrap(k, v) for k, v in names.items()}
        more = {}
        if "row_table" in host:
            more |= dict(row_table=gd.wrap("row", host["row_table"]), n_rows=gd.wrap("n_rows", i32(host["n_rows"])))
        if "sel" in host:
            more |= dict(sel=gd.wrap("sel", host["sel"]), n_sel=gd.wrap("n_sel", host["n_sel"]))
        ws = gd.ws("ws", csa.workspace_size(L, csa.OP_ATTEND_PAGES, nb, T, 1))
        err = gd.wrap("err", torch.zeros(1, dtype=torch.int32))
        pool = csa.Pages(t["codes"], t["scales"])
        got = csa.add_norm(L, t["x"], t["r"], t["w"], group=8, out=gd.empty("o", x.shape, L.dtype),
                           residual_out=gd.empty("ro", x.shape, L.dtype), codes=gd.empty("c", x.shape, torch.uint8),
                           scales=gd.empty("s", (nb, T, L.D // 8), torch.float32))
        want = csa.add_norm(L, x, r, w, group=8)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        csa.attend_pages(L, t["q"], pool, t["sink"], t["pos"], t["out"], token_table=t["tok"], first=3, n_new=t["n"],
                         inv_freq=t["freq"], ws=ws, err=err, **more)
        assert err.item() == 0
        verify(L, cache, q, t["out"], h, host)
        csa.append_pages(L, t["x"], pool, t["tok"], t["pos"], n_new=t["n"], weight=t["w"], norm=True, inv_freq=t["freq"], err=err)
        assert err.item() == 0
        for name, slab, size, _ in gd.slabs:
            assert (slab[:4096] == 0xFF).all() and (slab[4096 + size:] == 0xFF).all(), name
        same = {k for k in names if k not in ("out", "codes", "scales")}
        assert all(torch.equal(t[k].reshape(-1).view(torch.uint8), names[k].cuda().contiguous().reshape(-1).view(torch.uint8)) for k in same)


# ------------------------------------------------------------------------------------------------ together


@pytest.mark.parametrize("T", [1, 4])
def test_steps_of_a_layer(T):
    """A layer's steps as they would be served: the residual's norm, the compressed rows and the latent rows into pages,
    the queries' norm and rotation, the selection, the attention; each step against 64 bits on what it was given."""
    cfg = csa_synth.CONFIGS[3].replace(X=512)
    L = G.lib_layer(cfg)
    nb, steps, page, cap = 3, 9, 16, 200
    freq = csa_synth.inv_freq(cfg).cuda()
    comp = G.lib_comp(csa_synth.compressor(cfg, "attn"))
    g = gen(77)
    front = torch.zeros(nb, csa.frontier_slots(L.ratio), 2 * L.lanes * comp.d, device="cuda", dtype=L.dtype)
    w_kv, w_q = normal(g, L.X, L.D, scale=L.X ** -0.5, dtype=L.dtype), normal(g, L.X, L.H * L.D, scale=L.X ** -0.5, dtype=L.dtype)
    w_n, w_k, sink = 1 + 0.1 * normal(g, L.X), 1 + 0.1 * normal(g, L.D), normal(g, L.H)
    cache = P.Cache(L, page, nb * 40)
    total = steps * T
    tok, row = cache.table(nb, -(-total // page)), cache.table(nb, -(-(total // 4) // page))
    for b in range(nb):
        cache.place(tok, b, range(total))
        cache.place(row, b, range(max(1, total // 4)))
    dtok, drow = tok.cuda(), row.cuda()
    pos, n_rows = i32([0] * nb), i32([0] * nb)
    pool = torch.zeros(nb, cap, L.D, dtype=L.dtype, device="cuda")
    residual = normal(g, nb, T, L.X, dtype=L.dtype)
    for s in range(steps):
        x = normal(g, nb, T, L.X, dtype=L.dtype)
        got = csa.add_norm(L, x, residual, w_n, group=128)
        hh, y, e = norm_ref(L, x, residual, w_n)
        P.check(got.out, y, e + y.abs() * P.HALF[L.dtype], f"step {s}")
        P.check_codes(got.codes.view(nb, T, -1, 128), got.scales, y.view(nb, T, -1, 128), e.view(nb, T, -1, 128))
        residual, h = got.residual, got.out
        before = n_rows.clone()
        assert csa.compress_append(L, comp, h, pos, front, pool, n_rows, freq).item() == 0
        made = n_rows - before
        most = int(made.max())
        if most:
            new = torch.stack([pool[b, int(before[b]):int(before[b]) + most] for b in range(nb)])
            assert csa.append_pages(L, new, cache.pages, drow, before, n_new=made).item() == 0
        latent = h @ w_kv
        assert csa.append_pages(L, latent, cache.pages, dtok, pos, weight=w_k, norm=True, inv_freq=freq).item() == 0
        where = torch.tensor([phys(cache, tok, b, range(s * T, s * T + T)) for b in range(nb)], device="cuda")
        yk, ek = append_ref(L, latent, torch.arange(s * T, s * T + T, device="cuda").expand(nb, T), freq, w_k, 1)
        P.check_codes(cache.codes.view(-1, L.D)[where], cache.scales.view(-1)[where], yk, ek, f"step {s}")
        q = (h @ w_q).view(nb, T, L.H, L.D)
        q = csa.norm_rope(L, [q], pos=pos, inv_freq=freq)[0]
        out = torch.empty_like(q)
        assert csa.attend_pages(L, q, cache.pages, sink, pos, out, token_table=dtok, first=1, row_table=drow, n_rows=n_rows,
                                inv_freq=freq).item() == 0
        keys = []
        for b in range(nb):
            keys.append([])
            for i in range(T):
                p = s * T + i
                toks = sorted(set(range(max(0, p - L.W + 1), p + 1)) | {0})
                keys[-1].append(phys(cache, row, b, range(min(int(n_rows[b]), (p + 1) // 4))) + phys(cache, tok, b, toks))
        P.check(out, *expect(L, q, cache, keys, [s * T] * nb, sink, freq), f"step {s}")
        pos += T
