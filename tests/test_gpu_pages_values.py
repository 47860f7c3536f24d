"""attend_pages on values that its tensor-core kernel keeps in few bits, or far apart: tiles in which nothing counts beside keys
far below the largest logit, and many small weights that are alike."""
import math

import pytest
import torch

import deepseek_v4_compressed_csa_gb300 as csa
from tests import _pages as P
from tests.test_gpu_pages import gen, i32, normal
from tests.test_gpu_pages_edges import KINDS, expect, phys

pytestmark = pytest.mark.gpu

TILE = 64


def far_rows(L, n, nats, seed):
    """Rows [n, D] and a query [1, 1, H, D] whose logits are nats (fp32 [n]) and a little: the first value makes them, the
    others are noise."""
    x = normal(gen(seed), n, L.D)
    q = torch.zeros(1, 1, L.H, L.D, device="cuda")
    q[..., 0] = 64.0
    x[:, 0] = nats / (64.0 * L.D ** -0.5)
    return x, q.to(L.dtype)


def attend(L, cache, q, row, n, sel=None, sink=None):
    """One query over rows 0 .. n - 1 of a table, or a selection of them: (output, error word)."""
    out = torch.full_like(q, 7.0)
    more = {}
    if sel is not None:
        full = torch.full((1, 1, L.topk), 1 << 30, dtype=torch.int32)
        full[0, 0, : len(sel)] = torch.tensor(sel, dtype=torch.int32)
        more = dict(sel=full.cuda(), n_sel=i32([[len(sel)]]))
    err = csa.attend_pages(L, q, cache.pages, sink, i32([4 * n]), out, row_table=row.cuda(), n_rows=i32([n]), **more)
    return out, err.item()


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("form,tiles", [("whole", 2), ("whole", 3), ("whole", 4), ("cut", 2), ("cut", 3), ("cut", 4), ("cut", 9)])
@pytest.mark.parametrize("nats", [-60.0, -86.0, -90.0, -120.0])
def test_a_row_of_zeros_above_far_logits(kind, form, tiles, nats):
    """A row of scale 0 has the logit 0, far above every other's: it takes all of the weight and gives nothing."""
    small, page = KINDS[kind]
    L = P.layer(small, topk=TILE * 4)
    n = TILE * tiles
    x, q = far_rows(L, n, torch.full((n,), nats, device="cuda"), 3)
    for at in (0, TILE + 3, n - 1):
        cache = P.Cache(L, page, -(-n // page) + 3)
        row = cache.table(1, -(-n // page))
        x0 = x.clone()
        x0[at] = 0
        cache.put(row, 0, list(range(n)), x0)
        out, err = attend(L, cache, q, row, n, list(range(n)) if form == "whole" else None)
        assert err == 0
        P.check(out, *expect(L, q, cache, [[phys(cache, row, 0, range(n))]], [4 * n], None, None), f"at {at}")


@pytest.mark.parametrize("kind", ["small", "flash"])
@pytest.mark.parametrize("tiles", [2, 3, 4, 7])
@pytest.mark.parametrize("nats", [-70.0, -90.0, -140.0])
@pytest.mark.parametrize("what", ["selection", "table"])
def test_a_tile_without_keys_beside_far_logits(kind, tiles, nats, what):
    """Rows that are out of range, a tile full of them, are left out also where every other logit is far below 0."""
    small, page = KINDS[kind]  # (a tile is whole pages)
    L = P.layer(small, topk=TILE * 7)
    n = TILE * tiles
    x, q = far_rows(L, n, torch.full((n,), nats, device="cuda"), 4)
    for lost in range(min(tiles, 4)):
        cache = P.Cache(L, page, -(-n // page) + 3)
        row = cache.table(1, -(-n // page))
        cache.put(row, 0, list(range(n)), x)
        keys = [j for j in range(n) if j // TILE != lost]
        at = phys(cache, row, 0, keys)
        if what == "selection":
            sel = [j if j // TILE != lost else (-1 - j, 10 ** 6 + j)[j % 2] for j in range(n)]
            out, err = attend(L, cache, q, row, n, sel)
        else:
            row[0, lost * TILE // page : (lost + 1) * TILE // page] = -7
            out, err = attend(L, cache, q, row, n)
        assert err == csa.DEV_RANGE
        P.check(out, *expect(L, q, cache, [[at]], [4 * n], None, None), f"without tile {lost}")


@pytest.mark.parametrize("kind", ["small", "flash"])
@pytest.mark.parametrize("form", ["whole", "cut"])
@pytest.mark.parametrize("tiles", [3, 4])
def test_a_tile_of_zeros_behind_far_logits(kind, form, tiles):
    """A tile of rows of scale 0 as the last one: its logits are the largest, its rows nothing."""
    small, page = KINDS[kind]
    L = P.layer(small, topk=TILE * 4)
    n = TILE * tiles
    for nats in (-60.0, -90.0, -130.0):
        x, q = far_rows(L, n, torch.full((n,), nats, device="cuda"), 5)
        x[n - TILE:] = 0
        cache = P.Cache(L, page, -(-n // page) + 3)
        row = cache.table(1, -(-n // page))
        cache.put(row, 0, list(range(n)), x)
        out, err = attend(L, cache, q, row, n, list(range(n)) if form == "whole" else None)
        assert err == 0
        P.check(out, *expect(L, q, cache, [[phys(cache, row, 0, range(n))]], [4 * n], None, None), f"{nats}")


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("tiles", [2, 5])
def test_a_nan_in_a_tile_that_counts_for_nothing(small, tiles):
    """A row of a NaN scale among rows of scale 0 is NaN all the same."""
    kind = "small" if small else "flash"
    page = KINDS[kind][1]
    L = P.layer(small, topk=TILE * 5)
    n = TILE * tiles
    x, q = far_rows(L, n, torch.full((n,), -90.0, device="cuda"), 6)
    for lost in (0, 1):
        x0 = x.clone()
        x0[lost * TILE : (lost + 1) * TILE] = 0
        cache = P.Cache(L, page, -(-n // page) + 3)
        row = cache.table(1, -(-n // page))
        cache.put(row, 0, list(range(n)), x0)
        cache.scales.view(-1)[phys(cache, row, 0, [lost * TILE + 9])[0]] = math.nan
        for sel in (None, list(range(n))):
            out, err = attend(L, cache, q, row, n, sel)
            assert err == 0 and torch.isnan(out.float()).all()


@pytest.mark.parametrize("kind", ["small", "flash"])
@pytest.mark.parametrize("form", ["whole", "cut"])
@pytest.mark.parametrize("power", [-100.0, -117.0, -119.0, -122.0, -125.0])
def test_one_key_far_below_rows_of_zeros(kind, form, power):
    """A weight of 2^power beside one row of scale 0 and logit 0 reaches the output (as long as fp32 holds it as a normal
    number); the rows between them, further below, do not."""
    small, page = KINDS[kind]
    L = P.layer(small, topk=TILE * 4)
    n = 2 * TILE if form == "whole" else 8 * TILE
    for key in (TILE, 2 * TILE - 1):
        nats = torch.full((n,), -200.0, device="cuda")
        nats[0] = 0
        nats[key] = power * math.log(2)
        x, q = far_rows(L, n, nats, 7)
        others = [j for j in range(n) if j != key]
        x[others, 1:] = 0
        cache = P.Cache(L, page, -(-n // page) + 3)
        row = cache.table(1, -(-n // page))
        cache.put(row, 0, list(range(n)), x)
        out, err = attend(L, cache, q, row, n, list(range(n)) if form == "whole" else None)
        assert err == 0
        want, allow = expect(L, q, cache, [[phys(cache, row, 0, range(n))]], [4 * n], None, None)
        P.check(out[..., 1:], want[..., 1:], allow[..., 1:], f"key {key}")
        assert (want[..., 1:].abs() > allow[..., 1:]).any()


@pytest.mark.parametrize("depth,n", [(8, 256), (9, 512), (10, 1024), (11, 2048), (12, 4096), (14, 16384), (17, 131072)])
@pytest.mark.parametrize("ratio", [1.0, 1 / 16])
def test_many_small_weights_that_are_alike(depth, n, ratio):
    """n rows that are the same, each of x 2^-depth of one dominant row's weight and together about as much, in whole queries:
    what they are rounded to is right on the whole."""
    L = P.layer(ratio=1)
    nb, page = 160, 64
    codes = torch.zeros(-(-(n + 1) // page), page, L.D, dtype=torch.uint8, device="cuda")
    rows = codes.view(-1, L.D)
    rows[1:, 1:] = 0x38            # 1
    rows[1:, 2::2] = 0xB8          # -1
    rows[0, 0], rows[0, L.D // 2:] = 0x7E, 0x3C  # 448; 1.5
    q = torch.zeros(nb, 1, L.H, L.D, device="cuda", dtype=L.dtype)
    q[..., 0] = 8.0
    values = codes.view(P.F8).view(-1, L.D).to(P.F64)
    table = torch.arange(codes.shape[0], dtype=torch.int32, device="cuda").expand(nb, -1).contiguous()
    c = L.D ** -0.5
    for x in (1.0, 1.06, 1.124, 1.126, 1.2, 1.249, 1.251, 1.3, 1.374, 1.376, 1.45, 1.55, 1.624, 1.626, 1.7, 1.874, 1.876, 1.99):
        # weights are e^logit scale: the dominant row's is 2^depth / x times the others'
        s0 = math.log(2.0 ** depth / x * ratio) / (8.0 * 448 * c)
        scales = torch.full(codes.shape[:2], s0 * ratio, device="cuda")
        scales[0, 0] = s0
        out = torch.full_like(q, 7.0)
        err = csa.attend_pages(L, q, csa.Pages(codes, scales), None, i32([n] * nb), out, row_table=table, n_rows=i32([n + 1] * nb))
        assert err.item() == 0 and torch.equal(out, out[:1, :, :1].expand_as(out))
        s = scales.view(-1)[:2].to(P.F64)
        top = 8.0 * 448 * c * s[0]
        p = torch.stack((torch.ones_like(top), torch.exp(-top)))
        keys = values[:2] * s[:, None]
        Z = p[0] + n * p[1]
        want = (p[0] * keys[0] + n * p[1] * keys[1]) / Z
        A = (p[0] * keys[0].abs() + n * p[1] * keys[1].abs()) / Z
        # logits: sums of D products, a rounding each; sums of n weights.  The weights: fp16 (2^-11), then two parts, the nearest
        # (2^-8 of a large one).  Of small ones that are alike, while they are rounded to the nearest, what is lost stays below
        # 2^-9 of all weights and of the largest; from there on 32 thresholds are centred in a step of hi (1/64 of at most 1/4 of
        # the weight) or of lo (1/64 and 1/512 of 2^-9, of weights from 2^-7 on).  Where the dominant row breaks the row of 32,
        # one weight's quarter.
        allow = A * (2 * (L.D + 8) * P.U32 * top + (n + 33) * P.U32 + 2.0 ** -20 + 2.0 ** -11) + 2.0 ** -8 * p[0] / Z * keys[0].abs()
        w0, w1 = p[0] * s[0], p[1] * s[1]
        allow = allow + (2.0 ** -9 * (2 * w0 + n * w1) + 2.0 ** -8 * 1.125 * n * w1 + 0.25 * w1) / Z * values[1].abs()
        allow = allow + (want.abs() + allow) * P.HALF[L.dtype]
        P.check(out[0, 0, 0], want, allow, f"x {x}")


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("X", [128, 4096, 16384])
def test_rows_near_the_ends_of_the_type_are_normed(small, X):
    """Rows whose square sum passes fp32's range, up to the largest values there are, all of a size or one among small ones."""
    L = P.layer(small)
    g = gen(X)
    x = normal(g, 8, X).abs().clamp(0.5, 1.9) * torch.sign(normal(g, 8, X))
    for r, power in enumerate((56, 63, 70, 100, 120, 122, 125, 127)):
        x[r] *= 2.0 ** power
    x[7, : X // 2] *= 2.0 ** -40
    x = x.to(L.dtype)
    assert torch.isfinite(x).all()
    got = csa.add_norm(L, x, torch.zeros_like(x), group=64)
    h = x.to(P.F64)
    y = h / (h.pow(2).mean(-1, keepdim=True) + L.rms_eps).sqrt()
    err = y.abs() * 64 * P.U32  # (as in the other tests of it)
    P.check(got.out, y, err + y.abs() * P.HALF[L.dtype])
    P.check(got.residual, h, h.abs() * P.HALF[L.dtype])
    P.check_codes(got.codes.view(8, -1, 64), got.scales, y.view(8, -1, 64), err.view(8, -1, 64))


@pytest.mark.parametrize("kw", [dict(small=False), dict(small=True), dict(small=True, D=1024, R=8)])
def test_latent_rows_near_the_ends_of_the_type_are_normed(kw):
    L = P.layer(**kw)
    g = gen(L.D)
    x = (normal(g, 1, 8, L.D).abs().clamp(0.5, 1.9) * torch.sign(normal(g, 1, 8, L.D)))
    for r, power in enumerate((56, 63, 70, 100, 120, 122, 125, 127)):
        x[0, r] *= 2.0 ** power
    x = x.to(L.dtype)
    cache = P.Cache(L, 8, 2)
    table = cache.table(1, 1)
    at = torch.tensor(cache.place(table, 0, range(8)), device="cuda")
    assert csa.append_pages(L, x, cache.pages, table.cuda(), i32([0]), norm=True).item() == 0
    y = x[0].to(P.F64)
    y = y / (y.pow(2).mean(-1, keepdim=True) + L.rms_eps).sqrt()
    P.check_codes(cache.codes.view(-1, L.D)[at], cache.scales.view(-1)[at], y, y.abs() * 64 * P.U32)
