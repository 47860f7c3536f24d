"""The operators around a cache in pages and 8 bits, as measured workloads.

A server hands a layer's cache out in pages: `codes` [n_pages, page, D] (E4M3) and `scales` [n_pages, page] (fp32, one per
row), with a table per sequence that says which page holds its logical rows 0 .. page-1, page .. 2 page-1, and so on.
add_norm prepares the hidden states (residual addition, RMS norm, an 8-bit copy with a scale per group of values),
append_pages writes latent rows into their pages (norm, rotation and scale on the way), attend_pages attends: T queries a
sequence over the selected or all visible compressed rows, the last W tokens and a few first ones.

Shapes are the Flash layer's (hidden size 4096, 64 heads over a 512-dim latent, 128-token window, 512 selected rows) and,
for other types and sizes, the small fp32 layer of the tests.
"""
import math

import numpy as np
import torch

own = False

FLASH = dict(H=64, D=512, R=64, W=128, Hi=64, Di=128, topk=512, X=4096, dtype="bf16", base=160000.0)
SMALL = dict(H=8, D=64, R=16, W=32, Hi=4, Di=32, topk=16, X=128, dtype="f32", base=10000.0)
EPS = 1e-6
F8 = torch.float8_e4m3fn


def listed():
    return [
        # one token of one sequence: the least that a decode step does, all latency
        dict(name="add_norm_decode_n1", op="add_norm", layer="flash", N=1, group=128),
        # fp32 rows of an odd count
        dict(name="add_norm_f32_n61", op="add_norm", layer="small", N=61, group=32),
        # a prefill chunk's hidden states
        dict(name="add_norm_prefill_n4096", op="add_norm", layer="flash", N=4096, group=128),
        # a serving batch's new tokens, one each
        dict(name="append_decode_b32", op="append_pages", layer="flash", B=32, T=1, ctx=8192, page=64, rows="tokens", ragged=False),
        # a prefill chunk's tokens
        dict(name="append_prefill_t4096", op="append_pages", layer="flash", B=1, T=4096, ctx=65536, page=64, rows="tokens", ragged=False),
        # a dense layer (no compressed rows): window and four first tokens, one user
        dict(name="attend_window_b1", op="attend_pages", layer="flash", keys="window", ratio=128, B=1, T=1, ctx=8192, first=4, page=64, ragged=False),
        # a ratio-4 layer, one user: the selected rows and the window
        dict(name="attend_select_b1", op="attend_pages", layer="flash", keys="select", ratio=4, B=1, T=1, ctx=8192, first=0, page=64, ragged=False),
        # a serving batch that verifies four drafted tokens a sequence
        dict(name="attend_select_b32_t4", op="attend_pages", layer="flash", keys="select", ratio=4, B=32, T=4, ctx=32768, first=0, page=64, ragged=False),
        # a ratio-128 layer at a long context, small pages
        dict(name="attend_r128_b16", op="attend_pages", layer="flash", keys="all", ratio=128, B=16, T=1, ctx=262144, first=0, page=16, ragged=False),
        # one user whose ratio-4 layer reads every row
        dict(name="attend_all_b1", op="attend_pages", layer="flash", keys="all", ratio=4, B=1, T=1, ctx=131072, first=0, page=64, ragged=False),
        # a batch of such users: the largest cache
        dict(name="attend_all_b8", op="attend_pages", layer="flash", keys="all", ratio=4, B=8, T=1, ctx=262144, first=4, page=64, ragged=False),
        # fp32, odd sizes, sequences with fewer queries than the widest
        dict(name="attend_f32_b5_t3", op="attend_pages", layer="small", keys="all", ratio=4, B=5, T=3, ctx=1003, first=3, page=8, ragged=True),
    ]


def draw(rng):
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["add_norm", "append_pages", "attend_pages", "attend_pages"])
    if op == "add_norm":
        small = rng.random() < 0.25
        return dict(op=op, layer="small" if small else "flash", N=size(1, 4096), group=rng.choice([32, 64, 128]))
    layer = rng.choice(["flash", "flash", "flash", "small"])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "append_pages":
        B = size(1, 64)
        return dict(op=op, layer=layer, B=B, T=size(1, 4096 // B), ctx=size(64, 65536), page=page,
                    rows=rng.choice(["tokens", "tokens", "rows"]), ragged=rng.random() < 0.5)
    keys = rng.choice(["window", "select", "all"])
    B, T = size(1, 64), rng.choice([1, 1, 2, 3, 5, 8])
    ratio = rng.choice([4, 128]) if keys == "all" else 4
    most = (65536 if layer == "small" else 524288) // (B * T)  # keys a query, at most the largest case's in all
    ctx = size(16, min(262144, max(64, (most if keys == "all" else 65536) * (ratio if keys == "all" else 1))))
    return dict(op=op, layer=layer, keys=keys, ratio=ratio, B=B, T=T, ctx=ctx, first=rng.choice([0, 0, 1, 4, 7]), page=page,
                ragged=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------------- inputs


def dims(case):
    return dict(FLASH if case["layer"] == "flash" else SMALL)


def positions(case):
    """Each sequence's tokens before the call's: ragged, the longest ctx."""
    return [case["ctx"] - (61 * b) % (case["ctx"] // 4 + 1) for b in range(case["B"])]


def counts(case):
    """Each sequence's new tokens: T, or fewer (none now and then) where the batch is ragged."""
    T = case["T"]
    return [T if not case["ragged"] else max(0, T - b % (T + 1)) for b in range(case["B"])]


def old_rows(case):
    return [(p + case["T"]) // case["ratio"] for p in positions(case)]


def quantised(x):
    """Rows of values to (codes, scales): scale = amax / 448, E4M3 rounded to nearest."""
    s = x.abs().amax(-1, keepdim=True) / 448.0
    q = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0)
    return q.to(F8).view(torch.uint8), s[..., 0]


def in_use(case, c):
    """For each table, [B, pages a sequence] truth values: the pages that hold something; others are not handed out."""
    P, pos, T = case["page"], np.array(positions(case))[:, None], case["T"]
    k = np.arange((case["ctx"] + T + P - 1) // P)[None, :]
    tokens = (k * P < pos + T) & ((k + 1) * P > pos - c["W"])  # (a window further back than any query's)
    if case["op"] == "append_pages":
        return {"token_table": tokens}
    tokens |= (k * P < case["first"]) & (k * P < pos + T)
    found = {"token_table": tokens}
    if case["keys"] != "window":
        n = np.array(old_rows(case))[:, None]
        found["row_table"] = np.arange(max(1, -(-int(n.max()) // P)))[None, :] * P < n
    return found


def prepare(case, seed):
    c = dims(case)
    dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
    g = torch.Generator("cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = dict(case=case, c=c, kept={})
    if case["op"] == "add_norm":
        N, X = case["N"], c["X"]
        s |= dict(x=normal(N, X), residual=normal(N, X, scale=4.0), weight=1.0 + 0.1 * normal(X, dtype=torch.float32))
        s |= dict(out=torch.zeros_like(s["x"]), residual_out=torch.zeros_like(s["x"]),
                  codes=torch.zeros(N, X, dtype=torch.uint8, device="cuda"),
                  scales=torch.zeros(N, X // case["group"], device="cuda"))
        return s
    B, T, P, D = case["B"], case["T"], case["page"], c["D"]
    half = np.arange(c["R"] // 2, dtype=np.float64)
    s["inv_freq"] = torch.from_numpy((c["base"] ** (-2.0 * half / c["R"])).astype(np.float32)).cuda()
    s["pos"] = torch.tensor(positions(case), dtype=torch.int32, device="cuda")
    s["n_new"] = torch.tensor(counts(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
    used = in_use(case, c)
    n_pages = sum(int(u.sum()) for u in used.values()) + 3
    ids = np.random.RandomState(seed % (1 << 31)).permutation(n_pages).astype(np.int32)
    at = 0
    for name, u in used.items():
        table = np.full(u.shape, -1, dtype=np.int32)
        table[u] = ids[at : at + int(u.sum())]
        at += int(u.sum())
        s[name] = torch.from_numpy(table).cuda()
    if case["op"] == "append_pages":
        s["codes"] = torch.zeros(n_pages, P, D, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(n_pages, P, device="cuda")
        s["rows"] = normal(B, T, D, scale=3.0)
        s["weight"] = 1.0 + 0.1 * normal(D, dtype=torch.float32)
        return s
    s["codes"], s["scales"] = quantised(torch.randn(n_pages, P, D, generator=g, device="cuda"))
    s["q"] = normal(B, T, c["H"], D, scale=2.0)
    s["sink"] = normal(c["H"], dtype=torch.float32)
    s["out"] = torch.zeros_like(s["q"])
    s["n_rows"] = torch.tensor(old_rows(case), dtype=torch.int32, device="cuda") if case["keys"] != "window" else None
    s["sel"] = s["n_sel"] = None
    if case["keys"] == "select":
        p = s["pos"][:, None] + torch.arange(T, device="cuda")
        sees = torch.minimum(s["n_rows"][:, None], (p + 1) // case["ratio"])
        n = max(c["topk"], max(old_rows(case)))
        score = torch.rand(B, T, n, generator=g, device="cuda").masked_fill(torch.arange(n, device="cuda") >= sees[..., None], 2.0)
        took, k = torch.minimum(sees, torch.tensor(c["topk"], device="cuda")), torch.arange(c["topk"], device="cuda")
        rows = score.topk(c["topk"], largest=False).indices
        rows = rows.masked_fill(k >= took[..., None], n).sort().values
        s["sel"] = rows.masked_fill(rows == n, -1).int()
        s["n_sel"] = took.int()
    return s


# ---------------------------------------------------------------------------------------------------- plain forms


def rotate(x, p, inv_freq, R, sign):
    """The last R values of x [.., dim], pairs of neighbours, turned by sign * p * inv_freq (p [..], the library's angle:
    one fp32 product)."""
    a = (p.float()[..., None] * inv_freq).double()
    cs, sn = a.cos().float(), sign * a.sin().float()
    u, v = x[..., -R::2], x[..., -R + 1 :: 2]
    return torch.cat((x[..., :-R], torch.stack((u * cs - v * sn, u * sn + v * cs), -1).flatten(-2)), -1)


def plain_add_norm(s):
    x, g = s["x"], s["case"]["group"]
    h = x.float() + s["residual"].float()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"]
    codes, scales = quantised(y.view(*y.shape[:-1], -1, g))
    return dict(out=y.to(x.dtype), residual=h.to(x.dtype), codes=codes.flatten(-2).view(F8), scales=scales)


def places(table, logical, page):
    """Physical rows of logical rows [B, ..] (0 where there is none)."""
    at = torch.gather(table.long(), 1, (logical // page).clamp(0, table.shape[1] - 1).flatten(1)).view(logical.shape)
    return (at * page + logical % page).clamp(min=0)


def plain_append(s):
    case, c, x = s["case"], s["c"], s["rows"].float()
    i = torch.arange(case["T"], device="cuda")
    p = s["pos"].long()[:, None] + i
    if case["rows"] == "tokens":
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"]
        x = rotate(x, p, s["inv_freq"], c["R"], 1.0)
    codes, scales = quantised(x)
    at = places(s["token_table"], p, case["page"])
    if s["n_new"] is not None:
        on = i < s["n_new"][:, None]
        at, codes, scales = at[on], codes[on], scales[on]
    s["codes"].view(-1, c["D"])[at] = codes
    s["scales"].view(-1)[at] = scales
    return s["codes"].view(F8), s["scales"]


def plain_attend(s):
    case, c = s["case"], s["c"]
    B, T, P, D = case["B"], case["T"], case["page"], c["D"]
    p = s["pos"].long()[:, None] + torch.arange(T, device="cuda")
    back = p[..., None] - c["W"] + 1
    t = torch.cat((back + torch.arange(c["W"], device="cuda"), torch.arange(case["first"], device="cuda").expand(B, T, -1)), -1)
    sees = torch.cat((t[..., : c["W"]] >= 0, t[..., c["W"] :] < back), -1)
    at = places(s["token_table"], t.clamp(min=0), P)
    if case["keys"] != "window":
        if case["keys"] == "select":
            j = s["sel"].long()
            ok = torch.arange(c["topk"], device="cuda") < s["n_sel"][..., None]
        else:
            j = torch.arange(s["row_table"].shape[1] * P, device="cuda").expand(B, T, -1)
            ok = j < torch.minimum(s["n_rows"][:, None], (p + 1) // case["ratio"])[..., None]
        at = torch.cat((at, places(s["row_table"], j.clamp(min=0), P)), -1)
        sees = torch.cat((sees, ok), -1)
    keys = s["codes"].view(-1, D)[at].view(F8).float()
    keys = keys.mul_(s["scales"].view(-1)[at][..., None])
    lg = (s["q"].float() @ keys.transpose(-1, -2)) * D**-0.5
    lg = lg.masked_fill(~sees[..., None, :], -math.inf)
    m = torch.maximum(lg.amax(-1, keepdim=True), s["sink"][:, None])
    e = (lg - m).exp()
    o = (e @ keys) / (e.sum(-1, keepdim=True) + (s["sink"][:, None] - m).exp())
    o = rotate(o, p[..., None], s["inv_freq"], c["R"], -1.0).to(s["q"].dtype)
    if s["n_new"] is None:
        return o
    return torch.where((torch.arange(T, device="cuda") < s["n_new"][:, None])[..., None, None], o, s["out"])


def run(s):
    if own:
        return run_own(s)
    return {"add_norm": plain_add_norm, "append_pages": plain_append, "attend_pages": plain_attend}[s["case"]["op"]](s)


# ---------------------------------------------------------------------------------------------------- the framework's


def run_own(s):
    import deepseek_v4_compressed_csa_gb300 as csa

    case, c, kept = s["case"], s["c"], s["kept"]
    op = case["op"]
    if not kept:  # what a program keeps from call to call: the layer, the pages' handle, an error word, a workspace
        dt = torch.bfloat16 if c["dtype"] == "bf16" else torch.float32
        kept["layer"] = csa.Layer(dtype=dt, H=c["H"], D=c["D"], R=c["R"], W=c["W"], ratio=case.get("ratio", 4), Hi=c["Hi"],
                                  Di=c["Di"], topk=c["topk"], X=c["X"])
        kept["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if op != "add_norm":
            kept["pages"] = csa.Pages(s["codes"], s["scales"])
        if op == "attend_pages":
            need = csa.workspace_size(kept["layer"], csa.OP_ATTEND_PAGES, case["B"], case["T"], 1)
            kept["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    if op == "add_norm":
        csa.add_norm(kept["layer"], s["x"], s["residual"], s["weight"], group=case["group"], out=s["out"],
                     residual_out=s["residual_out"], codes=s["codes"], scales=s["scales"])
        return dict(out=s["out"], residual=s["residual_out"], codes=s["codes"].view(F8), scales=s["scales"])
    if op == "append_pages":
        more = dict(inv_freq=s["inv_freq"], weight=s["weight"], norm=True) if case["rows"] == "tokens" else {}
        csa.append_pages(kept["layer"], s["rows"], kept["pages"], s["token_table"], s["pos"], n_new=s["n_new"], err=kept["err"],
                         **more)
        return s["codes"].view(F8), s["scales"]
    csa.attend_pages(kept["layer"], s["q"], kept["pages"], s["sink"], s["pos"], s["out"], token_table=s["token_table"],
                     first=case["first"], row_table=s.get("row_table"), n_rows=s["n_rows"], sel=s["sel"], n_sel=s["n_sel"],
                     n_new=s["n_new"], inv_freq=s["inv_freq"], ws=kept["ws"], err=kept["err"])
    return s["out"]


# ---------------------------------------------------------------------------------------------------- what a pass needs


def work(case):
    c = dims(case)
    es = 2 if c["dtype"] == "bf16" else 4
    if case["op"] == "add_norm":
        n = case["N"] * c["X"]
        return dict(bytes=n * (4 * es + 1) + 4 * n / case["group"] + 4 * c["X"], flops=8 * n)
    if case["op"] == "append_pages":
        n = sum(counts(case))
        return dict(bytes=n * (c["D"] * (es + 1) + 8) + 4 * c["D"], flops=8 * n * c["D"])
    keys = held = 0
    for p, m, n in zip(positions(case), counts(case), old_rows(case) if case["keys"] != "window" else [0] * case["B"]):
        if not m:
            continue
        see = [min(n, (p + i + 1) // case["ratio"]) for i in range(m)]
        took = [min(v, c["topk"]) if case["keys"] == "select" else v for v in see]
        seen = [min(p + i + 1, c["W"]) + min(case["first"], max(0, p + i + 1 - c["W"])) for i in range(m)]
        keys += sum(took) + sum(seen)
        # the rows that m independent selections touch; a window's tokens are shared but for the newest
        held += n * (1 - (1 - took[-1] / max(1, n)) ** m) if case["keys"] == "select" else took[-1]
        held += min(seen[-1] + m - 1, p + m)
    n = sum(counts(case))
    return dict(bytes=held * (c["D"] + 4) + 2 * n * c["H"] * c["D"] * es, flops=4.0 * keys * c["H"] * c["D"])


# ---------------------------------------------------------------------------------------------------- in 64 bits


def _turned(x, p, inv_freq, sign):
    """x [heads, dim] (64 bits) turned as complex numbers by the angles that the layer defines (fp32 products)."""
    R = 2 * inv_freq.numel()
    th = (torch.tensor(float(p), dtype=torch.float32, device=x.device) * inv_freq).double()
    z = torch.view_as_complex(x[:, -R:].reshape(x.shape[0], R // 2, 2).contiguous())
    z = z * torch.polar(torch.ones_like(th), sign * th)
    return torch.cat((x[:, :-R], torch.view_as_real(z).reshape(x.shape[0], R)), 1)


def exact(case, seed):
    s = prepare(case, seed)
    c, d64 = s["c"], torch.float64
    if case["op"] == "add_norm":
        h = s["x"].to(d64) + s["residual"].to(d64)
        y = h / (h.pow(2).sum(-1, keepdim=True) / c["X"] + EPS).sqrt() * s["weight"].to(d64)
        amax = y.abs().reshape(case["N"], -1, case["group"]).max(-1).values
        return dict(out=y, residual=h, codes=None, scales=amax / 448)
    pos, new, P = positions(case), counts(case), case["page"]
    if case["op"] == "append_pages":
        scales = s["scales"].to(d64)
        table = s["token_table"].tolist()
        for b in range(case["B"]):
            x = s["rows"][b].to(d64)
            if case["rows"] == "tokens":
                x = x / (x.pow(2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * s["weight"].to(d64)
            for i in range(new[b]):
                t = pos[b] + i
                row = _turned(x[i : i + 1], t, s["inv_freq"], 1.0) if case["rows"] == "tokens" else x[i : i + 1]
                scales[table[b][t // P], t % P] = row.abs().max() / 448
        return None, scales
    if sum(new) * max([c["topk"]] + (old_rows(case) if case["keys"] == "all" else [])) > 1 << 21:
        return None
    out = s["out"].to(d64)
    value = s["codes"].view(F8).to(d64 if s["codes"].numel() < 1 << 27 else torch.float32)
    for b in range(case["B"]):
        for i in range(new[b]):
            p = pos[b] + i
            t = sorted(set(range(max(0, p - c["W"] + 1), p + 1)) | set(range(min(case["first"], p + 1))))
            where = [(s["token_table"], torch.tensor(t, device="cuda"))]
            if case["keys"] == "select":
                where.append((s["row_table"], s["sel"][b, i, : int(s["n_sel"][b, i])].long()))
            elif case["keys"] == "all":
                where.append((s["row_table"], torch.arange(min(old_rows(case)[b], (p + 1) // case["ratio"]), device="cuda")))
            keys = torch.cat([value[tab[b][j // P].long(), j % P].to(d64) * s["scales"][tab[b][j // P].long(), j % P].to(d64)[:, None] for tab, j in where])
            lg = torch.cat((s["q"][b, i].to(d64) @ keys.T / math.sqrt(c["D"]), s["sink"].to(d64)[:, None]), 1)
            out[b, i] = _turned(torch.softmax(lg, 1)[:, :-1] @ keys, p, s["inv_freq"], -1.0)
    return out
