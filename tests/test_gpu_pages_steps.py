"""A layer's steps over a cache in pages with the selection that the indexer makes, all on the device: nothing is read on the host
between the calls, so a step is captured into a graph and replayed."""
import math

import pytest
import torch

import csa_synth
import deepseek_v4_compressed_csa_gb300 as csa
from tests import _pages as P
from tests.test_gpu_pages import append_ref, gen, i32, norm_ref, normal
from tests.test_gpu_pages_edges import expect, phys

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    from tests import _gpu as G


class Server:
    """A layer, its weights and a cache that holds ctx[b] tokens of sequence b."""

    def __init__(self, small, T, ctx, page, steps, topk):
        cfg = csa_synth.CONFIGS[1 if small else 3].replace(X=128 if small else 512, topk=topk, rollback=T - 1)
        self.L = L = G.lib_layer(cfg)
        self.T, self.ctx, self.nb = T, ctx, len(ctx)
        self.freq = csa_synth.inv_freq(cfg).cuda()
        self.comp = [G.lib_comp(csa_synth.compressor(cfg, k)) for k in ("attn", "index")]
        g = gen(91)
        dt = L.dtype
        proj = lambda n: normal(g, L.X, n, scale=L.X ** -0.5, dtype=dt)  # noqa: E731
        self.w_kv, self.w_q, self.w_iq, self.w_iw = proj(L.D), proj(L.H * L.D), proj(L.Hi * L.Di), proj(L.Hi)
        self.w_n, self.w_k, self.sink = 1 + 0.1 * normal(g, L.X), 1 + 0.1 * normal(g, L.D), normal(g, L.H)
        last = [c + steps * T for c in ctx]
        n_rows = [c // L.ratio for c in ctx]
        self.cap = max(last) // L.ratio + 8
        self.cache = cache = P.Cache(L, page, sum(2 + -(-p // page) + -(-(p // L.ratio + 1) // page) for p in last) + 2)
        self.tok, self.row = cache.table(self.nb, -(-max(last) // page)), cache.table(self.nb, -(-self.cap // page))
        for b in range(self.nb):
            cache.place(self.tok, b, range(max(0, ctx[b] - L.W), last[b]))
            cache.place(self.tok, b, [0])
            cache.place(self.row, b, range(last[b] // L.ratio + 1))
            old = sorted({0} | set(range(max(0, ctx[b] - L.W), ctx[b]))) if ctx[b] else []
            for table, rows in ((self.tok, old), (self.row, list(range(n_rows[b])))):
                if rows:
                    cache.put(table, b, rows, normal(g, len(rows), L.D))
        self.dtok, self.drow = self.tok.cuda(), self.row.cuda()
        slots = csa.frontier_slots(L.ratio) + L.rollback
        state = dict(pos=i32(ctx), n_rows=i32(n_rows), n_rows_i=i32(n_rows), residual=normal(g, self.nb, T, L.X, dtype=dt),
                     pool=torch.zeros(self.nb, self.cap, L.D, dtype=dt, device="cuda"),
                     ikeys=normal(g, self.nb, self.cap, L.Di, dtype=dt), err=torch.zeros(1, dtype=torch.int32, device="cuda"))
        for k, c in zip("ai", self.comp):
            state["front_" + k] = normal(g, self.nb, slots, 2 * L.lanes * c.d, dtype=dt)
        self.state = state | dict(codes=cache.codes, scales=cache.scales)
        self.x = torch.zeros(self.nb, T, L.X, dtype=dt, device="cuda")
        self.made = -(-T // L.ratio)  # the most rows that T tokens complete

    def step(self):
        """One step on the state; what it made on the way."""
        L, s, nb, T = self.L, self.state, self.nb, self.T
        kept = dict(err=s["err"])
        pages = csa.Pages(s["codes"], s["scales"])
        h = csa.add_norm(L, self.x, s["residual"], self.w_n, residual_out=s["residual"]).out
        before = s["n_rows"].clone()
        csa.compress_append_pair(L, *self.comp, h, s["pos"], s["front_a"], s["pool"], s["n_rows"], s["front_i"], s["ikeys"],
                                 s["n_rows_i"], self.freq, **kept)
        at = (before[:, None] + torch.arange(self.made, device="cuda")).clamp(max=self.cap - 1).long()
        new = s["pool"].gather(1, at[..., None].expand(-1, -1, L.D))
        csa.append_pages(L, new, pages, self.drow, before, n_new=s["n_rows"] - before, **kept)
        latent = h @ self.w_kv
        csa.append_pages(L, latent, pages, self.dtok, s["pos"], weight=self.w_k, norm=True, inv_freq=self.freq, **kept)
        q = csa.norm_rope(L, [(h @ self.w_q).view(nb, T, L.H, L.D)], pos=s["pos"], inv_freq=self.freq, **kept)[0]
        iq, iw = (h @ self.w_iq).view(nb, T, L.Hi, L.Di), h @ self.w_iw
        sel = torch.empty(nb, T, L.topk, dtype=torch.int32, device="cuda")
        n_sel = torch.empty(nb, T, dtype=torch.int32, device="cuda")
        if T == 1:
            csa.index_topk(L, iq[:, 0].contiguous(), iw[:, 0].contiguous(), s["ikeys"], s["n_rows"], s["pos"], self.freq, sel.view(nb, -1),
                           n_sel.view(nb), **kept)
        else:
            csa.index_topk_verify(L, iq, iw, s["ikeys"], s["n_rows"], s["pos"], self.freq, sel, n_sel, **kept)
        out = torch.empty_like(q)
        csa.attend_pages(L, q, pages, self.sink, s["pos"], out, token_table=self.dtok, first=1, row_table=self.drow,
                         n_rows=s["n_rows"], sel=sel, n_sel=n_sel, inv_freq=self.freq, **kept)
        s["pos"] += T
        return dict(h=h, latent=latent, q=q, sel=sel, n_sel=n_sel, out=out, iq=iq, iw=iw)


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("T", [1, 3])
def test_steps_with_the_indexers_selection(small, T):
    """Each step's pages, selection and output against 64 bits on what the calls before it gave; captured and replayed, the same
    bits."""
    steps, topk, page = 6, 24, 16
    v = Server(small, T, [403, 90, 1001, 0, 3], page, steps, topk)
    L, nb = v.L, v.nb
    xs = [normal(gen(200 + k), nb, T, L.X, dtype=L.dtype) for k in range(steps)]
    start = {k: t.clone() for k, t in v.state.items()}
    eager = []
    for k in range(steps):
        res, n0 = v.state["residual"].clone(), v.state["n_rows"].tolist()
        v.x.copy_(xs[k])
        got = v.step()
        eager.append(got)
        assert v.state["err"].item() == 0
        pos, n_rows = [c + k * T for c in v.ctx], v.state["n_rows"].tolist()
        assert v.state["pos"].tolist() == [p + T for p in pos] and n_rows == [(p + T) // L.ratio for p in pos]
        hh, y, e = norm_ref(L, v.x, res, v.w_n)
        P.check(got["h"], y, e + y.abs() * P.HALF[L.dtype], f"step {k}")
        P.check(v.state["residual"], hh, hh.abs() * (P.HALF[L.dtype] + P.U32), f"step {k}")
        keys = []
        for b in range(nb):
            at = torch.tensor(phys(v.cache, v.tok, b, range(pos[b], pos[b] + T)), device="cuda")
            y, e = append_ref(L, got["latent"][b], pos[b] + torch.arange(T, device="cuda"), v.freq, v.w_k, 1)
            P.check_codes(v.cache.codes.view(-1, L.D)[at], v.cache.scales.view(-1)[at], y, e, f"step {k} tokens {b}")
            if n_rows[b] > n0[b]:
                at = torch.tensor(phys(v.cache, v.row, b, range(n0[b], n_rows[b])), device="cuda")
                y = v.state["pool"][b, n0[b]:n_rows[b]].to(P.F64)
                P.check_codes(v.cache.codes.view(-1, L.D)[at], v.cache.scales.view(-1)[at], y, torch.zeros_like(y), f"step {k} rows {b}")
            keys.append([])
            for i in range(T):
                p = pos[b] + i
                vis, n = min(n_rows[b], (p + 1) // L.ratio), int(got["n_sel"][b, i])
                assert n == min(vis, topk), (k, b, i)
                mine = got["sel"][b, i, :n].tolist()
                assert mine == sorted(set(mine)) and all(0 <= j < vis for j in mine)
                toks = sorted(set(range(max(0, p - L.W + 1), p + 1)) | {0})
                keys[-1].append(phys(v.cache, v.row, b, mine) + phys(v.cache, v.tok, b, toks))
        P.check(got["out"], *expect(L, got["q"], v.cache, keys, pos, v.sink, v.freq), f"step {k}")
    assert math.prod(eager[-1]["n_sel"].shape) and (eager[-1]["n_sel"] == topk).any()  # (more visible than are taken)
    end = {k: t.clone() for k, t in v.state.items()}
    for k, t in v.state.items():
        t.copy_(start[k])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        made = v.step()
    for k, t in v.state.items():
        t.copy_(start[k])
    for k in range(steps):
        v.x.copy_(xs[k])
        graph.replay()
        for name in ("h", "latent", "q", "sel", "n_sel", "out"):
            assert torch.equal(made[name], eager[k][name]), (k, name)
    for k, t in v.state.items():
        assert torch.equal(t.view(torch.uint8) if t.is_floating_point() else t, end[k].view(torch.uint8) if t.is_floating_point() else end[k]), k
