"""Trees of drafted tokens on the GPU (norm_rope, compress_tree, index_scores_tree, attend_tree, commit_tree) against
the definitions in float64, each alone over types, head layouts, topologies and lengths, then as the step that they
make together.

Tolerances (u = 2^-24, h = half a step of the model dtype at the value: 2^-9 of its binade's top in bf16):
  norm_rope   one rounding of an fp32 result: h, plus 2^-18 of the rotated pair's norm.  fp32: a sum of up to 1024
              squares over 32 lanes (32 + 5 adds deep, so 37 u), a square root, a division, three products and
              sincosf (2 ulp): under 64 u = 2^-18.
  rows        the rule of check_pool_rows on the GPU's own projections; projections by check_projection.
  scores      fp32 sums of Di + Hi products: (Di + Hi + 8) u of the sum of absolute products bounds each value in any
              order, doubled for an accumulator that truncates; over a row, errors are independent and the 2-norm
              stays within 2^-18 of the row's.
  attention   h, plus 2^-11 of the row's largest element: logits err by under 2^-16 (512 products of bf16 values in
              fp32), probabilities by 2^-16 (two bf16 parts), and the average over keys cannot exceed twice that; 2^-11
              leaves room for logits up to 32.  fp32: 1e-5 of the row's largest element.
  fp8 scores  as the scores, on the codes of keys and queries (products of two codes are exact in fp32); the folded
              weight is rounded twice more, 2 u relative to every head's term.
  selection   equal, for the scores that the call was given.
"""
import dataclasses

import numpy as np
import pytest
import torch

import csa_synth
from oracle import csa_oracle as O
from tests import _tree as TR
from tests._common import f64, oracle_comp, oracle_layer

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import deepseek_v4_compressed_csa_gb300 as csa
    from tests import _gpu as G

FLASH = csa_synth.CONFIGS[3].replace(X=512)
TINY = csa_synth.CONFIGS[1]
ODD = csa_synth.CONFIGS[1].replace(cid=61, dtype="bf16", H=5, D=72, R=24, W=9, Hi=3, Di=40, topk=7, X=64)
LAYERS = {"flash": FLASH, "flash_r128": FLASH.replace(cid=62, ratio=128), "tiny_f32": TINY,
          "tiny_f32_r8": TINY.replace(cid=63, ratio=8), "odd_bf16": ODD}
SENTINEL = 7.0


def rnd(cfg, shape, tag, scale=1.0, dtype=None):
    a = np.random.default_rng([5, cfg.cid, tag]).standard_normal(shape, dtype=np.float32) * np.float32(scale)
    return torch.from_numpy(a).to(dtype or cfg.storage).cuda()


def freqs(cfg):
    return csa_synth.inv_freq(cfg).cuda()


def parents(trees, T=None):
    T = T or max(len(t) for t in trees)
    return torch.tensor([TR.padded(t, T) for t in trees], dtype=torch.int32, device="cuda")


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def half_step(x, dtype):
    return 0.5 * G.ulp(x, dtype)


# ------------------------------------------------------------------------------------------------ norm_rope

NR_CASES = {
    # layer, B, T, trees (None: consecutive tokens), first position
    "flash_one_token": ("flash", 1, 1, None, 32767),
    "flash_batch_tree": ("flash", 3, 16, "bushy", 100001),
    "flash_chunk": ("flash", 1, 300, None, 5),
    "flash_long_chunk": ("flash", 1, 1400, None, 5),  # a block per token
    "tiny_f32_tree": ("tiny_f32", 4, 7, "bushy", 999),
    "odd_dims_tree": ("odd_bf16", 2, 64, "bushy", 0),
    "odd_dims_chain64": ("odd_bf16", 1, 64, "chain", 262143),
}


@pytest.mark.parametrize("case", list(NR_CASES))
@pytest.mark.parametrize("rotate", [True, False])
def test_norm_rope_against_float64(case, rotate):
    name, B, T, kind, p0 = NR_CASES[case]
    cfg = LAYERS[name]
    trees = None if kind is None else [getattr(TR, kind)(max(1, T - b)) for b in range(B)]
    par = None if trees is None else parents(trees, T)
    pos = torch.tensor([p0 + 13 * b for b in range(B)], dtype=torch.int32, device="cuda")
    invf = freqs(cfg)
    # q and kv out of one wide projection (strided tokens), index heads on their own, and one head without a head axis
    wide = rnd(cfg, (B, T, cfg.H * cfg.D + cfg.D + 8), 1, scale=2.0)
    q = wide[..., :cfg.H * cfg.D].unflatten(-1, (cfg.H, cfg.D))
    kv = wide[..., cfg.H * cfg.D:cfg.H * cfg.D + cfg.D]
    iq = rnd(cfg, (B, T, cfg.Hi, cfg.Di), 2)
    w = rnd(cfg, (cfg.D,), 3, dtype=torch.float32)
    outs = [torch.full_like(t, SENTINEL) for t in (q.contiguous(), kv.contiguous(), iq)]
    err = err_word()
    got = csa.norm_rope(G.lib_layer(cfg), [q, kv, iq], pos, invf if rotate else None, parent=par,
                        weights=[None, w, None], norm=[True, True, False], outs=outs, err=err)
    assert err.item() == 0 and got[0] is outs[0]
    f = f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    for b in range(B):
        paths = [list(range(i + 1)) for i in range(T)] if trees is None else TR.paths(TR.padded(trees[b], T))
        for i in range(T) if T <= 64 else (0, 1, 63, 64, T - 1):
            for x, o, wt, norm in ((q, outs[0], None, True), (kv[:, :, None], outs[1][:, :, None], w, True),
                                   (iq, outs[2], None, False)):
                g = f64(o[b, i])
                if paths[i] is None:
                    assert (g == SENTINEL).all()
                    continue
                ref = TR.norm_rope(x[b, i], wt, norm, cfg.rms_eps, int(pos[b]) + len(paths[i]) - 1, f if rotate else None)
                pair = np.repeat(np.hypot(ref[..., ::2], ref[..., 1::2]), 2, axis=-1)
                assert (np.abs(g - ref) <= half_step(np.abs(ref) + 2.0 ** -18 * pair, cfg.dtype) + 2.0 ** -18 * pair).all()


@pytest.mark.parametrize("name", ["flash", "tiny_f32"])
@pytest.mark.parametrize("T", [3, 1300])
def test_norm_rope_long_and_short_rows(name, T):
    """Rows of up to 1024 values (four chunks a lane) next to short ones, in one call."""
    cfg = LAYERS[name]
    f = f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    short = cfg.R + 8
    xs = [rnd(cfg, (2, T, 3, 1024), 7, scale=3.0), rnd(cfg, (2, T, 520), 8), rnd(cfg, (2, T, 5, short), 9)]
    ws = [None, rnd(cfg, (520,), 10, dtype=torch.float32), rnd(cfg, (short,), 11, dtype=torch.float32)]
    pos = torch.tensor([70000, 0], dtype=torch.int32, device="cuda")
    err = err_word()
    got = csa.norm_rope(G.lib_layer(cfg), xs, pos, freqs(cfg), weights=ws, err=err)
    assert err.item() == 0
    for x, w, o in zip(xs, ws, got):
        x4, o4 = (x, o) if x.dim() == 4 else (x[:, :, None], o[:, :, None])
        for b in range(2):
            for i in (0, 1, T - 1):
                ref = TR.norm_rope(x4[b, i], w, True, cfg.rms_eps, int(pos[b]) + i, f)
                pair = np.repeat(np.hypot(ref[..., ::2], ref[..., 1::2]), 2, axis=-1)
                tol = 2.0 ** -18 * pair
                assert (np.abs(f64(o4[b, i]) - ref) <= half_step(np.abs(ref) + tol, cfg.dtype) + tol).all()


def test_norm_rope_in_place_and_zero_rows():
    """out may be x; a row of zeros stays zeros (eps > 0)."""
    cfg = FLASH
    q = rnd(cfg, (2, 3, 64, 512), 4)
    q[0, 1, 5] = 0
    ref = csa.norm_rope(G.lib_layer(cfg), [q], torch.tensor([9, 10], dtype=torch.int32, device="cuda"), freqs(cfg))[0]
    got = csa.norm_rope(G.lib_layer(cfg), [q], torch.tensor([9, 10], dtype=torch.int32, device="cuda"), freqs(cfg),
                        outs=[q])[0]
    assert got is q and torch.equal(q, ref) and not ref[0, 1, 5].any()


def test_norm_rope_feeds_the_calls_that_rotate():
    """Normalised without rotation, then attend_decode rotates; or rotated here, then attend_tree: the same output."""
    cfg = FLASH.replace(ctx=300)
    host = csa_synth.synth_cache(cfg.replace(B=2), 100, B=2)
    st = G.DevCache(host)
    L = G.lib_layer(cfg)
    q, kv = rnd(cfg, (2, 1, 64, 512), 5, scale=3.0), rnd(cfg, (2, 1, 512), 6, scale=3.0)
    sink, invf = csa_synth.sinks(cfg).cuda(), freqs(cfg)
    par = parents([[-1], [-1]])
    tq, tkv = csa.norm_rope(L, [q, kv], st.pos, invf, parent=par)
    rows = torch.zeros(2, 1, 512, dtype=torch.bfloat16, device="cuda")
    out_t = torch.empty_like(q)
    err = csa.attend_tree(L, tq, tkv, sink, st.window, st.pool, rows, None, par, st.n_rows, st.pos, invf, out_t)
    nq, nkv = csa.norm_rope(L, [q, kv])
    out_d = torch.empty(2, 64, 512, dtype=torch.bfloat16, device="cuda")
    err2 = csa.attend_decode(L, nq[:, 0].contiguous(), nkv[:, 0].contiguous(), sink, st.window, st.pool, st.n_rows, None,
                             None, st.pos, invf, out_d)
    assert err.item() == 0 and err2.item() == 0
    # three more roundings to bf16 on the way (the rotated query and key, the output before its rotation)
    a, b = f64(out_t[:, 0]), f64(out_d)
    assert np.abs(a - b).max() <= 2.0 ** -6 * np.abs(b).max()


# ------------------------------------------------------------------------------------------------ compress_tree

CT_CASES = {
    # layer, trees, positions
    "flash": ("flash", [TR.bushy(16), TR.bushy(13, 1), TR.chain(16)], [0, 4097, 10]),
    "flash_star": ("flash", [TR.star(9)], [7]),
    "flash_deep": ("flash", [TR.chain(64)], [3]),
    "flash_r128": ("flash_r128", [TR.chain(40), TR.bushy(40), [-1]], [100, 127, 4095]),
    "tiny_f32": ("tiny_f32", [TR.bushy(11), TR.chain(5), TR.binary(11)], [2, 0, 77]),
    "tiny_f32_r8": ("tiny_f32_r8", [TR.chain(20), TR.bushy(20)], [5, 23]),
    "odd_bf16": ("odd_bf16", [TR.binary(31), [-1]], [1, 3]),
}


@pytest.mark.parametrize("case", list(CT_CASES))
def test_compress_tree_against_paths(case):
    name, trees, pos = CT_CASES[case]
    cfg = LAYERS[name]
    B, T = len(trees), max(len(t) for t in trees)
    layer, invf = oracle_layer(cfg), f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    hosts = {"a": csa_synth.compressor(cfg, "attn")}
    if cfg.has_indexer:
        hosts["i"] = csa_synth.compressor(cfg, "index")
    x = rnd(cfg, (B, T, cfg.X), 10)
    F = cfg.frontier_slots
    bufs = {}
    for k, h in hosts.items():
        wide = 2 * cfg.lanes * h.d
        bufs[k] = dict(frontier=rnd(cfg, (B, F, wide), 11 + ord(k)),
                       proj=torch.full((B, T, wide), SENTINEL, dtype=cfg.storage, device="cuda"),
                       rows=torch.full((B, T, h.d), SENTINEL, dtype=cfg.storage, device="cuda"))
    before = {k: v["frontier"].clone() for k, v in bufs.items()}
    index = {} if "i" not in hosts else dict(comp_i=G.lib_comp(hosts["i"]), frontier_i=bufs["i"]["frontier"],
                                             proj_i=bufs["i"]["proj"], rows_i=bufs["i"]["rows"])
    err = csa.compress_tree(G.lib_layer(cfg), G.lib_comp(hosts["a"]), x, parents(trees, T),
                            torch.tensor(pos, dtype=torch.int32, device="cuda"), bufs["a"]["frontier"],
                            bufs["a"]["proj"], bufs["a"]["rows"], freqs(cfg), **index)
    assert err.item() == 0
    for k, h in hosts.items():
        comp, b_ = oracle_comp(h), bufs[k]
        assert torch.equal(b_["frontier"], before[k])  # the cache is read only
        proj, rows, Ld = f64(b_["proj"]), f64(b_["rows"]), cfg.lanes * h.d
        kv_o, g_o = O.project(layer, comp, f64(x))
        ax = np.abs(f64(x))
        abs_dot = np.concatenate([ax @ np.abs(comp.wkv).T, ax @ np.abs(comp.wgate).T], -1)
        ref = np.concatenate([kv_o, g_o], -1)
        for b in range(B):
            for i, path in enumerate(TR.paths(TR.padded(trees[b], T))):
                if path is None:
                    assert (proj[b, i] == SENTINEL).all() and (rows[b, i] == SENTINEL).all()
                    continue
                G.check_projection(proj[b, i], ref[b, i], abs_dot[b, i], cfg.dtype)
                p = pos[b] + len(path) - 1
                if (p + 1) % cfg.ratio:
                    assert (rows[b, i] == SENTINEL).all()
                    continue
                # the row that sequential compression of the path emits last
                n0, cap = pos[b] // cfg.ratio, (p + 1) // cfg.ratio
                _, pool, n, e = O.compress_append(layer, comp, f64(x[b])[path][None], [pos[b]], f64(before[k][b:b + 1]),
                                                  np.zeros((1, cap, h.d)), [n0], invf,
                                                  proj=(proj[b][path][None, :, :Ld], proj[b][path][None, :, Ld:]))
                assert e == 0 and n[0] == cap
                G.check_pool_rows(rows[b, i], pool[0, cap - 1], cfg.dtype, f"{k} seq {b} node {i}", R=cfg.R)


def test_compress_tree_fp8_index_rows():
    """With index_fp8 the index rows are the fp8 rows of the ones that the plain layer writes."""
    cfg = FLASH
    trees, pos = [TR.bushy(12), TR.chain(9)], torch.tensor([6, 4001], dtype=torch.int32, device="cuda")
    par = parents(trees)
    ca, ci = (G.lib_comp(csa_synth.compressor(cfg, w)) for w in ("attn", "index"))
    x = rnd(cfg, (2, 12, cfg.X), 20)
    fa, fi = rnd(cfg, (2, 8, 2048), 21), rnd(cfg, (2, 8, 512), 22)
    got = {}
    for fp8 in (False, True):
        L = dataclasses.replace(G.lib_layer(cfg), index_fp8=fp8)
        rows_i = (torch.zeros(2, 12, csa.FP8_ROW_BYTES, dtype=torch.uint8, device="cuda") if fp8
                  else torch.zeros(2, 12, 128, dtype=torch.bfloat16, device="cuda"))
        z = lambda n: torch.zeros(2, 12, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        err = csa.compress_tree(L, ca, x, par, pos, fa, z(2048), z(512), freqs(cfg), comp_i=ci, frontier_i=fi,
                                proj_i=z(512), rows_i=rows_i)
        assert err.item() == 0
        got[fp8] = rows_i
    want = torch.zeros_like(got[True])
    csa.index_rows_fp8(dataclasses.replace(G.lib_layer(cfg), index_fp8=True), got[False], want)
    live = got[False].any(-1)
    assert live.any() and torch.equal(got[True][live], want[live]) and not got[True][~live].any()


# ------------------------------------------------------------------------------------------------ index_scores_tree

SC_CASES = {
    "flash": ("flash", [TR.bushy(16), TR.bushy(14, 2), TR.chain(16)], [4097, 3, 1030]),
    "flash_t1": ("flash", [[-1], [-1]], [2047, 0]),
    "flash_t64": ("flash", [TR.bushy(64)], [2050]),
    "flash_t13": ("flash", [TR.bushy(13)] * 5, [515, 512, 511, 6001, 129]),
    "tiny_f32": ("tiny_f32", [TR.bushy(9), TR.star(9)], [63, 200]),
    "odd_bf16": ("odd_bf16", [TR.binary(10), TR.chain(3)], [50, 7]),
}


@pytest.mark.parametrize("case", list(SC_CASES))
def test_index_scores_tree_against_float64(case):
    name, trees, pos = SC_CASES[case]
    cfg = LAYERS[name]
    B, T, cap = len(trees), max(len(t) for t in trees), max(pos) // cfg.ratio + 3
    layer = oracle_layer(cfg)
    iq, iw = rnd(cfg, (B, T, cfg.Hi, cfg.Di), 30), rnd(cfg, (B, T, cfg.Hi), 31)
    ikeys, rows = rnd(cfg, (B, cap, cfg.Di), 32), rnd(cfg, (B, T, cfg.Di), 33)
    for b in range(B):  # what no node may read: rows behind the last committed one, rows that no node completes
        ikeys[b, pos[b] // cfg.ratio:] = float("nan")
        for i, path in enumerate(TR.paths(TR.padded(trees[b], T))):
            if path is None or (pos[b] + len(path)) % cfg.ratio:
                rows[b, i] = float("nan")
    scores = torch.full((B, T, cap + T), SENTINEL, device="cuda")
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    err = csa.index_scores_tree(G.lib_layer(cfg), iq, iw, ikeys, rows, parents(trees, T), p // cfg.ratio, p, scores)
    assert err.item() == 0
    got = f64(scores)
    for b in range(B):
        n = pos[b] // cfg.ratio
        assert (got[b, :, n + T:] == SENTINEL).all()
        for i, path in enumerate(TR.paths(TR.padded(trees[b], T))):
            if path is None:
                assert (got[b, i] == SENTINEL).all()
                continue
            ref, bound = TR.scores_row(layer, iq[b, i], iw[b, i], torch.nan_to_num(ikeys[b]), torch.nan_to_num(rows[b]),
                                       path, pos[b])
            g = got[b, i, :n + T]
            fin = np.isfinite(ref)
            assert np.array_equal(g[~fin], ref[~fin])
            diff = g[fin] - ref[fin]
            assert (np.abs(diff) <= 2 * (cfg.Di + cfg.Hi + 8) * 2.0 ** -24 * bound[fin]).all()
            assert np.linalg.norm(diff) <= 2.0 ** -18 * max(np.linalg.norm(ref[fin]), 1e-30)


@pytest.mark.parametrize("case", ["flash", "flash_t1", "flash_t64", "flash_t13"])
def test_index_scores_tree_fp8_against_float64(case):
    """Keys as fp8 rows: the codes of the queries are exact (the rotated heads are bf16, as the oracle takes them)."""
    _, trees, pos = SC_CASES[case]
    cfg = FLASH
    B, T, cap = len(trees), max(len(t) for t in trees), max(pos) // 4 + 3
    layer, L = oracle_layer(cfg), dataclasses.replace(G.lib_layer(cfg), index_fp8=True)
    iq, iw = rnd(cfg, (B, T, 64, 128), 230), rnd(cfg, (B, T, 64), 231)
    iq[0, 0, 5] = 0  # a head of zeros: scale 0, zero codes
    src = [rnd(cfg, (B, cap, 128), 232), rnd(cfg, (B, T, 128), 233)]
    src[0][0, 0] = 0
    src[0][0, 1] *= 2.0 ** 40
    ikeys, rows = (torch.zeros(*t.shape[:2], csa.FP8_ROW_BYTES, dtype=torch.uint8, device="cuda") for t in src)
    for t, o in zip(src, (ikeys, rows)):
        csa.index_rows_fp8(L, t, o)
    keys8 = [(o[..., :128].cpu().numpy().astype(np.int64),
              np.ascontiguousarray(o[..., 128:132].cpu().numpy()).view(np.float32)[..., 0]) for o in (ikeys, rows)]
    for b in range(B):  # what no node may read: codes and scales that are NaN
        ikeys[b, pos[b] // 4:] = 0xFF
        for i, path in enumerate(TR.paths(TR.padded(trees[b], T))):
            if path is None or (pos[b] + len(path)) % 4:
                rows[b, i] = 0xFF
    scores = torch.full((B, T, cap + T), SENTINEL, device="cuda")
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    err = csa.index_scores_tree(L, iq, iw, ikeys, rows, parents(trees, T), p // 4, p, scores)
    assert err.item() == 0
    got = f64(scores)
    for b in range(B):
        n = pos[b] // 4
        assert (got[b, :, n + T:] == SENTINEL).all()
        codes = np.concatenate([keys8[0][0][b, :n], keys8[1][0][b]])
        scale = np.concatenate([keys8[0][1][b, :n], keys8[1][1][b]]).astype(np.float64)
        kv = O.e4m3_decode(codes)
        for i, path in enumerate(TR.paths(TR.padded(trees[b], T))):
            if path is None:
                assert (got[b, i] == SENTINEL).all()
                continue
            q = [O.quantize_fp8_row(f64(iq[b, i, h])) for h in range(64)]
            qc, qs = np.stack([c for c, _ in q]), np.array([x for _, x in q], dtype=np.float64)
            ref = O.index_scores_fp8(layer, qc, qs, f64(iw[b, i]), codes, scale)
            w = np.abs(f64(iw[b, i])) * (128 ** -0.5) * (64 ** -0.5) * qs / 128
            bound = (w[:, None] * (np.abs(O.e4m3_decode(qc)) @ np.abs(kv).T)).sum(0) * scale
            seen = np.zeros(n + T, dtype=bool)
            seen[TR.columns(layer, path, pos[b], T)] = True
            g = got[b, i, :n + T]
            assert (g[~seen] == -np.inf).all()
            assert (np.abs(g - ref)[seen] <= 2 * (cfg.Di + cfg.Hi + 8) * 2.0 ** -24 * bound[seen]).all()


def test_tree_step_with_fp8_index_rows():
    """The step and the commit of a layer whose index pool holds fp8 rows: scores on the rows that compress_tree wrote,
    a selection that is theirs, and the accepted rows moved byte for byte."""
    cfg, trees, pos = FLASH, [TR.bushy(9), TR.chain(7)], [2051, 4002]
    d = _step(cfg, trees, pos, 1100, seed=300)
    L = d["L"] = dataclasses.replace(d["L"], index_fp8=True)
    st, T = d["st"], 9
    keys16 = st.ikeys
    st.ikeys = torch.zeros(2, 1100, csa.FP8_ROW_BYTES, dtype=torch.uint8, device="cuda")
    csa.index_rows_fp8(L, keys16, st.ikeys)
    d["rows_i"] = torch.zeros(2, T, csa.FP8_ROW_BYTES, dtype=torch.uint8, device="cuda")
    err = err_word()
    run_step(cfg, d, err)
    assert err.item() == 0
    layer, invf = oracle_layer(cfg), f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    keep = st.ikeys.clone()
    for b in range(2):
        for i, path in enumerate(TR.paths(TR.padded(trees[b], T))):
            if path is not None:
                cols = TR.select(layer, f64(d["scores"][b, i]), path, pos[b], T)
                assert d["sel"][b, i, :len(cols)].tolist() == cols.tolist()
    leaf = [8, 6]
    run_commit(cfg, d, torch.tensor(leaf, dtype=torch.int32, device="cuda"), err)
    assert err.item() == 0
    for b in range(2):
        for k, node in enumerate(TR.paths(trees[b])[leaf[b]]):
            if (pos[b] + k + 1) % 4 == 0:
                keep[b, (pos[b] + k + 1) // 4 - 1] = d["rows_i"][b, node]
                assert d["rows_i"][b, node].any()
    assert torch.equal(st.ikeys, keep)


def test_calls_on_a_given_stream_own_what_they_allocate():
    """stream=: outputs, workspaces and the error word of the call's own are allocated and zeroed on that stream."""
    cfg = FLASH
    d = _step(cfg, [TR.bushy(8)] * 3, [3001, 3200, 57], 900, seed=400)
    st, L = d["st"], d["L"]
    want, side = None, torch.cuda.Stream()
    for stream in (None, side, side):
        side.wait_stream(torch.cuda.current_stream())
        big = torch.randn(4096, 4096, device="cuda")  # work on the current stream that the side stream does not await
        for _ in range(4):
            big = big @ big * 1e-3
        q, kv, iq = csa.norm_rope(L, [d["q"], d["kv"], d["iq"]], st.pos, d["invf"], parent=d["par"],
                                  norm=[True, True, False], stream=stream)
        errs = [csa.compress_tree(L, d["ca"], d["x"], d["par"], st.pos, st.front_attn, d["proj_a"], d["rows_a"],
                                  d["invf"], comp_i=d["ci"], frontier_i=st.front_index, proj_i=d["proj_i"],
                                  rows_i=d["rows_i"], stream=stream),
                csa.index_scores_tree(L, iq, d["iw"], st.ikeys, d["rows_i"], d["par"], d["n_a"], st.pos, d["scores"],
                                      stream=stream),
                csa.attend_tree(L, q, kv, d["sink"], st.window, st.pool, d["rows_a"], d["scores"], d["par"], d["n_a"],
                                st.pos, d["invf"], d["out"], sel_out=d["sel"], stream=stream)]
        torch.cuda.synchronize()
        assert all(e.item() == 0 for e in errs)
        got = [t.clone() for t in (q, kv, iq, d["scores"], d["out"], d["sel"])]
        if want is None:
            want = got
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for k in ("scores", "out", "sel"):
            d[k].zero_()


# ------------------------------------------------------------------------------------------------ attend_tree

AT_CASES = {
    # layer, trees, positions, kind of scores (None: no selection)
    "flash_sparse": ("flash", [TR.bushy(8), TR.bushy(7, 3)], [4097, 2049], "normal"),
    "flash_dense_to_sparse": ("flash", [TR.chain(16)], [2044], "normal"),  # 511 committed rows, up to 515 visible
    "flash_short": ("flash", [TR.bushy(6), [-1], TR.star(6)], [0, 1, 130], "normal"),
    "flash_ties": ("flash", [TR.bushy(5)], [3333], "ties"),
    "flash_extremes": ("flash", [TR.bushy(5), TR.chain(5)], [2803, 2900], "extremes"),
    "flash_all_rows": ("flash", [TR.bushy(4)], [1001], None),
    "flash_many": ("flash", [TR.bushy(16, s) for s in range(12)], [2100 + 37 * s for s in range(12)], "normal"),
    # more nodes than SMs: the selection kernel of many nodes; the last ones see fewer rows than they may keep
    "flash_many_ties": ("flash", [TR.bushy(16, s) for s in range(11)], [2100 + 53 * s for s in range(10)] + [900], "ties"),
    "flash_many_extremes": ("flash", [TR.bushy(32, s) for s in range(6)], [2801, 2300, 2044, 2045, 3000, 7], "extremes"),
    "flash_t64": ("flash", [TR.chain(64), TR.bushy(64)], [2500, 90], "normal"),
    "flash_long": ("flash", [TR.bushy(3)], [70001], "normal"),
    "flash_r128": ("flash_r128", [TR.chain(40), TR.bushy(33)], [120, 30000], None),
    "flash_r128_many": ("flash_r128", [TR.bushy(11, s) for s in range(16)], [127 + 1111 * s for s in range(16)], None),
    "tiny_f32": ("tiny_f32", [TR.bushy(9), TR.chain(9)], [150, 3], "normal"),
    "tiny_f32_r8": ("tiny_f32_r8", [TR.bushy(17)], [99], None),
    "odd_bf16": ("odd_bf16", [TR.binary(12), [-1]], [61, 2], "normal"),
}


def make_scores(cfg, B, T, cap, kind):
    if kind is None:
        return None
    s = rnd(cfg, (B, T, cap + T), 40, dtype=torch.float32)
    if kind == "ties":
        s = (s * 4).round() / 4  # many equal values, both zeros among them
    if kind == "extremes":
        s[..., ::7] = float("-inf")
        s[..., 3::11] = float("inf")
        s[..., 5::13] = torch.finfo(torch.float32).min
    return s


@pytest.mark.parametrize("case", list(AT_CASES))
def test_attend_tree_against_float64(case):
    name, trees, pos, kind = AT_CASES[case]
    cfg = LAYERS[name]
    B, T, cap = len(trees), max(len(t) for t in trees), max(pos) // cfg.ratio + 2
    layer, invf = oracle_layer(cfg), f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    sink = rnd(cfg, (cfg.H,), 41, dtype=torch.float32)
    q, kv = rnd(cfg, (B, T, cfg.H, cfg.D), 42), rnd(cfg, (B, T, cfg.D), 43)
    window, pool = rnd(cfg, (B, cfg.W, cfg.D), 44), rnd(cfg, (B, cap, cfg.D), 45)
    rows = rnd(cfg, (B, T, cfg.D), 46)
    scores = make_scores(cfg, B, T, cap, kind)
    for b in range(B):  # what no node may read
        pool[b, pos[b] // cfg.ratio:] = float("nan")
        if pos[b] < cfg.W:
            window[b, pos[b]:] = float("nan")
        for i, path in enumerate(TR.paths(TR.padded(trees[b], T))):
            if path is None:
                kv[b, i] = q[b, i] = float("nan")
            if path is None or (pos[b] + len(path)) % cfg.ratio:
                rows[b, i] = float("nan")
                if scores is not None:
                    scores[b, :, pos[b] // cfg.ratio + i] = float("nan")
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    out = torch.full((B, T, cfg.H, cfg.D), SENTINEL, dtype=cfg.storage, device="cuda")
    sel = None if scores is None else torch.full((B, T, cfg.topk), -9, dtype=torch.int32, device="cuda")
    state = [t.clone() for t in (kv, window, pool, rows)]
    err = csa.attend_tree(G.lib_layer(cfg), q, kv, sink, window, pool, rows, scores, parents(trees, T),
                          p // cfg.ratio, p, freqs(cfg), out, sel_out=sel)
    assert err.item() == 0
    for a, b_ in zip(state, (kv, window, pool, rows)):  # read only, bit for bit
        assert torch.equal(a.view(torch.uint8), b_.view(torch.uint8))
    check_tree_outputs(cfg, layer, trees, pos, q, kv, sink, window, pool, rows, scores, out, sel, invf)


def check_tree_outputs(cfg, layer, trees, pos, q, kv, sink, window, pool, rows, scores, out, sel, invf, sampled=24):
    B, T = out.shape[:2]
    todo = [(b, i) for b in range(B) for i in range(T)]
    step = max(1, len(todo) // sampled)
    for k, (b, i) in enumerate(todo):
        path = TR.paths(TR.padded(trees[b], T))[i]
        if path is None:
            assert (out[b, i] == SENTINEL).all() and (sel is None or (sel[b, i] == -9).all())
            continue
        cols = TR.select(layer, None if scores is None else f64(scores[b, i]), path, pos[b], T)
        if sel is not None:
            got = sel[b, i].cpu().numpy()
            assert got[:len(cols)].tolist() == cols.tolist() and (got[len(cols):] == -1).all(), (b, i)
        if k % step and i != T - 1:
            continue
        ref = TR.output(layer, q[b, i], kv[b], f64(sink), window[b], pool[b], rows[b], cols, path, pos[b], invf)
        g = f64(out[b, i])
        tol = (2.0 ** -11 if cfg.dtype == "bf16" else 1e-5) * np.abs(ref).max(-1, keepdims=True)
        bad = np.abs(g - ref) > half_step(np.abs(ref) + tol, cfg.dtype) + tol
        assert not bad.any(), (b, i, np.argwhere(bad)[:3], np.abs(g - ref).max())


EDGE_CASES = {
    # layer, trees, positions, selection: nodes whose keys a cluster of CTAs shares (all rows wanted; some nodes with
    # fewer tiles than CTAs), more nodes than SMs, splits of a tile (few nodes), odd sizes, the portable kernel
    "flash_rows_8_ways": ("flash", [TR.bushy(3), TR.star(4)], [9001, 5], False),
    "flash_rows_4_ways": ("flash", [TR.bushy(10), TR.chain(14)], [3300, 40], False),
    "flash_rows_2_ways": ("flash", [TR.bushy(20, s) for s in range(3)], [2004, 700, 1], False),
    "flash_left_over": ("flash", [TR.bushy(16, s) for s in range(10)], [2100 + 91 * s for s in range(9)] + [3], True),
    "flash_r128_left_over": ("flash_r128", [TR.bushy(19, s) for s in range(9)],
                             [60000 + 9091 * s for s in range(8)] + [99], False),
    "flash_few": ("flash", [TR.bushy(5), TR.chain(7)], [4097, 2301], True),
    "flash_few_4_splits": ("flash", [TR.bushy(9), TR.chain(8)], [3001, 2051], True),
    "flash_few_short": ("flash", [TR.bushy(7), TR.star(8)], [600, 3], True),
    "flash_many": ("flash", [TR.bushy(16, s) for s in range(11)], [2100 + 91 * s for s in range(11)], True),
    "flash_many_rows": ("flash_r128", [TR.bushy(16, s) for s in range(11)], [9000 + 1291 * s for s in range(11)], False),
    "flash_topk_odd": ("flash_topk", [TR.bushy(15, s) for s in range(12)], [900 + 77 * s for s in range(12)], True),
    "flash_topk_odd_few": ("flash_topk", [TR.bushy(6)], [1403], True),
    "flash_topk_1": ("flash_topk1", [TR.bushy(15, s) for s in range(12)], [77 * s for s in range(12)], True),
    "flash_topk_2048_few": ("flash_topk2048", [TR.bushy(6), TR.chain(5)], [12001, 8100], True),
    "flash_topk_2048_many": ("flash_topk2048", [TR.bushy(16, s) for s in range(10)],
                             [7000 + 997 * s for s in range(10)], True),
    "flash_wide_window_few": ("flash_wide", [TR.bushy(6), TR.chain(8)], [3001, 650], True),
    "flash_wide_window_many": ("flash_wide", [TR.bushy(16, s) for s in range(10)],
                               [300 + 397 * s for s in range(10)], True),
    "flash_window": ("flash_window", [TR.bushy(9, s) for s in range(18)], [801 + 13 * s for s in range(18)], True),
    "tiny_f32": ("tiny_f32", [TR.bushy(9), TR.chain(9)], [150, 70], True),
}
EDGE_LAYERS = {**LAYERS, "flash_topk": FLASH.replace(cid=65, topk=203), "flash_topk1": FLASH.replace(cid=66, topk=1),
               "flash_window": FLASH.replace(cid=67, W=77, topk=131, rollback=19),
               "flash_topk2048": FLASH.replace(cid=68, topk=2048), "flash_wide": FLASH.replace(cid=69, W=700, topk=300)}


@pytest.mark.parametrize("case", list(EDGE_CASES))
@pytest.mark.parametrize("loud", [1.0, 24.0])
def test_attend_tree_sinks_and_large_logits(case, loud):
    """Sinks from -infinity to far above every logit, and logits that grow along the keys, so that a head's largest one
    is found late and far above both the sink and everything before it.

    A logit is 512 products summed in fp32, by a pipe that may truncate: 32 steps of 16 products, each off by up to
    2^-23 of the sum of absolute products A; the scale and the reference that is taken from it round three times more,
    2^-22 of |logit| and of the reference.  With e the largest such error over a node's keys (in natural units), the
    probabilities err by 2 e + 2^-14 relative (2^-16 for two bf16 parts, the exponential and the sums), the average by
    that times the largest |key value|."""
    name, trees, pos, select = EDGE_CASES[case]
    cfg = EDGE_LAYERS[name]
    B, T, cap = len(trees), max(len(t) for t in trees), max(pos) // cfg.ratio + 2
    layer, invf = oracle_layer(cfg), f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    sink = rnd(cfg, (cfg.H,), 141, dtype=torch.float32)
    for h, v in enumerate((float("-inf"), -3e38, -1e4, -200.0, 0.0, 150.0, 1e4)):
        sink[h % cfg.H::cfg.H // 4] = v
    q, kv = rnd(cfg, (B, T, cfg.H, cfg.D), 142, scale=loud), rnd(cfg, (B, T, cfg.D), 143)
    ramp = torch.linspace(0.05, 2.0, cap, device="cuda")[None, :, None]
    window = rnd(cfg, (B, cfg.ring_slots, cfg.D), 144)
    pool = (rnd(cfg, (B, cap, cfg.D), 145).float() * ramp).to(cfg.storage)
    rows = rnd(cfg, (B, T, cfg.D), 146)
    scores = make_scores(cfg, B, T, cap, "normal" if select else None)
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    out = torch.full((B, T, cfg.H, cfg.D), SENTINEL, dtype=cfg.storage, device="cuda")
    again = out.clone()
    for o in (out, again):
        err = csa.attend_tree(G.lib_layer(cfg), q, kv, sink, window, pool, rows, scores, parents(trees, T),
                              p // cfg.ratio, p, freqs(cfg), o)
        assert err.item() == 0
    assert torch.equal(out, again)
    scale = cfg.D ** -0.5
    for b in range(0, B, max(1, B // 4)):
        for i in (0, T // 2, T - 1):
            path = TR.paths(TR.padded(trees[b], T))[i]
            if path is None:
                continue
            cols = TR.select(layer, None if scores is None else f64(scores[b, i]), path, pos[b], T)
            args = (layer, q[b, i], kv[b], f64(sink), window[b], pool[b], rows[b], cols, path, pos[b], invf)
            ref, keys = TR.output(*args), TR.keys(*args)
            dot, absdot = f64(q[b, i]) @ keys.T * scale, np.abs(f64(q[b, i])) @ np.abs(keys).T * scale
            e = 32 * 2.0 ** -23 * absdot.max(-1) + 2.0 ** -22 * (np.abs(dot).max(-1) + 100)
            tol = ((2 * e + 2.0 ** -14) * 2 * np.abs(keys).max())[:, None]
            g = f64(out[b, i])
            bad = np.abs(g - ref) > half_step(np.abs(ref) + tol, cfg.dtype) + tol
            assert np.isfinite(g).all() and not bad.any(), (b, i, np.argwhere(bad)[:3], np.abs(g - ref).max())


def test_attend_tree_with_unused_sequences_and_long_pools():
    """A batch whose sequences are all padding but two, one of which sees far more rows than a block's shared memory
    holds scores for; the padding's outputs stay as they were."""
    cfg = FLASH
    for B, T, long in ((3, 4, 60000), (12, 14, 20000)):
        trees = [[TR.NONE] * T for _ in range(B)]
        trees[0], trees[B - 1] = TR.bushy(T), TR.chain(T)
        pos = [0] * B
        pos[0], pos[B - 1] = 4 * long + 2, 30
        cap = long + 1
        layer, invf = oracle_layer(cfg), f64(csa_synth.inv_freq(cfg)).astype(np.float32)
        g = torch.Generator(device="cuda").manual_seed(5)
        q = torch.randn(B, T, 64, 512, device="cuda", generator=g).bfloat16()
        kv = torch.randn(B, T, 512, device="cuda", generator=g).bfloat16()
        window = torch.randn(B, 128, 512, device="cuda", generator=g).bfloat16()
        pool = torch.randn(1, cap, 512, device="cuda", generator=g).bfloat16().expand(B, cap, 512).contiguous()
        rows = torch.randn(B, T, 512, device="cuda", generator=g).bfloat16()
        scores = torch.randn(B, T, cap + T, device="cuda", generator=g)
        sink = rnd(cfg, (64,), 150, dtype=torch.float32)
        p = torch.tensor(pos, dtype=torch.int32, device="cuda")
        out = torch.full((B, T, 64, 512), SENTINEL, dtype=torch.bfloat16, device="cuda")
        sel = torch.full((B, T, 512), -9, dtype=torch.int32, device="cuda")
        err = csa.attend_tree(G.lib_layer(cfg), q, kv, sink, window, pool, rows, scores, parents(trees, T), p // 4, p,
                              freqs(cfg), out, sel_out=sel)
        assert err.item() == 0
        check_tree_outputs(cfg, layer, trees, pos, q, kv, sink, window, pool, rows, scores, out, sel, invf)


@pytest.mark.parametrize("T", [2, 40])
def test_attend_tree_rows_past_32_bit_offsets(T):
    """Two pools of 2.2 million rows (2.25e9 values): a few nodes (split kernel) and many (a CTA each)."""
    cfg, B, cap = FLASH, 2, 2200000
    layer, invf = oracle_layer(cfg), f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    trees, pos = [TR.chain(T), TR.bushy(T)], [4 * cap - 4 * T - 3, 4 * cap - 4 * T - 2]
    g = torch.Generator(device="cuda").manual_seed(9)
    n = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    pool, q, kv, window, rows = n(B, cap, 512), n(B, T, 64, 512), n(B, T, 512), n(B, 128, 512), n(B, T, 512)
    scores = torch.empty(B, T, cap + T, device="cuda").normal_(generator=g)
    sink = rnd(cfg, (64,), 160, dtype=torch.float32)
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    out, sel = torch.empty_like(q), torch.empty(B, T, 512, dtype=torch.int32, device="cuda")
    err = csa.attend_tree(G.lib_layer(cfg), q, kv, sink, window, pool, rows, scores, parents(trees, T), p // 4, p,
                          freqs(cfg), out, sel_out=sel)
    assert err.item() == 0
    for b in range(B):
        for i in (0, T - 1):
            path = TR.paths(trees[b])[i]
            seen = torch.full((cap + T,), float("-inf"), device="cuda")
            cols = TR.columns(layer, path, pos[b], T)
            cols = torch.tensor(cols[pos[b] // 4:], device="cuda", dtype=torch.long)  # the path's rows
            seen[:pos[b] // 4] = scores[b, i, :pos[b] // 4]
            seen[cols] = scores[b, i, cols]
            top = seen.topk(cfg.topk).indices.sort().values
            assert torch.equal(sel[b, i].long(), top) and top.max() > cap // 2
            ref = TR.output(layer, q[b, i], kv[b], f64(sink), window[b], pool[b], rows[b], top.tolist(), path, pos[b],
                            invf)
            tol = 2.0 ** -11 * np.abs(ref).max(-1, keepdims=True)
            assert (np.abs(f64(out[b, i]) - ref) <= half_step(np.abs(ref) + tol, cfg.dtype) + tol).all(), (b, i)


def test_attend_tree_of_a_chain_is_a_verify_block():
    """A tree without branches against csa_attend_verify on the same tokens and selections."""
    B, T = 3, 4
    cfg = FLASH.replace(B=B, rollback=T, ctx=2803)
    host = csa_synth.synth_cache(cfg, 720, B=B)
    st, L = G.DevCache(host), G.lib_layer(cfg)
    sink, invf = csa_synth.sinks(cfg).cuda(), freqs(cfg)
    q, kv = rnd(cfg, (B, T, 64, 512), 50), rnd(cfg, (B, T, 512), 51)
    rows = rnd(cfg, (B, T, 512), 52)
    n0 = 2803 // 4
    par = parents([TR.chain(T)] * B)
    scores = rnd(cfg, (B, T, 720 + T), 53, dtype=torch.float32)
    tq, tkv = csa.norm_rope(L, [q, kv], st.pos, invf, parent=par, norm=[False, False])
    out, sel = torch.empty_like(q), torch.empty(B, T, 512, dtype=torch.int32, device="cuda")
    err = csa.attend_tree(L, tq, tkv, sink, st.window, st.pool, rows, scores, par, st.n_rows, st.pos, invf, out,
                          sel_out=sel)
    # position 2803 completes row 700: node 0's row; the verify call finds it at its place in the pool
    st.pool[:, n0] = rows[:, 0]
    out_v = torch.empty_like(q)
    err2 = csa.attend_verify(L, q, kv, sink, st.window, st.pool, st.n_rows + 1, sel,
                             torch.full((B, T), 512, dtype=torch.int32, device="cuda"), st.pos, invf, out_v)
    assert err.item() == 0 and err2.item() == 0 and (sel <= n0).all() and (sel == n0).any()
    a, b = f64(out), f64(out_v)
    # the verify call rounds its output once more before the rotation
    assert (np.abs(a - b) <= 2.0 ** -10 * np.abs(b).max(-1, keepdims=True) + 2 * G.ulp(b, "bf16") +
            2 * G.ulp(np.repeat(np.hypot(b[..., ::2], b[..., 1::2]), 2, -1), "bf16")).all()


# ------------------------------------------------------------------------------------------------ commit_tree

CM_CASES = {
    # layer, trees, positions, accepted leaves
    "flash": ("flash", [TR.bushy(16), TR.bushy(16, 4), TR.chain(16), TR.star(3)], [4097, 2046, 0, 9], [15, -1, 15, 2]),
    "flash_long_path": ("flash", [TR.chain(64)], [126], [63]),
    "flash_r128": ("flash_r128", [TR.chain(64), TR.bushy(20)], [100, 4095], [50, 0]),
    "tiny_f32": ("tiny_f32", [TR.chain(64), TR.bushy(30)], [17, 0], [63, 29]),  # a path longer than the rings
    "odd_bf16": ("odd_bf16", [TR.binary(31), [-1]], [5, 3], [30, 0]),
    "odd_bf16_rollback": ("odd_bf16_rb", [TR.chain(40)], [33], [39]),
}


@pytest.mark.parametrize("case", list(CM_CASES))
@pytest.mark.parametrize("in_place", [True, False])
def test_commit_tree(case, in_place):
    name, trees, pos, leaf = CM_CASES[case]
    cfg = ODD.replace(cid=64, rollback=11) if name == "odd_bf16_rb" else LAYERS[name]
    B, T, cap = len(trees), max(len(t) for t in trees), max(pos) // cfg.ratio + 64 // cfg.ratio + 1
    dims = {"a": cfg.D, "i": cfg.Di} if cfg.has_indexer else {"a": cfg.D}
    kv, window = rnd(cfg, (B, T, cfg.D), 60), rnd(cfg, (B, cfg.ring_slots, cfg.D), 61)
    s = {k: dict(proj=rnd(cfg, (B, T, 2 * cfg.lanes * d), 62 + ord(k)), rows=rnd(cfg, (B, T, d), 63 + ord(k)),
                 frontier=rnd(cfg, (B, cfg.frontier_slots, 2 * cfg.lanes * d), 64 + ord(k)),
                 pool=rnd(cfg, (B, cap, d), 65 + ord(k))) for k, d in dims.items()}
    want_win = window.clone()
    want = {k: dict(frontier=v["frontier"].clone(), pool=v["pool"].clone()) for k, v in s.items()}
    end = []
    for b in range(B):
        path = [] if leaf[b] < 0 else TR.paths(trees[b])[leaf[b]]
        for k, node in enumerate(path):
            t = pos[b] + k
            want_win[b, t % cfg.ring_slots] = kv[b, node]
            for g in dims:
                want[g]["frontier"][b, t % cfg.frontier_slots] = s[g]["proj"][b, node]
                if (t + 1) % cfg.ratio == 0:
                    want[g]["pool"][b, (t + 1) // cfg.ratio - 1] = s[g]["rows"][b, node]
        end.append(pos[b] + len(path))
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    n = {k: p // cfg.ratio for k in dims}
    outs = dict(pos_out=torch.zeros_like(p), n_rows_a_out=torch.zeros_like(p))
    index = {}
    if "i" in dims:
        outs["n_rows_i_out"] = torch.zeros_like(p)
        index = dict(n_rows_i=n["i"], **{f"{f}_i": s["i"][f] for f in ("proj", "frontier", "rows", "pool")})
    if in_place:
        outs = {}
    err = csa.commit_tree(G.lib_layer(cfg), parents(trees, T), torch.tensor(leaf, dtype=torch.int32, device="cuda"), p,
                          n["a"], kv, window, s["a"]["proj"], s["a"]["frontier"], s["a"]["rows"], s["a"]["pool"],
                          **index, **outs)
    assert err.item() == 0
    assert torch.equal(window, want_win)
    for g in dims:
        assert torch.equal(s[g]["frontier"], want[g]["frontier"]) and torch.equal(s[g]["pool"], want[g]["pool"])
        got_n = n[g] if in_place else outs[f"n_rows_{g}_out"]
        assert got_n.tolist() == [e // cfg.ratio for e in end]
    assert (p if in_place else outs["pos_out"]).tolist() == end
    if not in_place:
        assert p.tolist() == pos


# ------------------------------------------------------------------------------------------------ device-side refusals


def _step(cfg, trees, pos, cap, seed=0, layer_kw=None):
    """Everything that one tree step of the layer needs, on the device."""
    B, T = len(trees), max(len(t) for t in trees)
    host = csa_synth.synth_cache(cfg.replace(cid=cfg.cid + 900 + seed, B=B, ctx=max(pos)), cap, B=B)
    st = G.DevCache(host)
    st.pos = torch.tensor(pos, dtype=torch.int32, device="cuda")
    st.n_rows = st.pos // cfg.ratio
    z = lambda *s, dt=cfg.storage: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    d = dict(L=G.lib_layer(cfg), st=st, par=parents(trees, T), invf=freqs(cfg), sink=csa_synth.sinks(cfg).cuda(),
             x=rnd(cfg, (B, T, cfg.X), 70 + seed), q=rnd(cfg, (B, T, cfg.H, cfg.D), 71 + seed),
             kv=rnd(cfg, (B, T, cfg.D), 72 + seed), iq=rnd(cfg, (B, T, cfg.Hi, cfg.Di), 73 + seed),
             iw=rnd(cfg, (B, T, cfg.Hi), 74 + seed), ca=G.lib_comp(csa_synth.compressor(cfg, "attn")),
             proj_a=z(B, T, 2 * cfg.lanes * cfg.D), rows_a=z(B, T, cfg.D), out=z(B, T, cfg.H, cfg.D),
             n_a=st.n_rows.clone(), n_i=st.n_rows.clone())
    d["q2"], d["kv2"], d["iq2"] = torch.zeros_like(d["q"]), torch.zeros_like(d["kv"]), torch.zeros_like(d["iq"])
    if cfg.has_indexer:
        d.update(ci=G.lib_comp(csa_synth.compressor(cfg, "index")), proj_i=z(B, T, 2 * cfg.lanes * cfg.Di),
                 rows_i=z(B, T, cfg.Di), scores=z(B, T, cap + T, dt=torch.float32),
                 sel=torch.zeros(B, T, cfg.topk, dtype=torch.int32, device="cuda"))
    return d


def run_step(cfg, d, err, ws=None):
    """norm_rope, compress_tree, index_scores_tree, attend_tree: what a verification runs before its logits."""
    st, ws = d["st"], ws or {}
    xs, outs, norm = [d["q"], d["kv"]], [d["q2"], d["kv2"]], [True, True]
    if cfg.has_indexer:
        xs, outs, norm = xs + [d["iq"]], outs + [d["iq2"]], norm + [False]
    csa.norm_rope(d["L"], xs, st.pos, d["invf"], parent=d["par"], norm=norm, outs=outs, err=err)
    index = {} if not cfg.has_indexer else dict(comp_i=d["ci"], frontier_i=st.front_index, proj_i=d["proj_i"],
                                                rows_i=d["rows_i"])
    csa.compress_tree(d["L"], d["ca"], d["x"], d["par"], st.pos, st.front_attn, d["proj_a"], d["rows_a"], d["invf"],
                      **index, ws=ws.get("c"), err=err)
    if cfg.has_indexer:
        csa.index_scores_tree(d["L"], d["iq2"], d["iw"], st.ikeys, d["rows_i"], d["par"], d["n_a"], st.pos,
                              d["scores"], err=err)
    csa.attend_tree(d["L"], d["q2"], d["kv2"], d["sink"], st.window, st.pool, d["rows_a"], d.get("scores"), d["par"],
                    d["n_a"], st.pos, d["invf"], d["out"], sel_out=d.get("sel"), ws=ws.get("a"), err=err)


def run_commit(cfg, d, leaf, err):
    st = d["st"]
    index = {} if not cfg.has_indexer else dict(n_rows_i=d["n_i"], proj_i=d["proj_i"], frontier_i=st.front_index,
                                                rows_i=d["rows_i"], pool_i=st.ikeys)
    csa.commit_tree(d["L"], d["par"], leaf, st.pos, d["n_a"], d["kv2"], st.window, d["proj_a"], st.front_attn,
                    d["rows_a"], st.pool, **index, err=err)


def test_bad_parents_and_states_are_flagged_and_skipped():
    cfg = TINY
    trees = [TR.bushy(8), TR.bushy(8), TR.bushy(8), TR.bushy(8)]
    d = _step(cfg, trees, [50, 60, 70, 80], 60)
    good = _step(cfg, trees, [50, 60, 70, 80], 60)
    run_step(cfg, good, err_word())
    d["par"][0, 3] = 3        # its own parent
    d["par"][1, 2] = -7       # an unused slot ...
    d["par"][1, 5] = 2        # ... with a node under it
    d["n_a"][2] += 1          # row count and position disagree
    for t in (d["out"], d["scores"], d["rows_a"], d["proj_a"]):
        t.fill_(SENTINEL)
    err = err_word()
    run_step(cfg, d, err)
    assert err.item() == csa.DEV_STATE
    dead0 = [i for i, pt in enumerate(TR.paths(trees[0])) if 3 in pt]
    assert 3 in dead0 and (d["out"][0, dead0] == SENTINEL).all() and (d["scores"][0, dead0] == SENTINEL).all()
    assert (d["out"][1, [2, 5]] == SENTINEL).all()
    assert (d["out"][2] == SENTINEL).all() and (d["scores"][2] == SENTINEL).all()
    assert torch.equal(d["out"][3], good["out"][3]) and torch.equal(d["scores"][3][:, :28], good["scores"][3][:, :28])
    # commits: a leaf that is no node, an unused slot, a bad tree, a wrong row count: nothing changes
    st = d["st"]
    keep = [t.clone() for t in (st.window, st.pool, st.ikeys, st.front_attn, st.front_index, st.pos, d["n_a"], d["n_i"])]
    for leaf in ([1, 2, 0, 8], [0, -2, 0, 99]):
        e = err_word()
        run_commit(cfg, d, torch.tensor(leaf, dtype=torch.int32, device="cuda"), e)
        assert e.item() == csa.DEV_STATE
        for a, b in zip(keep, (st.window, st.pool, st.ikeys, st.front_attn, st.front_index, st.pos, d["n_a"], d["n_i"])):
            assert torch.equal(a, b)


def test_commit_beyond_the_pool_is_refused():
    cfg = TINY
    d = _step(cfg, [TR.chain(8), TR.chain(8)], [58, 40], 15)
    run_step(cfg, d, err_word())
    st = d["st"]
    keep = [t.clone() for t in (st.window, st.pool, st.ikeys, st.front_attn)]
    e = err_word()
    run_commit(cfg, d, torch.tensor([7, 7], dtype=torch.int32, device="cuda"), e)  # 66 tokens: 16 rows of a pool of 15
    assert e.item() == csa.DEV_CAPACITY and st.pos.tolist() == [58, 48] and d["n_a"].tolist() == [14, 12]
    for a, b in zip(keep, (st.window, st.pool, st.ikeys, st.front_attn)):
        assert torch.equal(a[0], b[0]) and not torch.equal(a[1], b[1])


# ------------------------------------------------------------------------------------------------ the step as a whole

PIPE_CASES = {
    "flash": ("flash", [TR.bushy(8), TR.bushy(6, 1), TR.chain(8)], [2045, 4098, 515]),
    "flash_r128": ("flash_r128", [TR.bushy(8), TR.chain(8)], [1150, 380]),
    "tiny_f32": ("tiny_f32", [TR.bushy(12), TR.chain(9), TR.star(4)], [61, 0, 130]),
}


@pytest.mark.parametrize("case", list(PIPE_CASES))
def test_tree_steps_then_decode(case):
    """Three speculative steps, each verified node by node, with the accepted paths committed and checked against
    sequential decoding by the library's own single-token calls on a second cache; then both caches decode on."""
    name, trees, pos = PIPE_CASES[case]
    cfg = LAYERS[name]
    B, T = len(trees), max(len(t) for t in trees)
    cap = max(pos) // cfg.ratio + 40
    layer, invf = oracle_layer(cfg), f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    d = _step(cfg, trees, pos, cap)
    st = d["st"]
    ref = {k: getattr(st, k).clone() if getattr(st, k) is not None else None
           for k in ("pool", "ikeys", "window", "front_attn", "front_index", "pos", "n_rows")}
    err = err_word()
    for step in range(3):
        for k, t in (("x", 80), ("q", 81), ("kv", 82), ("iq", 83), ("iw", 84)):
            d[k] = rnd(cfg, tuple(d[k].shape), t + 10 * step)
        d["out"].fill_(SENTINEL)
        if "sel" in d:
            d["sel"].fill_(-9)
        run_step(cfg, d, err)
        assert err.item() == 0
        now = st.pos.tolist()
        check_tree_outputs(cfg, layer, trees, now, d["q2"], d["kv2"], d["sink"], st.window, st.pool, d["rows_a"],
                           d.get("scores"), d["out"], d.get("sel"), invf)
        leaf = [len(trees[b]) - 1 - (step + b) % 3 for b in range(B)]
        if step == 1:
            leaf[1] = -1
        run_commit(cfg, d, torch.tensor(leaf, dtype=torch.int32, device="cuda"), err)
        assert err.item() == 0
        # the same tokens one at a time
        L = d["L"]
        for b in range(B):
            path = [] if leaf[b] < 0 else TR.paths(trees[b])[leaf[b]]
            one = {k: None if v is None else v[b:b + 1] for k, v in ref.items()}
            for node in path:
                xb = d["x"][b:b + 1, node:node + 1].contiguous()
                nq, nkv = csa.norm_rope(L, [d["q"][b:b + 1, node:node + 1], d["kv"][b:b + 1, node:node + 1]])
                e1 = csa.compress_append(L, d["ca"], xb, one["pos"], one["front_attn"], one["pool"], one["n_rows"],
                                         d["invf"])
                assert e1.item() == 0
                out1 = torch.empty(1, cfg.H, cfg.D, dtype=cfg.storage, device="cuda")
                sel1 = n_sel1 = None
                if cfg.has_indexer:
                    n_i = one["pos"] // cfg.ratio
                    e2 = csa.compress_append(L, d["ci"], xb, one["pos"], one["front_index"], one["ikeys"], n_i,
                                             d["invf"])
                    sel1 = torch.empty(1, cfg.topk, dtype=torch.int32, device="cuda")
                    n_sel1 = torch.empty(1, dtype=torch.int32, device="cuda")
                    e3 = csa.index_topk(L, d["iq"][b:b + 1, node].contiguous(), d["iw"][b:b + 1, node].contiguous(),
                                        one["ikeys"], one["n_rows"], one["pos"], d["invf"], sel1, n_sel1)
                    assert e2.item() == 0 and e3.item() == 0
                e4 = csa.attend_decode(L, nq[:, 0].contiguous(), nkv[:, 0].contiguous(), d["sink"], one["window"],
                                       one["pool"], one["n_rows"], sel1, n_sel1, one["pos"], d["invf"], out1)
                assert e4.item() == 0
                csa.advance_positions(one["pos"], 1)
            for k, v in one.items():
                if v is not None:
                    ref[k][b:b + 1] = v
        assert st.pos.tolist() == ref["pos"].tolist() and d["n_a"].tolist() == ref["n_rows"].tolist()
        for got, want, what in ((st.window, ref["window"], "window"), (st.front_attn, ref["front_attn"], "frontier"),
                                (st.front_index, ref["front_index"], "index frontier")):
            if got is None:
                continue
            # A projection may round to the neighbouring value.  A window row of decoding is rounded between its norm
            # and its rotation, here it is not: each value of the pair is off by up to half a step h there, both by up to
            # sqrt(2) h of the pair's norm after the rotation, which is under one step of it; then either side rounds
            # once more, half a step of its value each.
            g, w = f64(got), f64(want)
            pair = np.repeat(np.hypot(w[..., ::2], w[..., 1::2]), 2, axis=-1)
            tol = 2 * G.ulp(np.abs(w), cfg.dtype) + (2.0 ** -12 if cfg.dtype == "bf16" else 1e-5) * np.abs(w).max()
            tol = tol + (G.ulp(pair, cfg.dtype) if what == "window" else 0)
            assert (np.abs(g - w) <= tol).all(), what
        for got, want, n in ((st.pool, ref["pool"], d["n_a"]), (st.ikeys, ref["ikeys"], d["n_i"])):
            if got is None:
                continue
            for b in range(B):
                m = int(n[b])
                g, w = f64(got[b, :m]), f64(want[b, :m])
                # a flipped projection moves a pooled value by up to one step of its entry
                tol = 2.0 ** -6 if cfg.dtype == "bf16" else 1e-4
                assert (np.abs(g - w) <= tol * np.abs(w).max()).all()
                assert (g == w).mean() > (0.98 if cfg.dtype == "bf16" else 0.2)


def test_graph_replay_other_stream_and_two_graphs():
    """The step captured and replayed on changed inputs, two graphs alternating with workspaces of their own, and the
    step on a side stream: the eager call's bits."""
    cfg = FLASH
    trees, pos = [TR.bushy(8), TR.bushy(5, 2)], [3001, 700]
    ds = [_step(cfg, trees, pos, 800, seed=s) for s in (0, 100)]
    errs = [err_word(), err_word()]
    T = 8
    wss = [dict(c=torch.empty(csa.workspace_size(d["L"], csa.OP_COMPRESS_TREE, 2, T, 1), dtype=torch.uint8,
                              device="cuda"),
                a=torch.empty(max(256, csa.workspace_size(d["L"], csa.OP_ATTEND_TREE, 2, T, 800)), dtype=torch.uint8,
                              device="cuda")) for d in ds]
    want = []
    for d, e, w in zip(ds, errs, wss):
        run_step(cfg, d, e, w)
        want.append([d[k].clone() for k in ("out", "sel", "scores", "rows_a", "rows_i", "proj_a")])
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for d, e, w in zip(ds, errs, wss):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                run_step(cfg, d, e, w)
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for d in ds:
            for k in ("out", "scores"):
                d[k].zero_()
            d["sel"].zero_()
        torch.cuda.synchronize()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for d, w in zip(ds, want):
            for k, t in zip(("out", "sel", "scores", "rows_a", "rows_i", "proj_a"), w):
                assert torch.equal(d[k], t), k
    # the replayed graph takes what its inputs hold then
    ds[0]["q"].copy_(ds[1]["q"])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert not torch.equal(ds[0]["out"], want[0][0])
    got = ds[0]["out"].clone()
    with torch.cuda.stream(side):
        ds[0]["out"].zero_()
        run_step(cfg, ds[0], errs[0], wss[0])
    torch.cuda.synchronize()
    assert torch.equal(ds[0]["out"], got) and errs[0].item() == 0 and errs[1].item() == 0


def test_commit_right_after_projections_that_complete_nothing():
    """No node completes a window, so that only the projections take long: a commit enqueued right behind them takes
    what they wrote."""
    cfg = FLASH
    B, T = 32, 16
    d = _step(cfg, [TR.star(T)] * B, [4 * b + 4 for b in range(B)], 40)
    leaf = torch.tensor([b % T for b in range(B)], dtype=torch.int32, device="cuda")
    st = d["st"]
    pos0, na, ni = st.pos.clone(), d["n_a"].clone(), d["n_i"].clone()
    for _ in range(20):
        for t in (d["proj_a"], d["proj_i"]):
            t.fill_(SENTINEL)
        for t, v in ((st.pos, pos0), (d["n_a"], na), (d["n_i"], ni)):
            t.copy_(v)
        err = err_word()
        torch.cuda.synchronize()
        csa.compress_tree(d["L"], d["ca"], d["x"], d["par"], st.pos, st.front_attn, d["proj_a"], d["rows_a"], d["invf"],
                          comp_i=d["ci"], frontier_i=st.front_index, proj_i=d["proj_i"], rows_i=d["rows_i"], err=err)
        run_commit(cfg, d, leaf, err)
        assert err.item() == 0
        for b in range(0, B, 5):
            at = int(pos0[b]) % cfg.frontier_slots
            assert torch.equal(st.front_attn[b, at], d["proj_a"][b, b % T])
            assert torch.equal(st.front_index[b, at], d["proj_i"][b, b % T])
            assert not (st.front_attn[b, at] == SENTINEL).all()


def test_step_after_commit_in_one_stream():
    """Commit and the next step's calls enqueued without waiting: the step sees the committed state."""
    cfg = FLASH
    trees, pos = [TR.bushy(8), TR.chain(8)], [2047, 3000]
    a, b = _step(cfg, trees, pos, 800), _step(cfg, trees, pos, 800)
    leaf = torch.tensor([7, 5], dtype=torch.int32, device="cuda")
    for d, wait in ((a, False), (b, True)):
        err = err_word()
        for _ in range(4):
            run_step(cfg, d, err)
            if wait:
                torch.cuda.synchronize()
            run_commit(cfg, d, leaf, err)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert err.item() == 0
    for k in ("out", "sel", "rows_a", "kv2"):
        assert torch.equal(a[k], b[k]), k
    assert torch.equal(a["st"].pool, b["st"].pool) and torch.equal(a["st"].window, b["st"].window)
