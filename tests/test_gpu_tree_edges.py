"""Trees of drafted tokens on the GPU: errors on every path of the kernels, selections at the borders of the order, sizes
at which one kernel takes over from another, and a committed cache in use afterwards.

Tolerances are those of tests/test_gpu_tree.py (its module docstring)."""
import dataclasses

import numpy as np
import pytest
import torch

import csa_synth
from tests import _tree as TR
from tests._common import f64, oracle_layer

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import deepseek_v4_compressed_csa_gb300 as csa
    from tests import _gpu as G
    from tests import test_gpu_tree as T0

FLASH = csa_synth.CONFIGS[3].replace(X=512)
TINY = csa_synth.CONFIGS[1]
SENTINEL = 7.0


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------ norm_rope's error word


@pytest.mark.parametrize("own", [False, True])
def test_norm_rope_reports_skipped_tokens(own):
    """A negative position and a bad parent: visible in the word that the call returns; the other tokens' rows are those
    of a call without them."""
    cfg = FLASH
    L, invf = G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda()
    x = T0.rnd(cfg, (3, 4, 8, 128), 900)
    good = csa.norm_rope(L, [x], i32(5, 6, 7), invf)
    assert good.err.item() == 0
    err = torch.zeros(1, dtype=torch.int32, device="cuda") if own else None
    out = torch.full_like(x, SENTINEL)
    got = csa.norm_rope(L, [x], i32(5, -1, 7), invf, outs=[out], err=err)
    assert got.err.item() == csa.DEV_STATE and (not own or got.err is err)
    assert (out[1] == SENTINEL).all() and torch.equal(out[::2], good[0][::2])
    par = i32(*[-1, 0, 2, 1] * 3).view(3, 4)  # node 2 is its own parent
    got = csa.norm_rope(L, [x], i32(5, 6, 7), invf, parent=par)
    assert got.err.item() == csa.DEV_STATE
    assert not got[0][:, 2].any() and torch.equal(got[0][:, :2], good[0][:, :2])


# ------------------------------------------------------------------------------------------------ order of calls


@pytest.mark.parametrize("select", [True, False])
def test_tree_calls_right_behind_a_decode_step(select):
    """attend_decode puts its token into the window ring and lets its successor start before it has; attend_tree behind
    it (its own positions in hand, nothing in between) sees that token all the same."""
    cfg = FLASH
    nb, T, cap = 2, 4, 700
    L, invf, sink = G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda(), csa_synth.sinks(cfg).cuda()
    pos, n = i32(2049, 1201), i32(512, 300)
    nxt = pos + 1
    pool, ring = T0.rnd(cfg, (nb, cap, 512), 910), T0.rnd(cfg, (nb, cfg.W, 512), 911)
    q, rows, par = T0.rnd(cfg, (nb, T, 64, 512), 912), T0.rnd(cfg, (nb, T, 512), 913), i32(*[-1, 0, 0, -1] * nb).view(nb, T)
    kv, q1 = T0.rnd(cfg, (nb, T, 512), 914), T0.rnd(cfg, (nb, 64, 512), 915)
    scores = T0.rnd(cfg, (nb, T, cap + T), 916, dtype=torch.float32) if select else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = [torch.empty(csa.workspace_size(L, op, nb, t, cap) + 256, dtype=torch.uint8, device="cuda")
          for op, t in ((csa.OP_ATTEND_DECODE, 1), (csa.OP_ATTEND_TREE, T))]
    outs, before = [], None
    for k in range(30):
        new = T0.rnd(cfg, (nb, 512), 920 + k, scale=8.0)
        for wait in (True, False):
            window, out, out1 = ring.clone(), torch.zeros_like(q), torch.zeros_like(q1)
            torch.cuda.synchronize()
            csa.attend_decode(L, q1, new, sink, window, pool, n, None, None, pos, invf, out1, ws=ws[0], err=err)
            if wait:
                torch.cuda.synchronize()
            csa.attend_tree(L, q, kv, sink, window, pool, rows, scores, par, n, nxt, invf, out, ws=ws[1], err=err)
            torch.cuda.synchronize()
            outs.append(out)
        assert torch.equal(outs[-1], outs[-2]) and err.item() == 0
        assert before is None or not torch.equal(outs[-1], before)
        before = outs[-1]


# ------------------------------------------------------------------------------------------------ selections


SELECTIONS = {
    # columns a node, trees: which kernel selects (few nodes: 256 threads up to 33 KB of keys, then keys in registers, in
    # shared memory, in global memory; more nodes than SMs: 256 threads)
    "small_blocks": (1000, [TR.chain(3)]),
    "registers": (12000, [TR.chain(3)]),
    "registers_64_nodes": (5000, [TR.bushy(64)]),
    "shared": (20000, [TR.chain(3), TR.star(2)]),
    "global": (60000, [TR.chain(3)]),
    "many_nodes": (1100, [TR.chain(64), TR.bushy(64), TR.bushy(64, 1)]),
    "many_nodes_15K": (15000, [TR.chain(64), TR.bushy(64), TR.bushy(25, 1)]),
}


def edge_scores(kind, shape, seed):
    r = np.random.default_rng([13, seed])
    lowest, inf = np.finfo(np.float32).min, np.float32(np.inf)
    s = r.standard_normal(shape, dtype=np.float32)
    if kind == "ties":
        s = r.integers(0, 4, shape).astype(np.float32)
    elif kind == "zeros":  # both zeros: one value
        s = np.where(r.random(shape) < 0.5, np.float32(0.0), np.float32(-0.0))
    elif kind == "minus_inf":  # nearly all of them: the selection has to take some
        s = np.where(r.random(shape) < 0.002, s, -inf)
    elif kind == "lowest":
        s = np.where(r.random(shape) < 0.002, s, np.where(r.random(shape) < 0.3, -inf, lowest))
    elif kind == "plus_inf":
        s = np.where(r.random(shape) < 0.9, inf, s)
    elif kind == "denormals":
        s = (r.integers(-5, 6, shape) * np.float32(1e-45)).astype(np.float32)
    elif kind == "ascending":
        s = np.broadcast_to(np.arange(shape[-1], dtype=np.float32) - 1e4, shape).copy()
    elif kind == "descending":
        s = np.broadcast_to(-np.arange(shape[-1], dtype=np.float32), shape).copy()
    return torch.from_numpy(s.astype(np.float32)).cuda()


@pytest.mark.parametrize("topk", [16, 700])
@pytest.mark.parametrize("where", list(SELECTIONS))
def test_selection_at_the_borders_of_the_order(where, topk):
    """Ties, both zeros, infinities, the lowest float and denormals, with the threshold among them, in every selection
    kernel; what a node does not see is NaN."""
    cap, trees = SELECTIONS[where]
    cfg = TINY.replace(topk=topk)
    nb, T = len(trees), max(len(t) for t in trees)
    pos = [4 * (cap - 20 - 7 * b) + 2 for b in range(nb)]
    p = i32(*pos)
    layer, invf = oracle_layer(cfg), f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    q, kv, sink = T0.rnd(cfg, (nb, T, cfg.H, cfg.D), 940), T0.rnd(cfg, (nb, T, cfg.D), 941), T0.rnd(cfg, (cfg.H,), 942)
    window, pool = T0.rnd(cfg, (nb, cfg.W, cfg.D), 943), T0.rnd(cfg, (1, cap, cfg.D), 944).expand(nb, -1, -1).contiguous()
    rows = T0.rnd(cfg, (nb, T, cfg.D), 945)
    for n, kind in enumerate(("ties", "zeros", "minus_inf", "lowest", "plus_inf", "denormals", "ascending", "descending")):
        scores = edge_scores(kind, (nb, T, cap + T), n)
        for b in range(nb):
            scores[b, :, pos[b] // 4 + T:] = float("nan")
            for i, path in enumerate(TR.paths(TR.padded(trees[b], T))):
                if path is None or (pos[b] + len(path)) % 4:
                    scores[b, :, pos[b] // 4 + i] = float("nan")
        out = torch.full((nb, T, cfg.H, cfg.D), SENTINEL, device="cuda")
        sel = torch.full((nb, T, topk), -9, dtype=torch.int32, device="cuda")
        err = csa.attend_tree(G.lib_layer(cfg), q, kv, sink, window, pool, rows, scores, T0.parents(trees, T), p // 4, p,
                              csa_synth.inv_freq(cfg).cuda(), out, sel_out=sel)
        assert err.item() == 0
        T0.check_tree_outputs(cfg, layer, trees, pos, q, kv, sink, window, pool, rows, scores, out, sel, invf, sampled=2)


# ------------------------------------------------------------------------------------------------ splits of a node's keys


SPLIT_LAYERS = {"topk16": FLASH.replace(cid=71, topk=16), "topk32": FLASH.replace(cid=72, topk=32),
                "topk150": FLASH.replace(cid=73, topk=150), "topk151_w99": FLASH.replace(cid=74, topk=151, W=99),
                "r128": FLASH.replace(cid=75, ratio=128)}
SPLIT_CASES = {
    # one split (window and selection in one tile of 160 rows), its last row used, two splits, no selection
    "one_split": ("topk16", [TR.bushy(9), TR.chain(7), TR.star(3)], [803, 41, 0], True),
    "one_split_full": ("topk32", [TR.bushy(16, s) for s in range(9)], [900 + 61 * s for s in range(9)], True),
    "one_split_short": ("topk32", [TR.bushy(5), [-1]], [70, 2], True),
    "two_splits": ("topk150", [TR.bushy(7), TR.chain(9)], [1201, 603], True),
    "two_splits_odd": ("topk151_w99", [TR.bushy(7), TR.chain(9)], [1201, 80], True),
    "one_split_rows": ("r128", [TR.bushy(7), TR.chain(8)], [900, 127], False),
}


@pytest.mark.parametrize("case", list(SPLIT_CASES))
@pytest.mark.parametrize("loud", [1.0, 24.0])
def test_attend_tree_in_few_splits(case, loud, monkeypatch):
    name, trees, pos, select = SPLIT_CASES[case]
    monkeypatch.setitem(T0.LAYERS, name, SPLIT_LAYERS[name])
    monkeypatch.setitem(T0.AT_CASES, case, (name, trees, pos, "normal" if select else None))
    monkeypatch.setitem(T0.EDGE_LAYERS, name, SPLIT_LAYERS[name])
    monkeypatch.setitem(T0.EDGE_CASES, case, (name, trees, pos, select))
    if loud == 1.0:
        T0.test_attend_tree_against_float64(case)
    T0.test_attend_tree_sinks_and_large_logits(case, loud)


# ------------------------------------------------------------------------------------------------ errors


ERROR_CASES = {
    # layer, nodes a sequence, sequences, first position, selection: the few nodes' kernel with eight, four and one
    # splits, a cluster of CTAs over a long list, a CTA per SM, fp8 index rows
    "few": ("flash", 3, 6, 2500, True),
    "few_4_splits": ("flash", 6, 6, 2500, True),
    "few_rows": ("flash", 3, 6, 9001, False),
    "many": ("flash", 16, 12, 2500, True),
    "many_rows": ("r128", 24, 8, 30000, False),
    "one_split": ("topk16", 4, 6, 900, True),
    "fp8": ("fp8", 7, 6, 2500, True),
}


@pytest.mark.parametrize("case", list(ERROR_CASES))
def test_errors_on_the_tensor_core_paths(case):
    """Sequence 0: parents at or above their node.  1: a node under an unused slot.  2: one row too many.  3: a negative
    position.  4: more rows than the pool has.  The call reports them, leaves those nodes' entries as they were and gives
    every other node what it gives without them."""
    name, T, nb, p0, select = ERROR_CASES[case]
    cfg = {"flash": FLASH, "fp8": FLASH, **SPLIT_LAYERS}[name]
    trees = [TR.bushy(T, s) for s in range(nb)]
    trees[0], trees[1] = TR.chain(T), TR.chain(T)
    pos = [p0 + 37 * b for b in range(nb)]
    cap = max(pos) // cfg.ratio + 20

    def state():
        d = T0._step(cfg, trees, pos, cap, seed=500)
        if name == "fp8":
            d["L"] = dataclasses.replace(d["L"], index_fp8=True)
            keys = torch.zeros(nb, cap, csa.FP8_ROW_BYTES, dtype=torch.uint8, device="cuda")
            csa.index_rows_fp8(d["L"], d["st"].ikeys, keys)
            d["st"].ikeys, d["rows_i"] = keys, torch.zeros(nb, T, csa.FP8_ROW_BYTES, dtype=torch.uint8, device="cuda")
        if not select:
            d.pop("scores", None)
            d.pop("sel", None)
        return d

    def run(d, err):
        if select or not cfg.has_indexer:
            return T0.run_step(cfg, d, err)
        T0.run_step(cfg, dict(d, scores=torch.zeros(nb, T, cap + T, device="cuda"), sel=None), err)
        csa.attend_tree(d["L"], d["q2"], d["kv2"], d["sink"], d["st"].window, d["st"].pool, d["rows_a"], None, d["par"],
                        d["n_a"], d["st"].pos, d["invf"], d["out"], err=err)

    good, bad = state(), state()
    err = T0.err_word()
    names = [k for k in ("q2", "kv2", "proj_a", "rows_a", "proj_i", "rows_i", "scores", "sel", "out") if k in good]
    for d in (good, bad):
        for k in names:
            d[k].fill_(7)
    run(good, err)
    assert err.item() == 0
    dead = torch.zeros(nb, T, dtype=torch.bool, device="cuda")  # by their tree or position: no call touches them
    bad["par"][0, T - 1] = T - 1
    bad["par"][0, 1] = 1000
    dead[0, 1:] = True  # (a chain: everything behind node 1)
    bad["par"][1, 0] = -9
    dead[1] = True
    bad["st"].pos[3] = -5
    dead[3] = True
    bad["n_a"][2] += 1
    bad["n_a"][4] = 1 << 30
    counted = dead.clone()  # and by their row count: the calls that take one
    counted[2] = counted[4] = True
    run(bad, err)
    assert err.item() == csa.DEV_STATE
    for k in names:
        gone = counted if k in ("scores", "sel", "out") else dead
        assert (bad[k][gone] == 7).all(), k
        assert torch.equal(bad[k][~gone], good[k][~gone]), k
    # each call by itself reports what it is given
    for k in range(2 if not cfg.has_indexer else 3):
        e = T0.err_word()
        d = bad
        if k == 0:
            csa.attend_tree(d["L"], d["q2"], d["kv2"], d["sink"], d["st"].window, d["st"].pool, d["rows_a"],
                            d.get("scores"), d["par"], d["n_a"], d["st"].pos, d["invf"], d["out"], err=e)
        elif k == 1:
            csa.compress_tree(d["L"], d["ca"], d["x"], d["par"], d["st"].pos, d["st"].front_attn, d["proj_a"],
                              d["rows_a"], d["invf"], err=e)
        else:
            csa.index_scores_tree(d["L"], d["iq2"], d["iw"], d["st"].ikeys, d["rows_i"], d["par"], d["n_a"], d["st"].pos,
                                  torch.zeros(nb, T, cap + T, device="cuda"), err=e)
        assert e.item() == csa.DEV_STATE, k


# ------------------------------------------------------------------------------------------------ after a commit


AFTER_CASES = {
    "flash": (FLASH, [TR.chain(8), TR.bushy(8)], [2045, 4098]),
    "flash_r128": (FLASH.replace(cid=76, ratio=128), [TR.chain(8), TR.bushy(8)], [1148, 380]),
    "tiny_f32": (TINY, [TR.chain(12), TR.bushy(12)], [61, 130]),
}


@pytest.mark.parametrize("case", list(AFTER_CASES))
def test_a_committed_cache_decodes_on(case):
    """A tree step and its commit, then decoding: projections, selections and outputs against the oracle, which starts
    from the committed cache."""
    from tests.test_gpu_parity import _oracle_decode_check, _seq_projs, _step_rows
    from tests._common import oracle_comp
    cfg, trees, pos = AFTER_CASES[case]
    d, err = T0._step(cfg, trees, pos, max(pos) // cfg.ratio + 40, seed=600), T0.err_word()
    st = d["st"]
    T0.run_step(cfg, d, err)
    T0.run_commit(cfg, d, i32(*[len(t) - 1 for t in trees]), err)
    assert err.item() == 0 and st.pos.tolist() == [p + len(TR.paths(t)[-1]) for p, t in zip(pos, trees)]
    st.n_rows = d["n_a"]
    run = G.Runner(cfg)
    layer, sink, invf = oracle_layer(cfg), f64(csa_synth.sinks(cfg)), f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    comps = [None if c is None else oracle_comp(c) for c in (run.ca_host, run.ci_host)]
    cut = lambda t, b: None if t is None else f64(t[b:b + 1])  # noqa: E731
    # (rows past the committed ones are not zero in this cache and never read)
    state = [dict(pool=cut(st.pool, b), ikeys=cut(st.ikeys, b), window=cut(st.window, b), front_a=cut(st.front_attn, b),
                  front_i=cut(st.front_index, b), n_rows=st.n_rows[b:b + 1].cpu().numpy().astype(np.int64),
                  pos=st.pos[b:b + 1].cpu().numpy().astype(np.int64)) for b in range(2)]
    for k in range(6):
        si = csa_synth.step_inputs(cfg.replace(cid=cfg.cid + 700), k, B=2)
        out, sel, n_sel = run.decode_step(st, si)
        torch.cuda.synchronize()
        assert run.err.item() == 0
        for b in range(2):
            _oracle_decode_check(layer, *comps, state[b], _step_rows(si, b), sink, invf, out[b].cpu(),
                                 None if sel is None else sel[b].cpu().numpy(),
                                 None if n_sel is None else int(n_sel[b]), f"step {k} seq {b}", _seq_projs(run, b))


@pytest.mark.parametrize("case", list(AFTER_CASES))
def test_trim_behind_a_commit_is_a_shorter_commit(case):
    """An accepted path rewound by csa_trim against the commit of its first nodes alone: the same state, and the same bits
    in every decode step after it."""
    cfg, trees, pos = AFTER_CASES[case]
    cfg = cfg.replace(cid=cfg.cid + 20, rollback=16)
    cap = max(pos) // cfg.ratio + 40
    a, b = (T0._step(cfg, trees, pos, cap, seed=700) for _ in range(2))
    paths = [TR.paths(t)[-1] for t in trees]
    back = [len(paths[0]) - 1, len(paths[1]) - 2]
    err = T0.err_word()
    for d in (a, b):
        T0.run_step(cfg, d, err)
    hw = a["st"].pos.clone()
    T0.run_commit(cfg, a, i32(*[p[-1] for p in paths]), err)
    T0.run_commit(cfg, b, i32(*[p[-1 - n] for p, n in zip(paths, back)]), err)
    csa.trim(a["L"], i32(*back), a["st"].pos, a["n_a"], a["n_i"] if cfg.has_indexer else None, hw, err=err)
    assert err.item() == 0
    assert torch.equal(a["st"].pos, b["st"].pos) and torch.equal(a["n_a"], b["n_a"])
    runs = [G.Runner(cfg) for _ in range(2)]
    for d in (a, b):
        d["st"].n_rows = d["n_a"]
    for k in range(10):
        si = csa_synth.step_inputs(cfg.replace(cid=cfg.cid + 700), k, B=2)
        got = [r.decode_step(d["st"], si) for r, d in zip(runs, (a, b))]
        for x, y in zip(*got):
            assert x is None or torch.equal(x, y), k
    assert all(r.err.item() == 0 for r in runs) and torch.equal(a["n_a"], b["n_a"])
    for s in range(2):
        n = int(a["n_a"][s])
        assert torch.equal(a["st"].pool[s, :n], b["st"].pool[s, :n])
    # beyond the margin: refused, nothing changed
    keep, refused = a["st"].pos.clone(), T0.err_word()
    csa.trim(a["L"], i32(17, 17), a["st"].pos, a["n_a"], a["n_a"].clone() if cfg.has_indexer else None, hw, err=refused)
    assert refused.item() == csa.DEV_ROLLBACK and torch.equal(a["st"].pos, keep)


# ------------------------------------------------------------------------------------------------ positions


@pytest.mark.parametrize("name", ["flash", "tiny_f32"])
def test_positions_near_the_end_of_32_bits(name):
    """A sequence whose nodes' positions would not fit (its row count agrees with it): reported and left alone by every
    call; the sequence next to it is served."""
    cfg = {"flash": FLASH, "tiny_f32": TINY}[name]
    trees, pos = [TR.chain(8), TR.bushy(8)], [2045, 1203]
    good, bad = (T0._step(cfg, trees, pos, 600, seed=800) for _ in range(2))
    names = ["q2", "kv2", "proj_a", "rows_a", "proj_i", "rows_i", "scores", "sel", "out"]
    for d in (good, bad):
        for k in names:
            d[k].fill_(7)
    end = 2 ** 31 - 3
    bad["st"].pos[1], bad["n_a"][1], bad["n_i"][1] = end, end // cfg.ratio, end // cfg.ratio
    errs = [T0.err_word() for _ in range(2)]
    for d, e in zip((good, bad), errs):
        T0.run_step(cfg, d, e)
    assert errs[0].item() == 0 and errs[1].item() == csa.DEV_STATE
    last = [i for i, p in enumerate(TR.paths(trees[1])) if end + len(p) - 1 > 2 ** 31 - 1]
    assert last
    for k in names:
        assert torch.equal(bad[k][0], good[k][0]), k
        gone = bad[k][1][last] if k in ("q2", "kv2") else bad[k][1]  # (norm_rope goes by the token)
        assert (gone == 7).all(), k
    st = bad["st"]
    keep = [t[1].clone() for t in (st.window, st.pool, st.ikeys, st.front_attn, st.front_index)]
    e = T0.err_word()
    T0.run_commit(cfg, bad, i32(7, 7), e)
    assert e.item() == csa.DEV_STATE and st.pos.tolist() == [2053, end]
    assert bad["n_a"].tolist() == [2053 // cfg.ratio, end // cfg.ratio]
    for a, b in zip(keep, (st.window, st.pool, st.ikeys, st.front_attn, st.front_index)):
        assert torch.equal(a, b[1])
    # a chunk without a tree: the tokens that fit are served
    x = T0.rnd(cfg, (1, 6, cfg.H, cfg.D), 990)
    got = csa.norm_rope(G.lib_layer(cfg), [x], i32(end), csa_synth.inv_freq(cfg).cuda(), outs=[torch.full_like(x, 7)])
    assert got.err.item() == csa.DEV_STATE and (got[0][0, 3:] == 7).all() and not (got[0][0, :3] == 7).all()


# ------------------------------------------------------------------------------------------------ the largest batches


@pytest.mark.parametrize("nb, T", [(65535, 1), (4096, 64)])
def test_largest_batches(nb, T):
    """As many sequences, and as many nodes, as the calls take: sequences from all over the batch against the same ones
    by themselves (the attention in float64: few and many nodes run different kernels)."""
    cfg = FLASH.replace(X=64)
    cap, ratio = 6, 4
    g = torch.Generator(device="cuda").manual_seed(17)
    n = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    one = TR.bushy(T)
    pos = torch.arange(nb, dtype=torch.int32, device="cuda") % (4 * cap - 3 if T == 1 else 3)
    par = torch.tensor(one, dtype=torch.int32, device="cuda").expand(nb, T).contiguous()
    L, invf, sink = G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda(), csa_synth.sinks(cfg).cuda()
    ca, ci = (G.lib_comp(csa_synth.compressor(cfg, w)) for w in ("attn", "index"))
    pick = [0, 1, nb // 2, nb - 2, nb - 1]

    def step(d, pos, par, err):
        b = par.shape[0]
        z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        o = dict(proj_a=z(b, T, 2048), rows_a=z(b, T, 512), proj_i=z(b, T, 512), rows_i=z(b, T, 128),
                 scores=z(b, T, cap + T, dt=torch.float32), out=torch.full((b, T, 64, 512), SENTINEL,
                                                                           dtype=torch.bfloat16, device="cuda"))
        o["q"], o["kv"], o["iq"] = csa.norm_rope(L, [d["q"], d["kv"], d["iq"]], pos, invf, parent=par, err=err)
        csa.compress_tree(L, ca, d["x"], par, pos, d["fa"], o["proj_a"], o["rows_a"], invf, comp_i=ci, frontier_i=d["fi"],
                          proj_i=o["proj_i"], rows_i=o["rows_i"], err=err)
        csa.index_scores_tree(L, o["iq"], d["iw"], d["keys"], o["rows_i"], par, pos // ratio, pos, o["scores"], err=err)
        csa.attend_tree(L, o["q"], o["kv"], sink, d["window"], d["pool"], o["rows_a"], o["scores"], par, pos // ratio,
                        pos, invf, o["out"], err=err)
        return o

    d = dict(q=n(nb, T, 64, 512), kv=n(nb, T, 512), iq=n(nb, T, 64, 128), iw=n(nb, T, 64), x=n(nb, T, 64),
             fa=n(nb, 8, 2048), fi=n(nb, 8, 512), keys=n(nb, cap, 128), pool=n(nb, cap, 512), window=n(nb, cfg.W, 512))
    err = T0.err_word()
    big = step(d, pos, par, err)
    small = step({k: v[pick].contiguous() for k, v in d.items()}, pos[pick].contiguous(), par[pick].contiguous(), err)
    assert err.item() == 0
    for k in ("q", "kv", "iq"):
        assert torch.equal(big[k][pick], small[k]), k
    layer, f = oracle_layer(cfg), f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    for k in ("proj_a", "proj_i"):  # fp32 sums of 64 products in another order: the neighbouring value at most
        a, b = f64(big[k][pick]), f64(small[k])
        assert (np.abs(a - b) <= G.ulp(np.abs(b), "bf16") + 2.0 ** -12 * np.abs(b).max()).all(), k
    at = [int(p) for p in pos[pick]]
    for j, b in enumerate(pick):
        for i, path in enumerate(TR.paths(one)):
            ref, bound = TR.scores_row(layer, big["iq"][b, i], d["iw"][b, i], d["keys"][b], big["rows_i"][b], path, at[j])
            got = f64(big["scores"][b, i, :at[j] // ratio + T])
            assert np.array_equal(np.isfinite(got), np.isfinite(ref))
            fin = np.isfinite(ref)
            assert (np.abs(got[fin] - ref[fin]) <= 2 * (128 + 64 + 8) * 2.0 ** -24 * bound[fin]).all()
    T0.check_tree_outputs(cfg, layer, [one] * len(pick), at, big["q"][pick], big["kv"][pick], f64(sink),
                          d["window"][pick], d["pool"][pick], big["rows_a"][pick], big["scores"][pick],
                          big["out"][pick], None, f)
    st = {k: d[k].clone() for k in ("window", "pool", "keys", "fa", "fi")}
    p2, na, ni = pos.clone(), pos // ratio, pos // ratio
    leaf = torch.full((nb,), T - 1, dtype=torch.int32, device="cuda")
    csa.commit_tree(L, par, leaf, p2, na, big["kv"], st["window"], big["proj_a"], st["fa"], big["rows_a"], st["pool"],
                    n_rows_i=ni, proj_i=big["proj_i"], frontier_i=st["fi"], rows_i=big["rows_i"], pool_i=st["keys"],
                    err=err)
    path = TR.paths(one)[-1]
    assert err.item() == 0 and torch.equal(p2, pos + len(path)) and torch.equal(na, p2 // ratio)
    for b, p in zip(pick, at):
        for k, node in enumerate(path):
            assert torch.equal(st["window"][b, (p + k) % cfg.W], big["kv"][b, node])
            if k >= len(path) - 8:
                assert torch.equal(st["fa"][b, (p + k) % 8], big["proj_a"][b, node])
            if (p + k + 1) % ratio == 0:
                assert torch.equal(st["pool"][b, (p + k + 1) // ratio - 1], big["rows_a"][b, node])


# ------------------------------------------------------------------------------------------------ other layers


MIXED = T0.ODD.replace(cid=80, D=64) if torch.cuda.is_available() else None  # one pool on the tensor cores, one not
MORE_LAYERS = {} if MIXED is None else {
    "attn_on_tc": MIXED,
    "index_on_tc": T0.ODD.replace(cid=81, Di=64),
    "flash_rollback": FLASH.replace(cid=82, rollback=37),
    "flash_r128_rollback": FLASH.replace(cid=83, ratio=128, rollback=5),
    "tiny_r1": TINY.replace(cid=84, ratio=1),
    "tiny_r3": TINY.replace(cid=85, ratio=3),
    "tiny_rollback": TINY.replace(cid=86, rollback=9),
    "flash_w1": FLASH.replace(cid=87, W=1, topk=64),
    "tiny_w1": TINY.replace(cid=88, W=1),
    "one_head": T0.ODD.replace(cid=89, H=1, Hi=1, D=24, R=8, Di=8),
    "wide_rows": TINY.replace(cid=90, D=1024, H=2),
}


@pytest.mark.parametrize("name", ["attn_on_tc", "index_on_tc", "flash_rollback", "flash_r128_rollback", "tiny_r1",
                                  "tiny_r3", "tiny_rollback", "one_head", "wide_rows"])
def test_compress_tree_of_other_layers(name, monkeypatch):
    """Pools that are projected on different units, rings with a rollback margin, ratios down to 1."""
    monkeypatch.setitem(T0.LAYERS, name, MORE_LAYERS[name])
    for k, (trees, pos) in enumerate((([TR.chain(20), TR.bushy(17)], [61, 0]), ([TR.bushy(64)], [259]),
                                      ([[-1], [-1], [-1]], [3, 127, 4]))):
        case = f"{name}_{k}"
        monkeypatch.setitem(T0.CT_CASES, case, (name, trees, pos))
        T0.test_compress_tree_against_paths(case)


@pytest.mark.parametrize("name", ["flash_w1", "tiny_w1", "one_head", "wide_rows", "tiny_r1", "tiny_r3", "flash_rollback"])
def test_attend_tree_of_other_layers(name, monkeypatch):
    """Windows of one token, one head, the widest rows, ratios down to 1."""
    cfg = MORE_LAYERS[name]
    monkeypatch.setitem(T0.LAYERS, name, cfg)
    monkeypatch.setitem(T0.EDGE_LAYERS, name, cfg)
    select = cfg.has_indexer
    for k, (trees, pos) in enumerate((([TR.chain(9), TR.bushy(7)], [400, 0]), ([TR.bushy(16, s) for s in range(11)],
                                                                               [300 + 7 * s for s in range(11)]))):
        case = f"{name}_{k}"
        monkeypatch.setitem(T0.EDGE_CASES, case, (name, trees, pos, select))
        if cfg.H >= 4:  # (that test gives every fourth head its sink)
            T0.test_attend_tree_sinks_and_large_logits(case, 1.0)
        if cfg.rollback == 0:
            monkeypatch.setitem(T0.AT_CASES, case, (name, trees, pos, "ties" if select else None))
            T0.test_attend_tree_against_float64(case)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [8, 24, 64])
def test_norm_rope_of_every_width(dtype, R):
    """Rows of every width from the rotated dims to 1024 values, odd head counts, strided and dense."""
    cfg = TINY.replace(cid=91, dtype=dtype, D=64, Di=64, R=R)
    f = f64(csa_synth.inv_freq(cfg)).astype(np.float32)
    L, invf, pos = G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda(), i32(777, 0)
    widths = sorted(set(range(R, 1025, 8)))
    for k in range(0, len(widths), 4):
        xs, ws, ref = [], [], []
        for j, dim in enumerate(widths[k:k + 4]):
            heads = (1, 3, 33, 2)[(k + j) % 4]
            wide = T0.rnd(cfg, (2, 3, heads * dim + 8 * (j % 2)), 1000 + dim, scale=2.0)
            xs.append(wide[..., :heads * dim].unflatten(-1, (heads, dim)))
            ws.append(T0.rnd(cfg, (dim,), 2000 + dim, dtype=torch.float32) if j != 1 else None)
        got = csa.norm_rope(L, xs, pos, invf, weights=ws)
        assert got.err.item() == 0
        for x, w, o in zip(xs, ws, got):
            for b in range(2):
                for i in range(3):
                    want = TR.norm_rope(x[b, i], w, True, cfg.rms_eps, int(pos[b]) + i, f)
                    pair = np.repeat(np.hypot(want[..., ::2], want[..., 1::2]), 2, axis=-1)
                    tol = 2.0 ** -18 * pair
                    assert (np.abs(f64(o[b, i]) - want) <= T0.half_step(np.abs(want) + tol, dtype) + tol).all(), x.shape
