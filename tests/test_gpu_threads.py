"""Calls from several host threads, each on a stream of its own with buffers of its own: every call succeeds and gives
what it gives alone, whatever the other threads call and whatever the thread did before."""
import dataclasses
import threading

import numpy as np
import pytest
import torch

import csa_synth
from tests import _tree as TR

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import deepseek_v4_compressed_csa_gb300 as csa
    from deepseek_v4_compressed_csa_gb300 import _binding as B
    from tests import _gpu as G

FLASH = csa_synth.CONFIGS[3].replace(X=512)
TINY = csa_synth.CONFIGS[1]
CALLS = 6000


def rnd(cfg, shape, tag, dtype=None):
    a = np.random.default_rng([6, cfg.cid, tag]).standard_normal(shape, dtype=np.float32)
    return torch.from_numpy(a).to(dtype or cfg.storage).cuda()


def z(*shape, dt=torch.bfloat16):
    return torch.zeros(*shape, dtype=dt, device="cuda")


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------ a thread's first call


def fresh_thread_jobs():
    """Every kind of call that describes tensors to the copy engine, its buffers and stream ready: name, call, all
    that it writes."""
    cfg, nb, T, cap, many = FLASH.replace(rollback=4), 2, 4, 600, 40
    L, invf, err, stream = G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda(), i32(0), torch.cuda.Stream()
    fp8 = dataclasses.replace(L, index_fp8=True)
    ca, ci = (G.lib_comp(csa_synth.compressor(cfg, w)) for w in ("attn", "index"))
    ws = {op: z(csa.workspace_size(layer, op, b, t, cap) + 256, dt=torch.uint8) for op, layer, b, t in (
        (csa.OP_COMPRESS, L, nb, T), (csa.OP_COMPRESS_PAIR, L, nb, 1), (csa.OP_INDEX_TOPK, L, nb * T, 1),
        (csa.OP_ATTEND_DECODE, L, nb * T, 1), (csa.OP_ATTEND_PREFILL, L, 1, 40), (csa.OP_ATTEND_TREE, L, many, T),
        (csa.OP_INDEX_SCORES_TREE, fp8, nb, T), (csa.OP_COMPRESS_TREE, L, nb, T))}
    pos, n = i32(2051, 1205), i32(512, 301)
    par = torch.tensor([TR.bushy(T)] * nb, dtype=torch.int32, device="cuda")
    x, iq, iw = rnd(cfg, (nb, T, cfg.X), 40), rnd(cfg, (nb, T, 64, 128), 41), rnd(cfg, (nb, T, 64), 42)
    keys, pool, window = rnd(cfg, (nb, cap, 128), 43), rnd(cfg, (nb, cap, 512), 44), rnd(cfg, (nb, cfg.ring_slots, 512), 45)
    fa, fi = rnd(cfg, (nb, cfg.frontier_slots, 2048), 46), rnd(cfg, (nb, cfg.frontier_slots, 512), 47)
    q, kv, sink = rnd(cfg, (nb, T, 64, 512), 48), rnd(cfg, (nb, T, 512), 49), z(64, dt=torch.float32)
    rows, rows_i, scores = rnd(cfg, (nb, T, 512), 50), rnd(cfg, (nb, T, 128), 51), rnd(cfg, (nb, T, cap + T), 52, torch.float32)
    keys8, rows8 = z(nb, cap, csa.FP8_ROW_BYTES, dt=torch.uint8), z(nb, T, csa.FP8_ROW_BYTES, dt=torch.uint8)
    csa.index_rows_fp8(fp8, keys, keys8)
    csa.index_rows_fp8(fp8, rows_i, rows8)
    iq1, iw1, q1, kv1, x1 = (t[:, :1].contiguous() for t in (iq, iw, q, kv, x))
    iq1, iw1, q1, kv1 = (t[:, 0] for t in (iq1, iw1, q1, kv1))
    chunk = [rnd(cfg, s, 60 + k) for k, s in enumerate(((40, 64, 512), (40, 512), (40, 64, 128), (40, 64)))]
    wide = [t[:1].expand(many, *t.shape[1:]).contiguous() for t in (q, kv, window, pool, rows, scores, par, n, pos)]
    out, out1, outm, outc = z(*q.shape), z(*q1.shape), z(*wide[0].shape), z(*chunk[0].shape)
    sel, n_sel = z(nb, cfg.topk, dt=torch.int32), z(nb, dt=torch.int32)
    proj, prow, iproj, irow = z(nb, T, 2048), z(nb, T, 512), z(nb, T, 512), z(nb, T, 128)
    got, got8 = z(nb, T, cap + T, dt=torch.float32), z(nb, T, cap + T, dt=torch.float32)
    p2, i2, f2, g2, na, ni = z(nb, cap, 512), z(nb, cap, 128), fa.clone(), fi.clone(), n.clone(), n.clone()
    win2, win1, n522 = window.clone(), window[0].clone(), i32(522)  # (the rows after the chunk)
    nq, nkv, leaf, cpos, cn, win3, f3, p3 = z(*q.shape), z(*kv.shape), i32(T - 1, 0), pos.clone(), n.clone(), \
        window.clone(), fa.clone(), pool.clone()
    proj0 = rnd(cfg, (nb, T, 2048), 53)
    ssel, sn_sel, vout, win4 = z(nb, cfg.topk, dt=torch.int32), z(nb, dt=torch.int32), z(*q.shape), window.clone()
    vsel, vn_sel = z(nb, T, cfg.topk, dt=torch.int32), z(nb, T, dt=torch.int32)
    vsel0 = torch.arange(cfg.topk, dtype=torch.int32, device="cuda").expand(nb, T, -1).contiguous()
    vn_sel0 = n[:, None].expand(nb, T).contiguous().clamp(max=256)
    k = dict(err=err, stream=stream)
    return err, [
        ("compress_tree", lambda: csa.compress_tree(
            L, ca, x, par, pos, fa, proj, prow, invf, comp_i=ci, frontier_i=fi, proj_i=iproj, rows_i=irow,
            ws=ws[csa.OP_COMPRESS_TREE], **k), (proj, prow, iproj, irow)),
        ("index_scores_tree", lambda: csa.index_scores_tree(L, iq, iw, keys, rows_i, par, n, pos, got, **k), (got,)),
        ("index_scores_tree, fp8 rows", lambda: csa.index_scores_tree(
            fp8, iq, iw, keys8, rows8, par, n, pos, got8, ws=ws[csa.OP_INDEX_SCORES_TREE], **k), (got8,)),
        ("attend_tree", lambda: csa.attend_tree(
            L, q, kv, sink, window, pool, rows, scores, par, n, pos, invf, out, ws=ws[csa.OP_ATTEND_TREE], **k), (out,)),
        ("attend_tree, many nodes", lambda: csa.attend_tree(
            L, *wide[:2], sink, *wide[2:], invf, outm, ws=ws[csa.OP_ATTEND_TREE], **k), (outm,)),
        ("compress_append", lambda: csa.compress_append(L, ca, x, pos, f2, p2, na, invf, ws=ws[csa.OP_COMPRESS], **k),
         (p2, f2, na)),
        ("compress_append_pair", lambda: csa.compress_append_pair(
            L, ca, ci, x1, pos, f2, p2, na, g2, i2, ni, invf, ws=ws[csa.OP_COMPRESS_PAIR], **k),
         (p2, i2, f2, g2, na, ni)),
        ("index_topk", lambda: csa.index_topk(L, iq1, iw1, keys, n, pos, invf, sel, n_sel, ws=ws[csa.OP_INDEX_TOPK], **k),
         (sel, n_sel)),
        ("attend_decode", lambda: csa.attend_decode(
            L, q1, kv1, sink, win2, pool, n, None, None, pos, invf, out1, ws=ws[csa.OP_ATTEND_DECODE], **k),
         (out1, win2)),
        ("norm_rope", lambda: csa.norm_rope(L, [q, kv], pos, invf, parent=par, outs=[nq, nkv], **k), (nq, nkv)),
        ("commit_tree", lambda: csa.commit_tree(L, par, leaf, cpos, cn, kv, win3, proj0, f3, rows, p3, **k),
         (cpos, cn, win3, f3, p3)),
        ("index_topk_static", lambda: csa.index_topk_static(L, iq1, iw1, keys, n, pos, invf, ssel, sn_sel, **k),
         (ssel, sn_sel)),
        ("index_topk_verify", lambda: csa.index_topk_verify(L, iq, iw, keys, n, pos, invf, vsel, vn_sel,
                                                            ws=ws[csa.OP_INDEX_TOPK], **k), (vsel, vn_sel)),
        ("attend_verify", lambda: csa.attend_verify(L, q, kv, sink, win4, pool, n, vsel0, vn_sel0, pos, invf, vout,
                                                    ws=ws[csa.OP_ATTEND_DECODE], **k), (vout, win4)),
        ("attend_prefill_chunk", lambda: csa.attend_prefill_chunk(
            L, *chunk, sink, 2051, win1, pool[0], keys[0], n522, invf, outc, ws=ws[csa.OP_ATTEND_PREFILL], **k),
         (outc, win1)),
    ]


def test_first_cuda_call_of_a_thread():
    """Each call as the first thing that a host thread does with CUDA: it has no current context before it."""
    err, jobs = fresh_thread_jobs()
    failures = []
    for name, call, written in jobs:
        before = [t.clone() for t in written]
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in written]
        assert not all(torch.equal(w, b) for w, b in zip(want, before)), name
        for t, b in zip(written, before):
            t.copy_(b)
        torch.cuda.synchronize()

        def work(call=call, name=name):
            try:
                call()
            except Exception as e:  # noqa: BLE001 (whatever it is, the test names it)
                failures.append((name, repr(e)))
        thread = threading.Thread(target=work)
        thread.start()
        thread.join()
        torch.cuda.synchronize()
        if not any(f[0] == name for f in failures):
            assert all(torch.equal(t, w) for t, w in zip(written, want)), name
        for t, b in zip(written, before):
            t.copy_(b)
    assert not failures and err.item() == 0, failures


# ------------------------------------------------------------------------------------------------ calls of different sizes


def recorded(call):
    """The library function that `call` uses and the arguments that it hands over, but for the stream (the last one)."""
    got = []

    class Recorder:
        def __getattr__(self, name):
            return lambda *args: got.append((name, args)) or 0
    keep = B.load_library, B._lib
    B.load_library, B._lib = (lambda: Recorder()), Recorder()
    try:
        call()
    finally:
        B.load_library, B._lib = keep
    (name, args), = [g for g in got if g[0] != "csa_workspace_size"]
    return getattr(csa.load_library(), name), args[:-1]


def side_by_side(jobs):
    """jobs: (call, outputs).  Each call by itself, then all of them CALLS times from a thread each, the C calls one
    behind the other (Python lets the other threads run while one is in them)."""
    alone, raw = [], []
    for call, outs in jobs:
        call()
        torch.cuda.synchronize()
        alone.append([o.clone() for o in outs])
        raw.append(recorded(call))
    torch.cuda.synchronize()
    failures, gate = [], threading.Barrier(len(jobs))

    def work(k):
        stream = torch.cuda.Stream()
        f, args = raw[k]
        gate.wait()
        for n in range(CALLS):
            code = f(*args, stream.cuda_stream)
            if code:
                failures.append((k, n, code))
                return
            if n % 100 == 99:
                stream.synchronize()

    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    for (_, outs), want in zip(jobs, alone):
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_compress_tree_of_different_sizes():
    """Token tiles and split counts, and with them the shared memory of the projections, go by the number of nodes."""
    cfg, jobs = FLASH, []
    comp, invf, L = G.lib_comp(csa_synth.compressor(cfg, "attn")), csa_synth.inv_freq(cfg).cuda(), G.lib_layer(cfg)
    for nb, T in ((1, 3), (8, 16), (32, 16)):
        x, frontier = rnd(cfg, (nb, T, cfg.X), 1 + nb), rnd(cfg, (nb, cfg.frontier_slots, 2048), 2 + nb)
        par = torch.tensor([TR.bushy(T, b) for b in range(nb)], dtype=torch.int32, device="cuda")
        pos, err, ws = torch.arange(nb, dtype=torch.int32, device="cuda") * 5, i32(0), z(256, dt=torch.uint8)
        proj, rows = z(nb, T, 2048), z(nb, T, 512)
        jobs.append((lambda a=(L, comp, x, par, pos, frontier, proj, rows, invf), ws=ws, err=err: csa.compress_tree(
            *a, ws=ws, err=err), (proj, rows, err)))
    side_by_side(jobs)


def test_attend_tree_selecting_from_different_capacities():
    """Selections whose keys fill different amounts of shared memory (pools of 17 to 50 thousand rows)."""
    cfg, jobs, T, n = TINY, [], 3, 1000
    L, invf = G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda()
    for cap in (17000, 30000, 50000):
        q, kv, sink = rnd(cfg, (1, T, cfg.H, cfg.D), 10), rnd(cfg, (1, T, cfg.D), 11), rnd(cfg, (cfg.H,), 12)
        window, pool, rows = rnd(cfg, (1, cfg.W, cfg.D), 13), rnd(cfg, (1, cap, cfg.D), 14), rnd(cfg, (1, T, cfg.D), 15)
        out, sel, err = torch.zeros_like(q), z(1, T, cfg.topk, dt=torch.int32), i32(0)
        ws = z(csa.workspace_size(L, csa.OP_ATTEND_TREE, 1, T, cap), dt=torch.uint8)
        a = (L, q, kv, sink, window, pool, rows, rnd(cfg, (1, T, cap + T), 16), i32(*TR.chain(T))[None], i32(n),
             i32(n * cfg.ratio), invf, out)
        jobs.append((lambda a=a, sel=sel, ws=ws, err=err: csa.attend_tree(*a, sel_out=sel, ws=ws, err=err),
                     (out, sel, err)))
    side_by_side(jobs)


def test_index_topk_of_different_capacities():
    cfg, jobs = TINY, []
    L, invf = G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda()
    for cap in (17000, 30000, 50000):
        iq, iw, keys = rnd(cfg, (1, cfg.Hi, cfg.Di), 20), rnd(cfg, (1, cfg.Hi), 21), rnd(cfg, (1, cap, cfg.Di), 22)
        sel, n_sel, err = z(1, cfg.topk, dt=torch.int32), i32(0), i32(0)
        ws = z(csa.workspace_size(L, csa.OP_INDEX_TOPK, 1, 1, cap), dt=torch.uint8)
        a = (L, iq, iw, keys, i32(1000), i32(1000 * cfg.ratio - 1), invf, sel, n_sel)
        jobs.append((lambda a=a, ws=ws, err=err: csa.index_topk(*a, ws=ws, err=err), (sel, n_sel, err)))
    side_by_side(jobs)


@pytest.mark.parametrize("pair", [False, True])
def test_compress_append_of_different_sizes(pair):
    """Three tokens a sequence from position 0: no window completes, so that a call can be made again and again."""
    cfg, jobs = FLASH, []
    comps = [G.lib_comp(csa_synth.compressor(cfg, w)) for w in ("attn", "index")]
    L, invf = G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda()
    for nb, T in ((2, 3), (16, 3), (40, 2)) if pair else ((1, 3), (16, 3), (100, 3)):
        x, pos, err = rnd(cfg, (nb, T, cfg.X), 30 + nb), z(nb, dt=torch.int32), i32(0)
        front = [z(nb, cfg.frontier_slots, 4 * d) for d in (512, 128)]
        pools, n = [z(nb, 8, d) for d in (512, 128)], [z(nb, dt=torch.int32) for _ in range(2)]
        ws = z(csa.workspace_size(L, csa.OP_COMPRESS_PAIR if pair else csa.OP_COMPRESS, nb, T, 8), dt=torch.uint8)

        def call(x=x, pos=pos, err=err, front=front, pools=pools, n=n, ws=ws):
            if pair:
                csa.compress_append_pair(L, *comps, x, pos, front[0], pools[0], n[0], front[1], pools[1], n[1], invf,
                                         ws=ws, err=err)
            else:
                csa.compress_append(L, comps[0], x, pos, front[0], pools[0], n[0], invf, ws=ws, err=err)
        jobs.append((call, (*pools, *front, *n, err)))
    side_by_side(jobs)


def test_attend_decode_of_layers_of_different_widths():
    jobs = []
    for D in (64, 256, 512):
        cfg = TINY.replace(D=D)
        q, kv, sink = rnd(cfg, (2, cfg.H, D), 70), rnd(cfg, (2, D), 71), rnd(cfg, (cfg.H,), 72)
        window, pool, out, err = rnd(cfg, (2, cfg.W, D), 73), rnd(cfg, (2, 40, D), 74), z(2, cfg.H, D, dt=cfg.storage), i32(0)
        L = G.lib_layer(cfg)
        ws = z(csa.workspace_size(L, csa.OP_ATTEND_DECODE, 2, 1, 40), dt=torch.uint8)
        a = (L, q, kv, sink, window, pool, i32(30, 17), None, None, i32(121, 70), csa_synth.inv_freq(cfg).cuda(), out)
        jobs.append((lambda a=a, ws=ws, err=err: csa.attend_decode(*a, ws=ws, err=err), (out, window, err)))
    side_by_side(jobs)
