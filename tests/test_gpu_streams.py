"""stream=: what a call allocates by itself, its workspace and its error word, belongs to the stream that it runs on."""
import numpy as np
import pytest
import torch

import csa_synth

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import deepseek_v4_compressed_csa_gb300 as csa
    from tests import _gpu as G

FLASH = csa_synth.CONFIGS[3].replace(X=512)


def rnd(shape, tag, dtype=torch.bfloat16):
    a = np.random.default_rng([8, tag]).standard_normal(shape, dtype=np.float32)
    return torch.from_numpy(a).to(dtype).cuda()


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def keep_busy():
    """Some milliseconds of work on the current stream."""
    a = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        a = a @ a * 1e-3
    return a


def jobs():
    """name, call(stream), expected error word: calls that report something, their error words their own."""
    cfg, nb = FLASH, 2
    L, invf, z = G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda(), torch.zeros
    comp = G.lib_comp(csa_synth.compressor(cfg, "attn"))
    x, front, pool = rnd((nb, 4, cfg.X), 1), rnd((nb, 8, 2048), 2), rnd((nb, 700, 512), 3)
    q, kv, window, sink = rnd((nb, 64, 512), 4), rnd((nb, 512), 5), rnd((nb, cfg.W, 512), 6), z(64, device="cuda")
    out, far = torch.empty_like(q), torch.full((nb, cfg.topk), 699, dtype=torch.int32, device="cuda")
    p0, p1, n0, n1, k, back, ten, ten2, hw = (i32(*v) for v in ((40, 41), (2000, 2001), (9, 11), (500, 500), (8, 8), (5, 5),
                                                               (10, 10), (10, 10), (40, 40)))
    p2 = hw.clone()
    return [
        ("compress_append", lambda s: csa.compress_append(L, comp, x, p0, front, pool, n0, invf, stream=s), csa.DEV_STATE),
        ("attend_decode", lambda s: csa.attend_decode(L, q, kv, sink, window, pool, n1, far, k, p1, invf, out, stream=s),
         csa.DEV_RANGE),
        ("trim", lambda s: csa.trim(L, back, p2, ten, ten2, hw, stream=s), csa.DEV_ROLLBACK),
    ]


def test_error_words_are_zeroed_on_the_calls_stream():
    """The current stream is busy, the call's is not: its report must not be wiped by a zeroing that comes later."""
    side = torch.cuda.Stream()
    for name, call, want in jobs():
        for stream in (None, side, side):
            torch.cuda.synchronize()
            big = keep_busy() if stream is not None else None
            err = call(stream)
            torch.cuda.synchronize()
            assert err.item() == want, (name, stream)
            del big


def test_workspaces_stay_with_the_calls_stream():
    """The call's stream is busy when it is made, so that its kernels run later: memory that others allocate and write on
    the current stream meanwhile is not its workspace."""
    cfg, nb, cap = FLASH, 4, 9000
    L, invf, side = G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda(), torch.cuda.Stream()
    iq, iw, keys = rnd((nb, 64, 128), 10), rnd((nb, 64), 11), rnd((nb, cap, 128), 12)
    n, pos = i32(8000, 7000, 8999, 3000), i32(32003, 28001, 35999, 12000)
    sel, n_sel = torch.zeros(nb, cfg.topk, dtype=torch.int32, device="cuda"), torch.zeros(nb, dtype=torch.int32, device="cuda")
    size = max(256, csa.workspace_size(L, csa.OP_INDEX_TOPK, nb, 1, cap))
    assert csa.index_topk(L, iq, iw, keys, n, pos, invf, sel, n_sel).item() == 0
    torch.cuda.synchronize()
    want = sel.clone(), n_sel.clone()
    for _ in range(5):
        sel.zero_()
        n_sel.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            keep_busy()
        err = csa.index_topk(L, iq, iw, keys, n, pos, invf, sel, n_sel, stream=side)
        others = [torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
        for _ in range(200):
            for t in others:
                t.fill_(0xFF)
        torch.cuda.synchronize()
        assert err.item() == 0 and torch.equal(sel, want[0]) and torch.equal(n_sel, want[1])


@pytest.mark.parametrize("graphs", [False, True])
def test_tree_steps_on_two_streams_at_once(graphs):
    """Whole tree steps of two batches of different sizes, enqueued (or replayed) on two streams without waiting for one
    another: each gives what it gives alone."""
    from tests import _tree as TR
    from tests import test_gpu_tree as T0
    cfg = FLASH
    shapes = (([TR.bushy(16, s) for s in range(12)], [2100 + 37 * s for s in range(12)]),
              ([TR.bushy(5), TR.chain(8)], [3001, 700]))
    names, T = ("out", "sel", "scores", "rows_a", "rows_i", "proj_a", "q2", "kv2"), [16, 8]
    ds = [T0._step(cfg, trees, pos, 900, seed=1000 + k) for k, (trees, pos) in enumerate(shapes)]
    errs, streams = [T0.err_word() for _ in ds], [torch.cuda.Stream() for _ in ds]
    wss = [dict(c=torch.empty(256, dtype=torch.uint8, device="cuda"),
                a=torch.empty(csa.workspace_size(d["L"], csa.OP_ATTEND_TREE, len(s[1]), t, 900), dtype=torch.uint8,
                              device="cuda")) for d, s, t in zip(ds, shapes, T)]
    want = []
    for d, e, w in zip(ds, errs, wss):
        T0.run_step(cfg, d, e, w)
        torch.cuda.synchronize()
        want.append([d[k].clone() for k in names])
    runs = []
    for d, e, w, s in zip(ds, errs, wss, streams):
        if graphs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                T0.run_step(cfg, d, e, w)
            runs.append(g.replay)
        else:
            runs.append(lambda d=d, e=e, w=w: T0.run_step(cfg, d, e, w))
    for _ in range(10):
        for d in ds:
            for k in names:
                d[k].zero_()
        torch.cuda.synchronize()
        for _ in range(8):
            for r, s in zip(runs, streams):
                with torch.cuda.stream(s):
                    r()
        torch.cuda.synchronize()
        for d, w in zip(ds, want):
            for k, t in zip(names, w):
                assert torch.equal(d[k], t), k
    assert all(e.item() == 0 for e in errs)


def test_streams_by_handle():
    """stream= takes any object that has a handle, a side stream's or the default stream's, with and without buffers of
    the caller's."""
    class Handle:
        def __init__(self, handle):
            self.cuda_stream = handle
    side = torch.cuda.Stream()
    cfg = FLASH
    x, L, invf = rnd((2, 3, 8, 128), 20), G.lib_layer(cfg), csa_synth.inv_freq(cfg).cuda()
    want = csa.norm_rope(L, [x], i32(7, 9), invf)[0]
    pos = i32(7, 9)
    torch.cuda.synchronize()
    for handle in (side.cuda_stream, torch.cuda.default_stream().cuda_stream):
        for name, call, word in jobs():
            torch.cuda.synchronize()
            err = call(Handle(handle))
            torch.cuda.synchronize()
            assert err.item() == word, (name, handle)
        got = csa.norm_rope(L, [x], pos, invf, stream=Handle(handle))
        torch.cuda.synchronize()
        assert torch.equal(got[0], want) and got.err.item() == 0
