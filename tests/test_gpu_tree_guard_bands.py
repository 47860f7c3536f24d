"""Guard bands (tests/test_gpu_guard_bands.py) around every buffer of the tree calls: whole steps and their commits, on
sizes that reach each of their kernels, with unused slots and reported errors among them."""
import dataclasses

import pytest
import torch

import csa_synth
from tests import _tree as TR

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import deepseek_v4_compressed_csa_gb300 as csa
    from tests import test_gpu_tree as T0
    from tests.test_gpu_guard_bands import Guards

FLASH = csa_synth.CONFIGS[3].replace(X=512)
TINY = csa_synth.CONFIGS[1]
ODD = TINY.replace(cid=61, dtype="bf16", H=5, D=72, R=24, W=9, Hi=3, Di=40, topk=7, X=64)
CASES = {
    # layer, trees, positions, rows behind the last one that a path completes
    "few": (FLASH, [TR.bushy(5), TR.chain(3)], [2045, 130], 0),
    "one_node": (FLASH, [[-1]], [7], 0),
    "many": (FLASH, [TR.bushy(16, s) for s in range(11)], [2045 + 37 * s for s in range(11)], 0),
    "t64": (FLASH, [TR.bushy(64), TR.chain(61)], [2500, 0], 0),
    "registers": (FLASH, [TR.bushy(20), TR.chain(25)], [17001, 900], 5),
    "shared": (FLASH, [TR.bushy(3)], [70001], 3),
    "global": (FLASH, [TR.bushy(3)], [210001], 3),
    "one_split": (FLASH.replace(cid=95, topk=16), [TR.bushy(7), TR.chain(5)], [803, 41], 0),
    "rollback": (FLASH.replace(cid=96, rollback=13), [TR.bushy(9), TR.chain(12)], [2045, 12], 0),
    "r128": (FLASH.replace(cid=97, ratio=128), [TR.bushy(9), TR.chain(40)], [3000, 120], 0),
    "r128_long": (FLASH.replace(cid=97, ratio=128), [TR.bushy(3), TR.chain(4)], [300001, 99], 0),
    "r128_many": (FLASH.replace(cid=97, ratio=128), [TR.bushy(16, s) for s in range(11)], [127 + 5000 * s for s in range(11)], 0),
    "fp8": (FLASH, [TR.bushy(13), TR.chain(9)], [4001, 515], 0),
    "tiny_f32": (TINY, [TR.bushy(9), TR.chain(12)], [61, 0], 0),
    "odd_bf16": (ODD, [TR.binary(12), [-1]], [61, 2], 0),
}


@pytest.mark.parametrize("case", list(CASES))
@pytest.mark.parametrize("errors", [False, True])
def test_guard_bands_of_tree_steps(case, errors):
    cfg, trees, pos, extra = CASES[case]
    nb, T = len(trees), max(len(t) for t in trees)
    cap = max((p + len(path)) // cfg.ratio for p, t in zip(pos, trees) for path in TR.paths(t)) + extra
    gd = Guards()
    d = T0._step(cfg, trees, pos, cap, seed=1100)
    st = d["st"]
    if case == "fp8":
        d["L"] = dataclasses.replace(d["L"], index_fp8=True)
        keys = torch.zeros(nb, cap, csa.FP8_ROW_BYTES, dtype=torch.uint8, device="cuda")
        csa.index_rows_fp8(d["L"], st.ikeys, keys)
        st.ikeys, d["rows_i"] = keys, torch.zeros(nb, T, csa.FP8_ROW_BYTES, dtype=torch.uint8, device="cuda")
    for k in [k for k, v in d.items() if isinstance(v, torch.Tensor)]:
        d[k] = gd.wrap(k, d[k])
    for k in ("pool", "ikeys", "window", "front_attn", "front_index", "pos"):
        if getattr(st, k) is not None:
            setattr(st, k, gd.wrap(k, getattr(st, k)))
    for k in ("ca", "ci"):
        if k in d:
            c = d[k]
            d[k] = dataclasses.replace(c, **{f: gd.wrap(k + f, getattr(c, f)) for f in ("wkv", "wgate", "ape", "norm_w")})
    err = gd.empty("err", (1,), torch.int32)
    L = d["L"]
    ws = {"c": gd.ws("ws_c", csa.workspace_size(L, csa.OP_COMPRESS_TREE, nb, T, cap)),
          "a": gd.ws("ws_a", csa.workspace_size(L, csa.OP_ATTEND_TREE, nb, T, cap))}
    leaf = gd.wrap("leaf", torch.tensor([len(t) - 1 for t in trees], dtype=torch.int32))
    if errors:
        d["par"][0, T - 1] = T + 1000
        if nb > 1:
            d["n_a"][1] = 1 << 30
            leaf[1] = 1 << 20
        if nb > 2:
            st.pos[2] = -(1 << 31)
            st.pos[3] = 2 ** 31 - 1
    T0.run_step(cfg, d, err, ws)
    if cfg.has_indexer and case != "fp8":  # every row wanted too
        csa.attend_tree(L, d["q2"], d["kv2"], d["sink"], st.window, st.pool, d["rows_a"], None, d["par"], d["n_a"], st.pos,
                        d["invf"], d["out"], ws=ws["a"], err=err)
    torch.cuda.synchronize()
    assert err.item() == (csa.DEV_STATE if errors else 0)
    gd.check()
    T0.run_commit(cfg, d, leaf, err)
    torch.cuda.synchronize()
    assert err.item() == (csa.DEV_STATE if errors else 0)
    gd.check()
    finite = [d["out"], d["q2"], d["kv2"], d["proj_a"], d["rows_a"], st.pool, st.window, st.front_attn]
    if cfg.has_indexer:
        assert not torch.isnan(d["scores"]).any()
        finite += [d["proj_i"], st.front_index] + ([] if case == "fp8" else [d["rows_i"], st.ikeys])
    for t in finite:
        assert torch.isfinite(t.float()).all()
