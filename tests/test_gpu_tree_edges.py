"""Trees of drafted tokens on the GPU: errors on every path of the kernels, selections at the borders of the order, sizes
at which one kernel takes over from another, and a committed cache in use afterwards.

Tolerances are those of tests/test_gpu_tree.py (its module docstring)."""
import dataclasses

import numpy as np
import pytest
import torch

import csa_synth
from oracle import csa_oracle as O
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
