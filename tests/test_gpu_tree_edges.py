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
