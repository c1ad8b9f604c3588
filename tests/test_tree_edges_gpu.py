"""GPU checks of the draft-tree calls at the edges of what they take."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_12_gb300 import _build, binding
from tests.test_tree_gpu import check, f64, i32, i64, make, run, workspace

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    binding.lib()


@pytest.mark.parametrize("lens,hkv", [([600] * 8, 2), ([3000, 2500, 4000], 2), ([500] * 100, 1)])
def test_first_loads_out_of_cold_memory(lens, hkv):
    """D = 256: V's first loads come behind K's first tile, whatever the caches hold.
    Pairs of CTAs, cut segments and whole ones; no wait runs out."""
    c = make(lens, [9] * len(lens), D=256, hq=4 * hkv, hkv=hkv, seed=len(lens))
    want = run(c)
    check(c, want)
    args = (c["k"], c["v"], i32(c["table"]), i32(c["first"]), i64(c["masks"]), i32(c["lens"]))
    out, ws, err = torch.full_like(want, 7.0), workspace(c), i32([0])
    cold = torch.zeros(1 << 28, dtype=torch.uint8, device=DEV)      # past the L2
    for i in range(50):
        if i % 2:
            cold.fill_(i)
        binding.paged_tree_attn_ws(c["q"], out, *args, c["most"], max(lens), ws, scale=c["scale"],
                                   err=err)
        if i % 2:
            assert torch.equal(out, want)
    torch.cuda.synchronize()
    assert err.item() == 0 and torch.equal(out, want)


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("window", [62, 63, 64, 65])
def test_windows_as_long_as_the_widest_mask(D, window):
    """Masks that are no tree: a row of all 64 bits is 64 deeper than one of none, and a
    window of 64 hides that key from it."""
    rng = np.random.default_rng(5)
    ns = [20, 64, 9]
    masks = [int(x) for x in rng.integers(0, 1 << 63, sum(ns))] + [1] * 3
    masks[30], masks[31], masks[40] = 0, (1 << 64) - 1, 1 << 63
    c = make([100, 64, 400], ns, D=D, masks=masks, window=window, seed=window)
    assert (oracle.tree_visible(masks[20:84], 64, window)[11, 10]) == (window > 64)
    check(c, run(c))
