"""GPU checks of the logit cap of the bf16 entry points."""
import pytest
import torch

import oracle
from paged_kv_attention_12_gb300 import _build, binding, workload
from tests.parity import assert_close, to_f64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    binding.lib()


def batch(D, L, n, softcap, **kw):
    return workload.make_batch(seq_lens=L, q_lens=n, num_q_heads=8, num_kv_heads=2, head_dim=D,
                               num_blocks=sum(-(-x // 16) for x in L) + 8, device=DEV, poison=True,
                               cfg_id=43, softcap=softcap, **kw)


def check(b):
    ref, _ = oracle.run_batch(workload.to_numpy_f64(b))
    out = torch.full_like(b.q, float("nan"))
    got = {"prefill": binding.run_batch(b, out).clone(), "mixed": binding.MixedBatch(b).run()}
    if max(b.q_lens_host) == 1:
        binding.paged_decode_attn(b.q, out, b.k_pool, b.v_pool, b.block_tables, b.seq_lens,
                                  b.max_seq_len, scale=b.scale, softcap=b.softcap)
        got.update({"decode": out, "split-K": binding.DecodeSplitK(b).run(),
                    "fused": binding.DecodeFused(b).run()})
    for name, x in got.items():
        assert_close(to_f64(x), ref, name)


SHAPES = [([300, 200, 33], [130, 200, 1]), ([900, 40, 1], [1, 1, 1])]


@pytest.mark.parametrize("softcap", [2.0, 8.0, 50.0])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("L,n", SHAPES)
def test_negative_scale(D, L, n, softcap):
    """Logits on both sides of the cap's bend, of either sign of the scale."""
    check(batch(D, L, n, softcap, scale=-0.25))


@pytest.mark.parametrize("softcap", [1e-40, 1e-12, 1e-3, 1.5e38, 3.4e38])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("L,n", SHAPES)
def test_ends_of_the_range(D, L, n, softcap):
    """A cap near 0 makes every key alike, one near the largest float none
    different, and queries of zeros average their values under both."""
    b = batch(D, L, n, softcap, seed=1)
    b.q[:max(1, n[0] // 2)] = 0.0
    check(b)


@pytest.mark.parametrize("softcap", [64.5, 300.0, 1e4, 1e6, 1e9, 1e20])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("L,n", SHAPES)
def test_caps_far_above_the_logits(D, L, n, softcap):
    check(batch(D, L, n, softcap, seed=2))
