"""GPU checks of NaN in keys and queries: it reaches every query head that sees
it and no other row, with a logit cap and without."""
import math

import pytest
import torch

import oracle
from paged_kv_attention_12_gb300 import _build, binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    _build.build()
    binding.lib()


def kv4_case(D, lens, softcap, seed=0):
    """A call over random codes with scales from 0.25 to 4, pages in random order."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    nbs = [-(-n // 16) for n in lens]
    shape = (sum(nbs) + 3, 2, D // 128, 1152)
    k, v = (torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
            for _ in range(2))
    for p in (k, v):
        p[..., 1024:] = p[..., 1024:] % 33 + 0x28
    perm = torch.randperm(shape[0], generator=torch.Generator().manual_seed(seed))
    table = torch.full((len(lens), max(nbs) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(nbs):
        table[b, :n] = perm[at:at + n]
        at += n
    q = torch.randn((len(lens), 8, D), generator=g, device=DEV).to(torch.bfloat16)
    return dict(pool=binding.Kv4Pool(k, v, 0.2, 0.1), table=table.to(DEV), q=q, softcap=softcap,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), most=max(lens))


def kv4_run(c):
    B, hq, D = c["q"].shape
    n = binding.paged_kv4_decode_attn_ws_bytes(B, hq, 2, D, c["most"])
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    out = torch.full_like(c["q"], 7.0)
    binding.paged_kv4_decode_attn_ws(c["q"], out, c["pool"], c["table"], c["lens"], c["most"], ws,
                                     scale=1 / math.sqrt(D), softcap=c["softcap"])
    return out


@pytest.mark.parametrize("softcap", [0.0, 2.0, 50.0])
@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("lens,t", [([90, 70], 53), ([9000, 70], 4805), ([9000, 70], 8999)])
def test_kv4_decode(D, lens, t, softcap):
    """A visible key whose group holds a NaN scale, in whole and cut segments;
    then a query with a NaN element."""
    c = kv4_case(D, lens, softcap)
    clean = kv4_run(c)
    assert torch.isfinite(clean).all()
    unit = c["pool"].k[int(c["table"][0, t // 16]), 1, D // 128 - 1]
    at = oracle.kv4_place(t % 16, 32, False)[2]
    held = int(unit[at])
    unit[at] = 127
    out = kv4_run(c)
    assert torch.isnan(out[0, 4:]).all()
    assert torch.equal(out[0, :4], clean[0, :4]) and torch.equal(out[1], clean[1])
    unit[at] = held
    c["q"][0, 2, D - 3] = NAN
    out = kv4_run(c)
    assert torch.isnan(out[0, 2]).all()
    out[0, 2] = clean[0, 2]
    assert torch.equal(out, clean)
