"""route_rows on row counts to both sides of those that change its kernel, for
every width of a row: a part against the definition in 64 bits, all others bit for
bit as that part, and the choice as a call of a few rows has it, by another kernel.

Many rows take as few lanes as hold a row's columns at up to 32 each: 4 lanes to
128 columns (for at most eight experts a row), 8 to 256, 16 to 512, 32 above. Few
rows take 8 columns a lane."""
import math

import pytest
import torch

import choices_ref as R
import row_wise_softmax_ce_gb300 as ce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
PART = 24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def crossing(E):
    """Rows behind the count from which a lane has up to 32 columns, at any SM count of this card's size."""
    lanes = 8
    while lanes < 32 and 8 * lanes < E:
        lanes *= 2
    return 12 * 32 * torch.cuda.get_device_properties(0).multi_processor_count // lanes + 301


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,k,G,t", [
    (60, 8, 1, 1), (64, 12, 4, 2), (128, 4, 1, 1), (128, 20, 1, 1),      # 4 and 8 lanes
    (160, 6, 8, 3), (256, 9, 8, 4),                                      # 8
    (257, 1, 1, 1), (384, 8, 1, 1), (384, 8, 6, 2), (384, 16, 12, 5),    # 16, groups of whole lanes, and of 2 and 1
    (480, 6, 32, 4), (511, 17, 1, 1), (512, 8, 8, 4), (512, 32, 16, 4),  # groups that are no whole lanes; 17 and more slots
    (513, 9, 1, 1), (1024, 24, 32, 8)])
def test_many_rows(dtype, E, k, G, t):
    rows = crossing(E)
    g = torch.Generator().manual_seed(E + k)
    x = (1.5 * torch.randn(PART, E, generator=g)).to(TYPES[dtype])
    x[torch.rand(PART, E, generator=g) < 0.05] = -math.inf
    x[3] = -math.inf
    x[7, E // 2] = math.nan
    x[8, E - 1] = math.inf
    x[9:14] = x[9:14].float().nan_to_num(neginf=-9.0).round().to(x.dtype)  # ties
    x[14] = torch.finfo(x.dtype).min
    w = torch.ones(PART)
    w[21], w[23] = 0.0, 0.0
    b = 0.2 * torch.randn(E, generator=g)
    at = torch.arange(rows) % PART
    for score, bias, renorm, top, pad in (("sigmoid", b, True, 2, 0), ("softmax", None, False, 2, 0), ("softmax", b, True, 1, 3),
                                          ("sigmoid", None, False, 1, 0)):
        kw = dict(score=score, groups=G, top_groups=t, group_top=top, renormalise=renorm, scale=1.25)
        more = dict(kw, bias=None if bias is None else bias.to(DEV))
        many = torch.zeros(rows, E + pad, dtype=x.dtype, device=DEV)
        many[:, :E] = x.to(DEV)[at.to(DEV)]
        wide = w[at].to(DEV)
        chosen, gates, counts = ce.route_rows(many[:, :E], k, weights=wide, counts=True, **more)
        part = chosen[:PART].cpu()
        R.check_routed(x, k, part, gates[:PART].cpu(), torch.bincount(part[part >= 0], minlength=E), bias=bias, weights=w, **kw)
        on = at.to(DEV)
        assert torch.equal(chosen, chosen[:PART][on])
        assert torch.equal(gates.view(torch.int32), gates[:PART][on].view(torch.int32))
        assert torch.equal(counts, torch.bincount(chosen[chosen >= 0], minlength=E))
        if bias is None or score == "sigmoid":  # a softmax's sum depends on how its row is split
            assert torch.equal(chosen[:PART], ce.route_rows(x.to(DEV), k, weights=w.to(DEV), **more)[0])
