"""Drawn columns on the GPU, to the rounding of what they are drawn from
(draws_ref.py): rows of many steps, and what is left of a looked-up draft's row."""
import math

import pytest
import torch

import choices_ref as R
import draws_ref as D
import row_wise_softmax_ce_gb300 as ce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def replaced(x, drafts, u, T=1.0):
    """Every row a request of one looked-up draft, refused by its number: the tokens that take its place."""
    pairs = torch.stack([torch.full_like(u, math.nan), u], 1)
    accepted, tokens, logp = ce.verify_drafts(x, drafts.to(DEV), torch.arange(len(u) + 1, device=DEV), pairs.to(DEV),
                                              temperature=T, logp=True)
    assert accepted.tolist() == [0] * len(u)
    return tokens.cpu(), logp.cpu()


# -- a looked-up draft that holds nearly all of its row -----------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [700, 50176, 200001])
@pytest.mark.parametrize("bits", [10, 18, 22, 30, 40, 100])
def test_rest_of_a_looked_up_draft(dtype, vocab, bits):
    """The other columns hold 2^-bits of the row: drawn from as finely as any others."""
    g = gen(vocab + bits)
    n = 24
    x = (0.5 * torch.randn(n, vocab, generator=g)).to(TYPES[dtype])
    x[0] = 0.0  # all the same
    drafts = torch.randint(0, vocab, (n,), generator=g)
    drafts[0], drafts[1] = 0, vocab - 1
    lse = torch.logsumexp(x.double(), 1)
    x[torch.arange(n), drafts] = (lse + bits * math.log(2)).to(x.dtype)
    u = torch.rand(n, generator=g)
    u[2], u[3] = 0.0, 1 - 2.0 ** -24
    tokens, logp = replaced(x.to(DEV), drafts, u)
    for r in range(n):
        d, token = int(drafts[r]), int(tokens[r])
        assert token != d, r
        D.check_own(x[r], 1.0, float(u[r]), token, leave=d, what=(r, bits))
        R.check_logp(x[r], 1.0, token, float(logp[r]), r)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [5, 3001, 60001])
def test_nothing_beside_a_looked_up_draft(dtype, vocab):
    """Others that are masked, by -inf or by the type's lowest value, or weigh less than 2^-126 of the draft: it
    is drawn for itself, as from a row of its own."""
    x = torch.empty(3, vocab, dtype=TYPES[dtype])
    x[0], x[1], x[2] = -math.inf, torch.finfo(x.dtype).min, -100.0
    drafts = torch.tensor([0, vocab - 1, vocab // 2])
    x[torch.arange(3), drafts] = 1.0
    tokens, logp = replaced(x.to(DEV), drafts, torch.tensor([0.0, 0.5, 0.99]))
    assert tokens.tolist() == drafts.tolist()
    assert float(logp.abs().max()) <= 2.0 ** -100
