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


# -- rows of many steps ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,T", [(40, 20011, 1.0), (300, 30011, 0.8), (12, 200001, 1.0), (2, 1 << 22, 1.3)])
def test_places(dtype, rows, vocab, T):
    """Nearly equal columns: a place a few columns wide. Short rows of few steps by a CTA, the others by k_sample."""
    g = gen(vocab)
    stride, lead = vocab + rows % 3, rows % 5
    buf = torch.zeros(lead + rows * stride, dtype=TYPES[dtype])
    x = buf[lead:].view(rows, stride)[:, :vocab]
    x.copy_(0.5 * torch.randn(rows, vocab, generator=g))
    u = torch.rand(rows, generator=g)
    wide = buf.to(DEV)[lead:].view(rows, stride)[:, :vocab]
    tokens, logp = [t.cpu() for t in ce.sample_rows(wide, u.to(DEV), temperature=T, logp=True)]
    for r in range(rows):
        D.check_own(x[r], T, float(u[r]), int(tokens[r]), what=r)
        R.check_logp(x[r], T, int(tokens[r]), float(logp[r]), r)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(12, 50257), (6, 200001), (2, 1 << 22)])
def test_rest_places(dtype, rows, vocab):
    """What draft rows leave, at other phases than the target's."""
    g = gen(vocab + 1)
    x = torch.randn(rows, vocab, generator=g)
    y = (x + 0.7 * torch.randn(rows, vocab, generator=g)).to(TYPES[dtype])
    x = x.to(TYPES[dtype])
    drafts = y.float().argmax(1)
    u = torch.rand(rows, generator=g)
    pairs = torch.stack([torch.full_like(u, math.nan), u], 1).to(DEV)
    ends = torch.arange(rows + 1, device=DEV)
    wide = torch.zeros(rows, vocab + 3, dtype=TYPES[dtype], device=DEV)
    wide[:, :vocab] = y.to(DEV)
    accepted, tokens, logp = ce.verify_drafts(x.to(DEV), drafts.to(DEV), ends, pairs, draft_logits=wide, vocab=vocab, logp=True)
    assert accepted.tolist() == [0] * rows
    for r in range(rows):
        assert D.check_rest(x[r], y[r], 1.0, float(u[r]), int(tokens[r]), r) is not None
        R.check_logp(x[r], 1.0, int(tokens[r]), float(logp[r]), r)


def heavy_columns(vocab, n, g):
    """Columns at both ends of the row, of steps of 1024 and 2048 columns, of warps, lanes and vectors."""
    at = {0, 1, 7, 8, 31, 255, 256, 1023, 1024, 2047, 2048, 32 * 2048 - 1, 32 * 2048, vocab - 2049, vocab - 9, vocab - 1}
    at |= {8 * 32 * 1024 + 5, 9 * 1024 * 17 + 1023, vocab // 2, vocab // 3 | 1, vocab - 1024 * 3}
    at = {a for a in at if 0 <= a < vocab}
    while len(at) < n:
        at.add(int(torch.randint(0, vocab, (1,), generator=g)))
    return torch.tensor(sorted(at))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [50257, 200001, 1 << 24])
def test_heavy_columns(dtype, vocab):
    """Columns that hold all but a thousandth: a number in the middle of one's share draws that one and no other,
    from a row, beside a looked-up draft and from what a draft row leaves. 2^24 columns: 17 steps and more a lane."""
    g = gen(vocab)
    heavy = heavy_columns(vocab, 40, g)
    base = (0.5 * torch.randn(vocab, generator=g)).to(TYPES[dtype])
    row = base.clone()
    row[heavy] = 20.0
    p = torch.softmax(row.double(), 0)
    assert float(p[heavy].sum()) > 0.999
    n = 8

    def middles(w):
        upto = w.cumsum(0)
        return ((upto[heavy] - 0.5 * w[heavy]) / upto[-1]).float()

    x = row.to(DEV).expand(n, vocab).contiguous()
    ends, none = torch.arange(n + 1, device=DEV), torch.full((n,), math.nan)

    def emitted(drafts, u, draft_logits=None):
        pairs = torch.stack([none, u], 1).to(DEV)
        return ce.verify_drafts(x, torch.full((n,), drafts, device=DEV), ends, pairs, draft_logits=draft_logits)[1]
    for part, u in zip(heavy.split(n), middles(p).split(n)):
        assert ce.sample_rows(x, u.to(DEV)).tolist() == part.tolist()
        assert emitted(-1, u).tolist() == part.tolist()
    # one heavy column is the looked-up draft, or all that the draft row has
    for d in (int(heavy[0]), int(heavy[len(heavy) // 2]), int(heavy[-1])):
        beside = p.clone()
        beside[d] = 0.0
        draft = base.clone()
        draft[d] = 40.0
        left = (p - torch.softmax(draft.double(), 0)).clamp(min=0)
        rows = draft.to(DEV).expand(n, vocab).contiguous()
        for part, u, v in zip(heavy.split(n), middles(beside).split(n), middles(left).split(n)):
            on = part != d
            assert emitted(d, u).cpu()[on].tolist() == part[on].tolist()
            assert emitted(d, v, rows).cpu()[on].tolist() == part[on].tolist()


@pytest.mark.parametrize("rows,vocab,dtype", [(4096, 5004, "f32"), (4096, 6016, "bf16"), (300, 20000, "bf16"), (150, 8192, "f32")])
def test_whole_distribution_of_many_steps(rows, vocab, dtype):
    """Evenly spaced numbers draw each column within one of its share of them, in order: a border is off by less
    than 2^-16 of the row (draws_ref.py: 2 (3 |y| + 65) + 3 |y| + 14 U, |y| < 11 on average at 20000 columns), 4096 / 2^15 of a number for two.
    4096 rows by k_sample, the others a CTA a row."""
    g = gen(vocab)
    row = (2 * torch.randn(vocab, generator=g)).to(TYPES[dtype])
    row[::3] = -math.inf
    row[7] = 9.0
    x = row.to(DEV).expand(rows, vocab).contiguous()
    u = (torch.arange(rows) + 0.5) / rows
    tokens = ce.sample_rows(x, u.to(DEV)).cpu()
    p = torch.softmax(row.double(), 0)
    counts = torch.bincount(tokens, minlength=vocab)
    assert float((counts - rows * p).abs().max()) <= 1.0 + 2.0 ** -3
    assert bool((tokens.diff() >= 0).all())
