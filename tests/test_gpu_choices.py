"""sample_rows, verify_drafts, route_rows and route_grad on the GPU against
their definitions in 64 bits (choices_ref.py): types, odd sizes, strides and
phases, masks, rows that are no distribution, every temperature, ragged
requests, groups and ties; whole distributions; a serving step of all of them;
captured, on another stream, from threads, and between guards."""
import math
import threading

import pytest
import torch

import choices_ref as R
import row_wise_softmax_ce_gb300 as ce
from objectives_ref import HALF_STEP, LEAST

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


def rows_of(rows, vocab, dtype, g, stride=None, lead=0, sigma=3.0, mask=0.0):
    """Rows inside a buffer of NaN and +1e4: what lies beside the columns must not be read."""
    stride = vocab if stride is None else stride
    buf = torch.full((lead + rows * stride + 16,), 1e4)
    buf[::2] = math.nan
    x = sigma * torch.randn(rows, vocab, generator=g)
    if mask:
        x[torch.rand(rows, vocab, generator=g) < mask] = -math.inf
    buf[lead:lead + rows * stride].view(rows, stride)[:, :vocab] = x
    dev = buf.to(dtype).to(DEV)
    return dev[lead:lead + rows * stride].view(rows, stride)[:, :vocab]


# -- sampling -------------------------------------------------------------------------

def sampled(x, u, T, logp=True):
    got = ce.sample_rows(x, u.to(DEV), temperature=T.to(DEV) if isinstance(T, torch.Tensor) else T, logp=logp)
    return [t.cpu() for t in got] if logp else (got.cpu(), None)


def check_all(x, u, T, tokens, logp):
    host = x.cpu()
    for r in range(len(u)):
        t = float(T[r]) if isinstance(T, torch.Tensor) else T
        R.check_sampled(host[r], float(u[r]), t, int(tokens[r]), None if logp is None else float(logp[r]), r)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 7), (4, 31), (4, 33), (7, 100), (9, 1000), (6, 4097),
                                        (3, 32000), (2, 50257), (40, 5003), (1, 200001)])
@pytest.mark.parametrize("T", [1.0, 0.6])
def test_sample(dtype, rows, vocab, T):
    g = gen(rows * 1000003 + vocab)
    x = rows_of(rows, vocab, TYPES[dtype], g, stride=vocab + rows % 4, lead=vocab % 5, mask=0.1 if vocab > 30 else 0.0)
    u = torch.rand(rows, generator=g)
    tokens, logp = sampled(x, u, T)
    check_all(x, u, T, tokens, logp)


@pytest.mark.parametrize("dtype", TYPES)
def test_sample_ends(dtype):
    """Numbers at and past the ends: 0, the last below 1, 1, below 0, NaN, infinities."""
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 7.0, -1.0, math.nan, math.inf, -math.inf, 2.0 ** -149, 0.5])
    for vocab in (1, 5, 3001, 60000):
        g = gen(vocab)
        x = rows_of(len(u), vocab, TYPES[dtype], g, sigma=1.0)
        if vocab > 4:
            x[:, 0] = x[:, 1] = x[:, -1] = -math.inf  # never drawn, whatever the number
        tokens, logp = sampled(x, u, 1.0)
        check_all(x, u, 1.0, tokens, logp)


@pytest.mark.parametrize("dtype", TYPES)
def test_sample_temperatures(dtype):
    g = gen(11)
    T = torch.tensor([0.0, 1.0, 0.0, 0.25, 4.0, 1e-6, 1e6, -1.0, math.nan, math.inf, 1e-7, 2e6, 0.0, 0.8])
    for vocab in (9, 2048, 40001):
        x = rows_of(len(T), vocab, TYPES[dtype], g, lead=1)
        x[2] = x[2].clamp(max=1.0)  # many equal largest values
        u = torch.rand(len(T), generator=g)
        tokens, logp = sampled(x, u, T)
        # at T = 1e-6 and 1e6 the softmax is one-hot, or flat
        check_all(x, u, T, tokens, logp)
        for r in (0, 2, 12):
            assert int(tokens[r]) == int(ce.argmax_rows(x[r:r + 1].float())[0])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [3, 40, 9000])
def test_sample_rows_that_are_none(dtype, vocab):
    g = gen(5)
    lowest = torch.finfo(TYPES[dtype]).min
    x = rows_of(8, vocab, TYPES[dtype], g, sigma=1.0)
    x[0] = -math.inf
    x[1, vocab // 2] = math.nan
    x[2, vocab - 1] = math.inf
    x[3] = lowest                       # a uniform distribution
    x[4] = lowest
    x[4, vocab - 1] = 0.0               # all of the mass in the last column
    x[5] = -math.inf
    x[5, vocab // 2] = 0.0
    x[6] = torch.finfo(TYPES[dtype]).max
    before = ce.device_error_count()[0]
    for T in (1.0, 0.0):
        u = torch.rand(8, generator=g)
        tokens, logp = sampled(x, u, T)
        check_all(x, u, T, tokens, logp)
    assert ce.device_error_count()[0] == before + 6


@pytest.mark.parametrize("vocab", [5, 700])
def test_sample_whole_distribution(vocab):
    """4096 evenly spaced numbers draw each column within one of its share of them."""
    n = 4096
    g = gen(vocab)
    row = 2 * torch.randn(vocab, generator=g)
    x = row.to(DEV).expand(n, vocab).contiguous()
    u = (torch.arange(n) + 0.5) / n
    tokens = ce.sample_rows(x, u.to(DEV)).cpu()
    p = torch.softmax(row.double(), 0)
    counts = torch.bincount(tokens, minlength=vocab)
    assert float((counts - n * p).abs().max()) <= 1.01
    assert bool((tokens.diff() >= 0).all())


def test_sample_outputs():
    g = gen(1)
    x = rows_of(6, 500, torch.float32, g)
    u = torch.rand(6, generator=g).to(DEV)
    out, lp = torch.empty(6, dtype=torch.int64, device=DEV), torch.empty(6, device=DEV)
    got = ce.sample_rows(x, u, logp=lp, out=out)
    assert got[0] is out or got[0].data_ptr() == out.data_ptr()
    assert got[1].data_ptr() == lp.data_ptr()
    ref, ref_lp = ce.sample_rows(x, u, logp=True)
    assert torch.equal(ref, out) and torch.equal(ref_lp, lp)
    assert torch.equal(ce.sample_rows(x, u), out)
    # the same log-probability as logp_rows gives the token
    assert float((ce.logp_rows(x, out) - lp).abs().max()) <= 2 * (R.adds(500) + 40) * R.U * 10
    assert ce.sample_rows(x[:0], u[:0]).shape == (0,)
    first = ce.sample_rows(x, u, vocab=77)
    assert int(first.max()) < 77 and torch.equal(first, ce.sample_rows(x[:, :77], u))


# -- verification ----------------------------------------------------------------------

def drafted(lengths, vocab, dtype, seed, lookup=False, noise=1.0, stride=None, lead=0, tail=0, T=1.0, mask=0.0, q_lead=None):
    """Requests of `lengths` rows (drafts and one more), with drafts drawn from the draft rows."""
    g = gen(seed)
    rows = sum(lengths) + tail
    x = rows_of(rows, vocab, dtype, g, stride, lead, mask=mask)
    ends = torch.tensor([0] + lengths).cumsum(0)
    near = x.cpu().float() + noise * torch.randn(rows, vocab, generator=g)
    y = rows_of(rows, vocab, dtype, g, stride, lead if q_lead is None else q_lead)
    y.copy_(near)
    t = T if isinstance(T, torch.Tensor) else torch.full((rows,), float(T))
    warm = torch.where(t > 0, t, torch.ones(()))
    q = torch.softmax(y.cpu().double() / warm.clamp(1e-6, 1e6)[:, None].double(), 1).nan_to_num(0.0) + 1e-30
    drafts = torch.multinomial(q, 1, generator=g)[:, 0]
    if lookup:
        likely = torch.where(torch.rand(rows, generator=g) < 0.7, x.cpu().float().nan_to_num(0.0).argmax(1), drafts)
        drafts = likely
    for s, n in enumerate(lengths):
        if n:
            drafts[int(ends[s + 1]) - 1] = -1
    u = torch.rand(rows, 2, generator=g)
    return x, drafts, ends, u, None if lookup else y, t


def verified(x, drafts, ends, u, y, T, logp=True):
    got = ce.verify_drafts(x, drafts.to(DEV), ends.to(DEV), u.to(DEV), draft_logits=y,
                           temperature=T.to(DEV) if isinstance(T, torch.Tensor) else T, logp=logp)
    return [None if t is None else t.cpu() for t in got]


def check_batch(batch, T=None):
    x, drafts, ends, u, y, t = batch
    accepted, tokens, logp = verified(x, drafts, ends, u, y, t if T is None else T)
    host = x.cpu()
    return R.check_verified(host, drafts, ends, u, None if y is None else y.cpu(), t, accepted, tokens, logp)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("lengths,vocab", [([1], 1), ([2], 5), ([3, 1, 2], 33), ([5, 5, 5, 5], 1000), ([9, 2, 1, 4], 4099),
                                           ([3, 4], 32000), ([2, 3], 50257), ([4] * 40, 611), ([2] * 90, 2003)])
def test_verify(dtype, lookup, lengths, vocab):
    seed = vocab + len(lengths)
    ends = check_batch(drafted(lengths, vocab, TYPES[dtype], seed, lookup, stride=vocab + vocab % 3, lead=vocab % 7,
                               tail=seed % 3, mask=0.05 if vocab > 30 else 0.0), T=1.0)
    if len(lengths) >= 40:
        assert {"accepted", "rest"} <= set(ends)
    if len(lengths) == 90:
        assert "drawn" in ends  # behind a request's last draft


@pytest.mark.parametrize("dtype", TYPES)
def test_verify_phases(dtype):
    """Target and draft rows of different strides and starts: columns that share no 16-byte vector."""
    for lead, q_lead, pad in ((0, 1, 0), (3, 0, 1), (1, 6, 5), (2, 2, 3)):
        x, d, ends, u, y, t = drafted([3, 2, 4], 1201, TYPES[dtype], lead + 10, stride=1201 + pad, lead=lead, q_lead=q_lead)
        check_batch((x, d, ends, u, y.contiguous(), t), T=1.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("lookup", [False, True])
def test_verify_temperatures(dtype, lookup):
    lengths = [3, 2, 4, 1, 3, 2, 2, 5]
    per = [0.0, 0.7, 1.5, 0.0, math.nan, 1e-6, -2.0, 0.0]
    T = torch.tensor(per).repeat_interleave(torch.tensor(lengths))
    for vocab in (13, 3000):
        batch = drafted(lengths, vocab, TYPES[dtype], vocab, lookup, T=T)
        x, drafts, ends, u, y, t = batch
        for s in (0, 7):  # greedy requests whose first drafts are right
            for r in range(int(ends[s]), int(ends[s + 1]) - 1 - (s == 7)):
                drafts[r] = int(x[r].float().cpu().nan_to_num(-1e9).argmax())
        x[int(ends[7]) + 1] = x[int(ends[7]) + 1].clamp(max=0.5)  # equal largest values
        how = check_batch((x, drafts, ends, u, y, T))
        assert "greedy" in how and "bad" in how


@pytest.mark.parametrize("dtype", TYPES)
def test_verify_rows_that_are_none(dtype):
    lowest = torch.finfo(TYPES[dtype]).min
    for vocab in (6, 5000):
        x, drafts, ends, u, y, t = drafted([3] * 8, vocab, TYPES[dtype], vocab + 1, noise=0.5)
        u[:, 0] = 0.01          # accept what can be
        x[0] = -math.inf
        x[4, 1] = math.nan
        x[6, vocab - 1] = math.inf
        y[9] = -math.inf        # a draft row that is no distribution
        y[12, 2] = math.nan
        y[15] = lowest
        x[18] = lowest
        drafts[21] = vocab      # a draft that is no token
        drafts[22] = 1 << 40
        before = ce.device_error_count()[0]
        check_batch((x, drafts, ends, u, y, t), T=1.0)
        assert ce.device_error_count()[0] > before


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [4, 2500])
def test_verify_same_rows(dtype, vocab):
    """Where target and draft rows are the same every draft is accepted, and a number of 1 or NaN that
    accepts nothing draws from p."""
    x, drafts, ends, u, y, t = drafted([4, 3, 5], vocab, TYPES[dtype], 3)
    u[:, 0] *= 0.999
    accepted, tokens, _ = verified(x, drafts, ends, u, x.clone(), 1.0)
    assert accepted.tolist() == [3, 2, 4]
    u[:, 0] = torch.tensor([1.0, math.nan] * 6)
    accepted, tokens, _ = verified(x, drafts, ends, u, x.clone(), 1.0)
    assert accepted.tolist() == [0, 0, 0]
    for r in (0, 4, 7):
        R.check_sampled(x[r].cpu(), float(u[r, 1]), 1.0, int(tokens[r]), None, r)


def test_verify_one_column_left():
    """Looked-up drafts that hold all of the mass, and none of it."""
    x = torch.full((4, 300), -math.inf, device=DEV)
    x[:, 7] = 0.0
    x[2:, 9] = -1.0
    drafts = torch.tensor([7, 9, 7, 9])
    u = torch.tensor([[1.0, 0.5], [0.5, 0.5], [0.9, 0.2], [0.5, 0.99]])
    accepted, tokens, logp = verified(x, drafts, torch.tensor([0, 1, 2, 3, 4]), u, None, 1.0)
    # 1.0 < p = 1 fails, and nothing but the draft is left; p(9) = 0; p(7) = 0.73 < 0.9; p(9) = 0.27 < 0.5
    assert accepted.tolist() == [0, 0, 0, 0]
    assert tokens.tolist() == [7, 7, 9, 7]
    R.check_logp(x[2].cpu(), 1.0, 9, float(logp[2]), "left")


@pytest.mark.parametrize("lookup", [False, True])
def test_verify_drafts_that_cannot_be(lookup):
    """A draft that the target bans is not accepted, whatever the number; one that the draft row bans is."""
    x, drafts, _, u, y, t = drafted([6], 900, torch.float32, 4, lookup)
    drafts = torch.full((6,), 33)
    x[:, 33] = -math.inf
    for a in (0.0, -1.0, -math.inf, 0.5, math.nan, math.inf):
        u[:, 0] = a
        accepted, tokens, _ = verified(x, drafts, torch.arange(7), u, y, 1.0)
        assert accepted.tolist() == [0] * 6 and bool((tokens != 33).all()) and bool((tokens >= 0).all())
    if not lookup:
        x[:, 33] = 0.0
        y[:, 33] = -math.inf
        u[:, 0] = 0.999
        accepted, tokens, _ = verified(x, drafts, torch.arange(7), u, y, 1.0)
        assert accepted.tolist() == [1] * 6 and tokens.tolist() == [33] * 6


def test_longest_rows():
    """2^24 columns: more steps than a warp holds at hand."""
    V = 1 << 24
    x = torch.randn(3, V, device=DEV)
    x[1, :V - 5] = -math.inf
    u = torch.tensor([0.3, 0.6, 0.999])
    tokens, logp = sampled(x, u, 0.9)
    check_all(x, u, 0.9, tokens, logp)
    assert int(ce.sample_rows(x, u.to(DEV), temperature=0.0)[2]) == int(x[2].argmax())
    y = (x + 0.3 * torch.randn(3, V, device=DEV)).nan_to_num(neginf=-50.0)
    drafts = torch.tensor([int(y[0].argmax()), 5, -1])
    check_batch((x, drafts, torch.tensor([0, 1, 2, 3]), torch.tensor([[0.99, 0.2], [0.5, 0.5], [0.0, 0.7]]), y, torch.ones(3)), T=1.0)


def test_past_2_31_elements():
    """Rows that cross the 2^31st element and lie behind it."""
    rows, V = 17000, 131073
    x = torch.empty(rows, V + 7, dtype=torch.bfloat16, device=DEV)
    for a in range(0, rows, 2000):
        x[a:a + 2000].normal_(generator=torch.Generator(DEV).manual_seed(a))
    x = x[:, :V]
    g = gen(1)
    u = torch.rand(rows, generator=g)
    tokens, logp = sampled(x, u, 0.5)
    assert int(tokens.min()) >= 0 and int(tokens.max()) < V
    some = [0, 16382, 16383, 16384, 16999]
    for r in some:
        R.check_sampled(x[r].cpu(), float(u[r]), 0.5, int(tokens[r]), float(logp[r]), r)
    drafts = torch.full((rows,), -1)
    drafts[some] = torch.tensor([int(x[r].argmax()) for r in some])
    pairs = torch.stack([u, u.flip(0)], 1)
    pairs[:, 0] *= 1e-5
    accepted, got, _ = verified(x, drafts, torch.arange(rows + 1), pairs, x, 0.5, logp=False)
    assert accepted.nonzero()[:, 0].tolist() == some and got[some].tolist() == drafts[some].tolist()
    del x
    z = torch.empty(2100000, 1024, dtype=torch.bfloat16, device=DEV).normal_(generator=torch.Generator(DEV).manual_seed(5))
    chosen, gates, counts = ce.route_rows(z, 4, counts=True)
    assert int(counts.sum()) == 4 * z.shape[0]
    tail = ce.route_rows(z[-64:], 4)
    assert torch.equal(chosen[-64:], tail[0]) and torch.equal(gates[-64:], tail[1])
    G = torch.ones_like(gates)
    G[:, 0] = 2.0
    for renorm in (True, False):
        end = ce.route_grad(z[-64:], tail[0], G[-64:], renormalise=renorm)
        got = ce.route_grad(z, chosen, G, renormalise=renorm)
        assert torch.equal(got[-64:], end)
        del got


@pytest.mark.parametrize("lookup", [False, True])
def test_verify_whole_distribution(lookup):
    """Over a grid of number pairs and every draft, what is emitted is distributed as the target."""
    V, n = 5, 96
    p, q = torch.tensor([0.1, 0.35, 0.05, 0.3, 0.2]), torch.tensor([0.3, 0.1, 0.25, 0.05, 0.3])
    grid = (torch.arange(n) + 0.5) / n
    a, b = torch.meshgrid(grid, grid, indexing="ij")
    rows = V * n * n
    x, y = p.log().expand(rows, V).contiguous().to(DEV), q.log().expand(rows, V).contiguous().to(DEV)
    drafts = torch.arange(V).repeat_interleave(n * n)
    u = torch.stack([a.flatten(), b.flatten()], 1).repeat(V, 1)
    ends = torch.arange(rows + 1)
    accepted, tokens, _ = verified(x, drafts, ends, u, None if lookup else y, 1.0, logp=False)
    out = torch.zeros(V, dtype=torch.float64)
    for d in range(V):
        hit = torch.bincount(tokens[d * n * n:(d + 1) * n * n], minlength=V).double() / (n * n)
        want = float(p[d]) if lookup else min(1.0, float(p[d] / q[d]))
        assert abs(float(accepted[d * n * n:(d + 1) * n * n].double().mean()) - want) <= 1.01 / n
        # a draft that is always the same token is accepted by p and replaced by the rest
        out += hit * (0.2 if lookup else float(q[d]))
        if lookup:
            assert float((hit - p).abs().max()) <= 3.0 / n
    if not lookup:
        assert float((out - p).abs().max()) <= 3.0 / n


def test_verify_layouts():
    """No requests, empty requests, rows in none, and a last row that has a draft."""
    x, drafts, _, u, y, t = drafted([12], 400, torch.float32, 9, noise=0.2)
    drafts = x.cpu().argmax(1)
    u[:, 0] = 0.0  # everything that weighs anything is accepted
    ends = torch.tensor([2, 2, 5, 5, 9, 9])
    accepted, tokens, logp = verified(x, drafts, ends, u, y, 1.0)
    assert accepted.tolist() == [0, 3, 0, 4, 0]
    assert tokens.tolist() == [-1, -1] + drafts[2:9].tolist() + [-1] * 3
    assert float(logp[9:].abs().sum()) == 0 and float(logp[:2].abs().sum()) == 0
    none = verified(x, drafts, torch.tensor([4]), u, y, 1.0)
    assert none[0].shape == (0,) and none[1].tolist() == [-1] * 12
    empty = verified(x[:0], drafts[:0], torch.tensor([0, 0, 0]), u[:0], None, 1.0)
    assert empty[0].tolist() == [0, 0] and empty[1].shape == (0,)
    # drafts in the padding of a fixed layout: a request stops at its first row without one
    drafts[4] = -1
    accepted, tokens, _ = verified(x, drafts, torch.tensor([2, 9]), u, y, 1.0)
    assert accepted.tolist() == [2] and tokens[:4].tolist() == [-1, -1] + drafts[2:4].tolist()
    assert int(tokens[4]) >= 0 and tokens[5:].tolist() == [-1] * 7


@pytest.mark.parametrize("ends", [[0, 5, 3, 8], [-4, 2, 8], [0, 4, 900], [0, 1 << 40, 8], [8, 0], [3, -(1 << 50), 8]])
def test_verify_bad_tables(ends):
    """Nothing out of range is read or written; valid ranges of the table keep their lengths' bounds."""
    x, drafts, _, u, y, t = drafted([8], 300, torch.bfloat16, 2)
    buf = torch.full((40,), -77, dtype=torch.int64, device=DEV)
    before = ce.device_error_count()[0]
    accepted, tokens, _ = verified(x, drafts, torch.tensor(ends), u, y, 1.0)
    bad = [not (0 <= a <= b <= 8) for a, b in zip(ends, ends[1:])]
    assert [int(v) == -1 for v in accepted] == bad
    assert ce.device_error_count()[0] == before + sum(bad)
    assert bool(((tokens >= -1) & (tokens < 300)).all()) and bool((buf == -77).all())


def test_verify_large():
    """Sizes of a serving batch; every row checked."""
    batch = drafted([5] * 20 + [3] * 9, 30011, torch.bfloat16, 77, noise=0.7)
    check_batch(batch, T=1.0)


# -- routing ---------------------------------------------------------------------------

def routers():
    for E, k in ((1, 1), (4, 2), (8, 2), (31, 5), (60, 4), (64, 6), (64, 32), (128, 8), (160, 6), (256, 8), (257, 3), (384, 8),
                 (513, 9), (1024, 16), (1023, 32)):
        yield E, k, 1, 1
    for E, k, G, t in ((8, 2, 4, 2), (64, 6, 8, 3), (60, 4, 4, 2), (160, 6, 8, 3), (256, 8, 8, 4), (256, 8, 32, 5), (96, 5, 3, 1),
                       (1024, 12, 16, 4), (20, 2, 20, 3), (256, 16, 2, 1)):
        yield E, k, G, t


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,t", list(routers()))
def test_route(dtype, score, E, k, G, t):
    g = gen(E * 100 + k)
    rows = 33 if E < 500 else 11
    for bias, top, renorm, mask, pad in ((False, 2, True, 0.0, 0), (True, 2, True, 0.1, 3), (True, 1, False, 0.0, 1),
                                         (False, 1, False, 0.3, 0)):
        x = rows_of(rows, E, TYPES[dtype], g, stride=E + pad, lead=pad, sigma=1.5, mask=mask)
        b = 0.2 * torch.randn(E, generator=g) if bias else None
        w = (torch.rand(rows, generator=g) > 0.1).float() if mask else None
        kw = dict(score=score, groups=G, top_groups=t, group_top=top, renormalise=renorm, scale=1.25)
        chosen, gates, counts = ce.route_rows(x, k, bias=None if b is None else b.to(DEV),
                                              weights=None if w is None else w.to(DEV), counts=True, **kw)
        R.check_routed(x.cpu(), k, chosen.cpu(), gates.cpu(), counts.cpu(), bias=b, weights=w, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G,t", [(1, 1), (4, 2)])
def test_route_ties(dtype, G, t):
    """Few different values: the lowest expert of equals comes first, in groups too."""
    g = gen(8)
    x = torch.randint(-2, 3, (64, 32), generator=g).float()
    x[0] = 0.0
    x[1] = -0.0
    x[2, ::2] = 0.0
    x[2, 1::2] = -0.0
    x = x.to(TYPES[dtype])
    for score in ("softmax", "sigmoid"):
        kw = dict(score=score, groups=G, top_groups=t)
        chosen, gates, _ = ce.route_rows(x.to(DEV), 6, **kw)
        R.check_routed(x, 6, chosen.cpu(), gates.cpu(), None, **kw)
        assert chosen[0].tolist() == list(range(6)) == chosen[1].tolist() == chosen[2].tolist()
        zero = torch.zeros(32, device=DEV)
        assert torch.equal(ce.route_rows(x.to(DEV), 6, bias=zero, **kw)[0], chosen)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("G,t", [(1, 1), (4, 2)])
def test_route_extremes(dtype, score, G, t):
    top = torch.finfo(TYPES[dtype])
    g = gen(3)
    x = torch.randn(12, 40, generator=g)
    x[0] = -math.inf                    # nothing to choose
    x[1] = -math.inf
    x[1, 33] = 0.0                      # one expert left
    x[2, 5] = math.nan
    x[3, 39] = math.inf
    x[4] = top.min                      # masks of the lowest value
    x[4, 7] = 1.0
    x[5] = top.min
    x[6] = top.max
    x[7, :20] = -math.inf               # whole groups masked
    x[8] = -80.0 + x[8]                 # sigmoids next to nothing, their shares are not
    x[9] = 30.0 + x[9]                  # sigmoids that round to 1
    x[10] = -200.0 + x[10]
    x = x.to(TYPES[dtype])
    before = ce.device_error_count()[0]
    for renorm in (True, False):
        kw = dict(score=score, groups=G, top_groups=t, renormalise=renorm)
        chosen, gates, counts = ce.route_rows(x.to(DEV), 5, counts=True, **kw)
        R.check_routed(x, 5, chosen.cpu(), gates.cpu(), counts.cpu(), **kw)
        if renorm:
            assert float((gates[[8, 9, 10]].sum(1) - 1).abs().max()) <= 1e-6
    assert ce.device_error_count()[0] == before + 4
    # a bias that bans, and one that is no number
    b = torch.zeros(40)
    b[3], b[4], b[9] = -math.inf, math.nan, math.inf
    kw = dict(score=score, groups=G, top_groups=t, bias=b)
    chosen, gates, _ = ce.route_rows(x.to(DEV), 5, **{**kw, "bias": b.to(DEV)})
    assert not bool(((chosen == 3) | (chosen == 4)).any())
    ok = [8, 9, 11] if score == "sigmoid" else [8, 9, 10, 11]
    assert bool((chosen[ok][:, 0] == 9).all())


def test_route_no_rows_and_padding():
    x = torch.randn(5, 16, device=DEV)
    chosen, gates, counts = ce.route_rows(x[:0], 3, counts=True)
    assert chosen.shape == (0, 3) and gates.shape == (0, 3) and counts.tolist() == [0] * 16
    w = torch.tensor([1.0, 0.0, -0.0, 5.0, math.nan], device=DEV)
    x[1] = math.nan  # padding is not read
    chosen, gates, counts = ce.route_rows(x, 3, weights=w, counts=True)
    assert (chosen[:, 0] >= 0).tolist() == [True, False, False, True, True]
    assert int(counts.sum()) == 9
    grad = ce.route_grad(x, chosen, torch.randn(5, 3, device=DEV), renormalise=False, weights=w)
    assert (grad.abs().sum(1) > 0).tolist() == [True, False, False, True, True]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (7, 3), (60, 4), (64, 32), (130, 6), (256, 8), (384, 8), (1024, 9), (777, 32)])
def test_route_grad(dtype, score, renorm, E, k):
    g = gen(E + k)
    rows = 21
    for pad, mask in ((0, 0.0), (3, 0.2)):
        x = rows_of(rows, E, TYPES[dtype], g, stride=E + pad, lead=pad, sigma=1.5, mask=mask if E > 1 else 0.0)
        w = (torch.rand(rows, generator=g) > 0.15).float() if pad else None
        kw = dict(score=score, renormalise=renorm, scale=2.5)
        chosen, _, _ = ce.route_rows(x, k, weights=None if w is None else w.to(DEV), **kw)
        if pad:
            chosen[3] = -1
            chosen[4, 0] = chosen[4, -1]  # an expert named twice
            chosen[5, :] = int(chosen[5, 0])
        G = torch.randn(rows, k, generator=g)
        got = ce.route_grad(x, chosen, G.to(DEV), weights=None if w is None else w.to(DEV), **kw)
        want, err = R.route_grad64(x.cpu(), chosen.cpu(), G, weights=w, **kw)
        bound = err + HALF_STEP[TYPES[dtype]] * (want.abs() + err) + LEAST[TYPES[dtype]]
        assert got.dtype == TYPES[dtype] and got.is_contiguous()
        assert bool(((got.cpu().double() - want).abs() <= bound).all())
        # in place, and into rows of another stride, whose padding stays
        wide = torch.full((rows, E + 5), 7.0, dtype=TYPES[dtype], device=DEV)
        ce.route_grad(x, chosen, G.to(DEV), weights=None if w is None else w.to(DEV), grad=wide, **kw)
        assert torch.equal(wide[:, :E], got) and bool((wide[:, E:] == 7.0).all())
        ce.route_grad(x, chosen, G.to(DEV), weights=None if w is None else w.to(DEV), grad=x, **kw)
        assert torch.equal(x, got)


def test_route_grad_against_differences():
    """The kernel's gates, moved by a step of each logit of a row."""
    g = gen(6)
    E, k, h = 24, 4, 1.0 / 64
    x = 1.5 * torch.randn(1, E, generator=g)
    G = torch.randn(1, k, generator=g)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            chosen, _, _ = ce.route_rows(x.to(DEV), k, score=score, renormalise=renorm)
            grad = ce.route_grad(x.to(DEV), chosen, G.to(DEV), score=score, renormalise=renorm).cpu()[0]
            steps = x.repeat(2 * E, 1)
            at = torch.arange(E)
            steps[at, at] += h
            steps[at + E, at] -= h
            both, gates, _ = ce.route_rows(steps.to(DEV), k, score=score, renormalise=renorm)
            # the choice may change its order for a step, not its members' gates
            value = torch.zeros(2 * E)
            for r in range(2 * E):
                of = dict(zip(both[r].tolist(), gates[r].tolist()))
                if set(of) != set(chosen[0].tolist()):
                    value[r] = math.nan
                    continue
                value[r] = sum(float(G[0, i]) * of[c] for i, c in enumerate(chosen[0].tolist()))
            num = (value[:E] - value[E:]) / (2 * h)
            ok = ~torch.isnan(num)
            assert int(ok.sum()) >= E - 6
            # h^2 / 6 of a third derivative below 1 times sum |G| (< 10), and U sum |G| / h of rounding, with room for
            # the shares' further steps
            assert float((num - grad)[ok].abs().max()) <= 10 * h * h + 10 * R.U * 8 / h


def test_route_grad_bad_experts():
    x = torch.randn(3, 10, device=DEV)
    chosen = torch.tensor([[2, 10], [-5, 3], [1 << 40, -1]], device=DEV)
    G = torch.randn(3, 2)
    before = ce.device_error_count()[0]
    got = ce.route_grad(x, chosen, G.to(DEV), renormalise=False)
    assert ce.device_error_count()[0] == before + 3
    want, err = R.route_grad64(x.cpu(), chosen.cpu(), G, renormalise=False)
    assert bool(((got.cpu().double() - want).abs() <= err + 2.0 ** -24 * want.abs()).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,k", [(40, 5), (256, 8), (600, 20)])
def test_route_grad_no_experts(dtype, score, renorm, E, k):
    """Zeros in a row that chose nothing, whatever it holds, beside rows that did."""
    x = torch.randn(6, E, generator=gen(E)).to(TYPES[dtype]).to(DEV)
    x[1, 5] = math.nan
    x[2, 6] = math.inf
    x[3] = -math.inf
    x[4, :] = torch.finfo(TYPES[dtype]).max
    kw = dict(score=score, renormalise=renorm)
    chosen, _, _ = ce.route_rows(x, k, **kw)
    chosen[4] = -1
    assert (chosen[:, 0] >= 0).tolist() == [True, False, False, False, False, True]
    got = ce.route_grad(x, chosen, torch.full((6, k), math.nan, device=DEV).where(chosen < 0, torch.ones((), device=DEV)), **kw)
    assert bool((got[1:5] == 0).all()) and not bool(torch.isnan(got).any())


# -- drawn cases ---------------------------------------------------------------------------

@pytest.mark.parametrize("seed", range(20))
def test_drawn_choices(seed):
    """Drawn sizes, types, strides, phases, masks, temperatures and requests."""
    import random
    rng = random.Random(seed)
    g = gen(seed)
    dtype = rng.choice(list(TYPES.values()))
    vocab = int(round(math.exp(rng.uniform(0, math.log(40000)))))
    pad, lead = rng.choice([0, 0, 1, 5, 64]), rng.randint(0, 9)
    lengths = [rng.choice([0, 1, 1, 2, 3, 5, 9]) for _ in range(rng.randint(1, 12))]
    rows = sum(lengths)
    per = torch.tensor([rng.choice([0.0, 0.5, 1.0, 1.0, 1.7, 30.0]) for _ in lengths])
    T = per.repeat_interleave(torch.tensor(lengths))
    mask = rng.choice([0.0, 0.0, 0.3, 0.97])
    lookup = rng.random() < 0.3
    x, drafts, ends, u, y, t = drafted(lengths, vocab, dtype, seed, lookup, noise=rng.choice([0.2, 1.0, 3.0]), stride=vocab + pad,
                                       lead=lead, q_lead=rng.choice([lead, 0, 3]), tail=0, T=T, mask=mask)
    check_batch((x, drafts, ends, u, y, T))
    if rows:
        draws = torch.rand(rows, generator=g)
        tokens, logp = sampled(x, draws, T)
        check_all(x, draws, T, tokens, logp)


@pytest.mark.parametrize("seed", range(20))
def test_drawn_routing(seed):
    import random
    rng = random.Random(1000 + seed)
    g = gen(seed)
    dtype = rng.choice(list(TYPES.values()))
    G = rng.choice([1, 1, 2, 4, 5, 8, 16, 32])
    E = G * rng.randint(1, max(1, min(60, 1024 // G)))
    tg = rng.randint(1, G)
    k = rng.randint(1, min(32, tg * (E // G)))
    rows = rng.choice([1, 3, 17, 64])
    pad = rng.choice([0, 0, 1, 8])
    kw = dict(score=rng.choice(["softmax", "sigmoid"]), renormalise=rng.random() < 0.5, scale=rng.choice([1.0, 2.5, -0.5]))
    x = rows_of(rows, E, dtype, g, stride=E + pad, lead=rng.randint(0, 9), sigma=rng.choice([0.3, 1.5, 6.0]), mask=rng.choice([0.0, 0.2, 0.9]))
    if rng.random() < 0.4:  # few different values
        x.copy_(x.float().nan_to_num(neginf=-9.0).round().clamp(-2, 2))
    b = rng.choice([0.0, 0.1, 5.0]) * torch.randn(E, generator=g) if rng.random() < 0.5 else None
    w = (torch.rand(rows, generator=g) > 0.2).float() if rng.random() < 0.5 else None
    dw = None if w is None else w.to(DEV)
    chosen, gates, counts = ce.route_rows(x, k, bias=None if b is None else b.to(DEV), groups=G, top_groups=tg,
                                          group_top=rng.choice([1, 2]) if tg == G else (top := rng.choice([1, 2])), weights=dw, counts=True, **kw)
    R.check_routed(x.cpu(), k, chosen.cpu(), gates.cpu(), counts.cpu(), bias=b, groups=G, top_groups=tg,
                   group_top=2 if tg == G else top, weights=w, **kw)
    grads = torch.randn(rows, k, generator=g)
    got = ce.route_grad(x, chosen, grads.to(DEV), weights=dw, **kw)
    want, err = R.route_grad64(x.cpu(), chosen.cpu(), grads, weights=w, **kw)
    bound = err + HALF_STEP[dtype] * (want.abs() + err) + LEAST[dtype]
    assert bool(((got.cpu().double() - want).abs() <= bound).all())


def test_route_many_rows():
    """Row counts around those that change the shape, against calls of a few rows."""
    g = gen(2)
    for E, kw in ((256, dict(score="sigmoid", groups=8, top_groups=4)), (60, dict(renormalise=False)), (128, dict())):
        x = rows_of(3001, E, torch.bfloat16, g, sigma=1.5)
        b = (0.1 * torch.randn(E, generator=g)).to(DEV)
        chosen, gates, counts = ce.route_rows(x, 8, bias=b, counts=True, **kw)
        total = torch.zeros_like(counts)
        for a in range(0, 3001, 100):
            c, t, n = ce.route_rows(x[a:a + 100], 8, bias=b, counts=True, **kw)
            assert torch.equal(c, chosen[a:a + 100]) and torch.equal(t, gates[a:a + 100])
            total += n
        assert torch.equal(total, counts)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E,k,G,t", [(16, 4, 1, 1), (31, 1, 1, 1), (32, 8, 4, 1), (60, 4, 1, 1), (60, 4, 4, 2), (64, 6, 1, 1), (64, 8, 4, 2),
                                     (64, 3, 8, 3), (100, 5, 1, 1), (128, 8, 4, 2), (127, 2, 1, 1), (128, 9, 1, 1)])
def test_route_small_rows_in_numbers(dtype, E, k, G, t):
    """Many rows of few experts, eight to a warp: a part of them against the definition, the rest among themselves."""
    g = gen(E + k)
    rows, part = 10007, 48
    x = rows_of(part, E, TYPES[dtype], g, sigma=1.5, mask=0.05)
    x[3] = -math.inf
    x[7, E // 2] = math.nan
    x[8, E - 1] = math.inf
    x[9:20] = x[9:20].float().round().to(TYPES[dtype])  # ties
    w = torch.ones(part)
    w[30], w[44] = 0.0, 0.0
    b = 0.2 * torch.randn(E, generator=g)
    at = torch.arange(rows) % part
    for score, bias, renorm, pad in (("sigmoid", b, True, 0), ("softmax", None, False, 1), ("softmax", b, True, 0)):
        many = torch.zeros(rows, E + pad, dtype=TYPES[dtype])
        many[:, :E] = x.cpu()[at]
        kw = dict(score=score, groups=G, top_groups=t, renormalise=renorm)
        chosen, gates, counts = ce.route_rows(many.to(DEV)[:, :E], k, bias=None if bias is None else bias.to(DEV),
                                              weights=w[at].to(DEV), counts=True, **kw)
        assert torch.equal(counts, torch.bincount(chosen[chosen >= 0], minlength=E))
        chosen, gates = chosen.cpu(), gates.cpu()
        of = torch.bincount(chosen[:part][chosen[:part] >= 0], minlength=E)
        R.check_routed(x.cpu(), k, chosen[:part], gates[:part], of, bias=bias, weights=w, **kw)
        assert torch.equal(chosen, chosen[:part][at])
        assert torch.equal(gates.view(torch.int32), gates[:part][at].view(torch.int32))


# -- together, and how they are called ---------------------------------------------------

def step(x, y, ends, u, draws, router, w, G):
    """Drafts drawn from the draft rows, verified against the target's, and the rows' routing with its gradient."""
    drafts = ce.sample_rows(y, draws, temperature=0.8)
    drafts = drafts.masked_fill(torch.zeros_like(drafts).index_fill_(0, ends[1:] - 1, 1).bool(), -1)
    accepted, tokens, logp = ce.verify_drafts(x, drafts, ends, u, draft_logits=y, temperature=0.8, logp=True)
    chosen, gates, counts = ce.route_rows(router, 4, score="sigmoid", bias=w, groups=4, top_groups=2, counts=True)
    grad = ce.route_grad(router, chosen, G, score="sigmoid")
    return [drafts, accepted, tokens, logp, chosen, gates, counts, grad]


def step_inputs(seed, vocab=5003):
    g = gen(seed)
    lengths = [4, 2, 5, 1, 3]
    x = rows_of(15, vocab, torch.bfloat16, g).to(DEV)
    y = (x.float() + 0.7 * torch.randn(15, vocab, generator=g).to(DEV)).bfloat16()
    ends = torch.tensor([0] + lengths).cumsum(0).to(DEV)
    u, draws = torch.rand(15, 2, generator=g).to(DEV), torch.rand(15, generator=g).to(DEV)
    router = torch.randn(15, 64, generator=g).to(DEV)
    return [x, y, ends, u, draws, router, 0.1 * torch.randn(64, generator=g).to(DEV), torch.randn(15, 4, generator=g).to(DEV)]


def test_serving_step():
    inputs = step_inputs(1)
    x, y, ends, u, draws, router, b, G = inputs
    drafts, accepted, tokens, logp, chosen, gates, counts, grad = [t.cpu() for t in step(*inputs)]
    for r in range(15):
        if int(drafts[r]) >= 0:
            R.check_sampled(y[r].cpu(), float(draws[r]), 0.8, int(drafts[r]), None, r)
    R.check_verified(x.cpu(), drafts, ends.cpu(), u.cpu(), y.cpu(), [0.8] * 15, accepted, tokens, logp)
    # what is emitted goes on as a policy's sampled tokens: its log-probabilities are logp_rows'
    on = tokens >= 0
    same = ce.logp_rows(x, tokens.clamp(min=0).to(DEV), weights=on.float().to(DEV), temperature=0.8).cpu()
    assert float((same - logp).abs().max()) <= 1e-5
    kw = dict(score="sigmoid", groups=4, top_groups=2)
    R.check_routed(router.cpu(), 4, chosen, gates, counts, bias=b.cpu(), **kw)
    want, err = R.route_grad64(router.cpu(), chosen, G.cpu(), score="sigmoid")
    assert bool(((grad.double() - want).abs() <= err + 2.0 ** -24 * want.abs()).all())


def test_captured_and_replayed():
    """One capture, replayed on new contents of its inputs; two graphs side by side."""
    a, b = step_inputs(1), step_inputs(2)
    want = [[t.clone() for t in step(*v)] for v in (a, b)]
    held = [t.clone() for t in a]
    graphs, outs = [], []
    for inputs in (held, [t.clone() for t in b]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(*inputs))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for out, ref in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(out, ref))
    for dst, src in zip(held, b):
        dst.copy_(src)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(outs[0], want[1]))


def test_first_calls_captured():
    """No call of the process before the capture: the graph's results are the eager calls'."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    program = """
import sys
sys.path[:0] = ['.', 'tests']
import torch
import test_gpu_choices as C
import row_wise_softmax_ce_gb300 as ce
inputs = C.step_inputs(4)
wide = torch.randn(40, 1000, device='cuda')
def everything():
    return C.step(*inputs) + [ce.sample_rows(wide, torch.full((40,), 0.4, device='cuda'))] + list(
        ce.route_rows(wide, 32, counts=True)) + [ce.route_grad(wide, torch.zeros(40, 8, dtype=torch.int64, device='cuda'),
        torch.ones(40, 8, device='cuda'))] + [ce.route_grad(wide, torch.zeros(40, 1, dtype=torch.int64, device='cuda'),
        torch.ones(40, 1, device='cuda'), renormalise=False)]
ce.lib()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = everything()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, everything()))
print("same", *ce.device_error_count())
"""
    r = subprocess.run([sys.executable, "-c", program], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.split() == ["same", "0", "0"]


def test_streams_and_threads():
    """The same bits on every stream and from every thread, side by side."""
    sets = [step_inputs(s, vocab=20011) for s in range(4)]
    want = [[t.clone() for t in step(*v)] for v in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(6):
                got = step(*sets[i])
                stream.synchronize()
                if not all(torch.equal(p, q) for p, q in zip(got, want[i])):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("cap", [1, 2, 5])
def test_grid_cap(cap):
    """Few clusters that take many rows each: the same bits."""
    inputs = step_inputs(3, vocab=9001)
    want = [t.clone() for t in step(*inputs)]
    ce.debug_grid_cap(cap)
    try:
        got = step(*inputs)
        torch.cuda.synchronize()
    finally:
        ce.debug_grid_cap(0)
    # the row's split follows its rows, not the cap
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert ce.device_error_count()[1] == 0


def test_binding_refusals():
    x = torch.randn(6, 16, device=DEV)
    u, d, e = torch.rand(6, device=DEV), torch.zeros(6, dtype=torch.int64, device=DEV), torch.tensor([0, 6], device=DEV)
    u2 = torch.rand(6, 2, device=DEV)
    for bad in (dict(uniforms=u[1:]), dict(uniforms=u.double()), dict(uniforms=u.cpu()), dict(uniforms=u2), dict(logp=u[1:]),
                dict(out=u), dict(out=d[1:]), dict(temperature=u[1:]), dict(vocab=17), dict(logits=x.t())):
        with pytest.raises(ValueError):
            ce.sample_rows(**{**dict(logits=x, uniforms=u), **bad})
    for bad in (dict(temperature=-1.0), dict(temperature=math.nan), dict(logp=u)):
        with pytest.raises(ce.CeError):
            ce.sample_rows(**{**dict(logits=x, uniforms=u), **bad})
    for bad in (dict(drafts=d[1:]), dict(drafts=d.int()), dict(offsets=e.int()), dict(offsets=e.cpu()), dict(offsets=e[:0]),
                dict(uniforms=u), dict(uniforms=u2.t().contiguous().t()), dict(draft_logits=x.half()), dict(draft_logits=x[:3]),
                dict(draft_logits=x[:, :8]), dict(draft_logits=x.t()), dict(draft_logits=x.cpu()), dict(temperature=u.double())):
        with pytest.raises(ValueError):
            ce.verify_drafts(**{**dict(logits=x, drafts=d, offsets=e, uniforms=u2), **bad})
    for bad in (dict(score="relu"), dict(bias=u), dict(weights=u2)):
        with pytest.raises(ValueError):
            ce.route_rows(**{**dict(logits=x, k=2), **bad})
    for bad in (dict(k=0), dict(k=17), dict(k=-3), dict(k=1 << 40), dict(groups=3), dict(groups=4, top_groups=5),
                dict(group_top=3), dict(scale=math.inf), dict(groups=4, top_groups=1, k=5), dict(groups=0)):
        with pytest.raises(ce.CeError):
            ce.route_rows(**{**dict(logits=x, k=2), **bad})
    c, g = torch.zeros(6, 2, dtype=torch.int64, device=DEV), torch.zeros(6, 2, device=DEV)
    for bad in (dict(chosen=c[1:]), dict(chosen=c.int()), dict(chosen=d), dict(gates_grad=g[:, :1]), dict(gates_grad=g.half()),
                dict(grad=x.half()), dict(grad=x[:, :8])):
        with pytest.raises(ValueError):
            ce.route_grad(**{**dict(logits=x, chosen=c, gates_grad=g), **bad})
    with pytest.raises(ce.CeError):
        ce.route_grad(x, c[:, :0], g[:, :0])
    with pytest.raises(TypeError):
        ce.sample_rows(x, None)


def test_changed_in_place():
    """A tensor that a call writes to counts as changed for autograd."""
    x = torch.randn(4, 8, device=DEV)
    version = x._version
    c, g = torch.zeros(4, 2, dtype=torch.int64, device=DEV), torch.zeros(4, 2, device=DEV)
    ce.route_grad(x, c, g, grad=x)
    assert x._version == version + 1
    out = torch.zeros(4, dtype=torch.int64, device=DEV)
    ce.sample_rows(torch.randn(4, 8, device=DEV), torch.rand(4, device=DEV), out=out)
    assert out._version == 1


def test_behind_other_work():
    """Each call behind a kernel, a copy, another stream's event and the calls themselves, eager and
    captured: their inputs are made right before them, on the same memory, and their outputs used right after."""
    x = torch.randn(4, 64, 30000, device=DEV)
    u = torch.rand(4, 64, device=DEV)
    want = [ce.sample_rows(x[i] * 2, u[i]) for i in range(4)]
    routed = [ce.route_rows(x[i][:, :64].contiguous(), 4, counts=True) for i in range(4)]
    torch.cuda.synchronize()
    buf, num, cols = torch.empty_like(x[0]), torch.empty_like(u[0]), torch.empty(64, 64, device=DEV)
    side = torch.cuda.Stream()

    def chain():
        out = []
        for i in range(4):
            buf.copy_(x[i])
            buf.mul_(2)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                num.copy_(u[i])
            torch.cuda.current_stream().wait_stream(side)
            tokens = ce.sample_rows(buf, num)
            again = ce.sample_rows(buf, num)
            buf.fill_(0)
            cols.copy_(x[i][:, :64])
            chosen, gates, counts = ce.route_rows(cols, 4, counts=True)
            cols.fill_(math.nan)
            out.append((tokens + 0, again, chosen, gates * 1, counts))
        return out

    def check(out):
        for i in range(4):
            tokens, again, chosen, gates, counts = out[i]
            assert torch.equal(tokens, want[i]) and torch.equal(again, want[i])
            assert all(torch.equal(p, q) for p, q in zip((chosen, gates, counts), routed[i]))
    for _ in range(5):
        check(chain())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    check(out)
