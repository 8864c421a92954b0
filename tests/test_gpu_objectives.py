"""The objectives over sampled answers and pairs of answers on the GPU, against
their 64-bit definition (tests/objectives_ref.py), every output within the
bound of its own rounding errors."""
import math

import pytest
import torch

import objectives_ref as R
import row_wise_softmax_ce_gb300 as ce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    ce.debug_force(0, 0, 0)
    ce.device_error_reset()
    yield
    assert ce.device_error_count()[1] == 0, "a bounded wait gave up"
    ce.device_error_reset()


def ids(v):
    return str(v).replace("torch.", "") if isinstance(v, torch.dtype) else None


def logits_at(rows, vocab, stride, dtype, seed, sigma=2.0, offset=0, pad=math.nan):
    """[rows, vocab] view of logits `offset` elements into a buffer whose padding and margins hold NaN."""
    g = torch.Generator(DEV).manual_seed(seed)
    buf = torch.full((offset + rows * stride + 64,), pad, dtype=dtype, device=DEV)
    x = buf[offset:offset + rows * stride].view(rows, stride)[:, :vocab]
    x.copy_(sigma * torch.randn(rows, vocab, generator=g, device=DEV))
    return x, g


def inputs(rows, vocab, g, x, masked, T=1.0):
    """Labels, weights, old, ref and advantages; what rows of weight 0 hold must not matter."""
    y = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    w = None
    if masked:
        w = torch.rand(rows, generator=g, device=DEV) + 0.5
        w[torch.rand(rows, generator=g, device=DEV) < masked] = 0.0
    lp = R.logp64(x, y, w, T)["logp"][0].float()
    old = lp + 0.2 * torch.randn(rows, generator=g, device=DEV)
    for edge in (0.8, 1.2, 1.3):  # not within rounding of a clip border
        old = torch.where(((lp - old).exp() - edge).abs() < 1e-3, old + 0.01, old)
    ref = lp + 0.3 * torch.randn(rows, generator=g, device=DEV)
    adv = torch.randn(rows, generator=g, device=DEV)
    if w is not None:
        dead = w == 0
        x[dead] = math.nan
        y[dead] = -100
        for t in (old, ref, adv):
            t[dead] = math.nan
    return y, w, old, ref, adv


def check(got, want, what):
    for name, t in got.items():
        if t is not None:
            R.assert_near(t, want[name], f"{what}: {name}")


# rows, vocab, stride, elements before the first row
SHAPES = [(1, 1, 1, 0), (3, 2, 5, 1), (1, 7, 7, 3), (5, 8, 8, 0), (4, 129, 131, 7), (33, 1000, 1000, 0),
          (2, 4097, 4100, 2), (7, 32000, 32000, 0), (1, 50257, 50257, 5), (160, 5003, 5011, 1), (500, 513, 513, 0),
          (3, 151936, 152064, 0), (2, 200003, 200003, 1)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("entropy,masked,T", [(False, 0.0, 1.0), (True, 0.3, 0.7)])
def test_logp_rows(dtype, shape, entropy, masked, T):
    rows, vocab, stride, offset = shape
    x, g = logits_at(rows, vocab, stride, dtype, seed=rows + vocab, offset=offset)
    y, w, *_ = inputs(rows, vocab, g, x, masked, T)
    got = ce.logp_rows(x, y, weights=w, temperature=T, entropy=entropy)
    got = {"logp": got[0], "entropy": got[1]} if entropy else {"logp": got}
    check(got, R.logp64(x, y, w, T), f"{shape}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kl,bonus,masked,T", [(0.0, 0.0, 0.0, 1.0), (0.1, 0.0, 0.3, 0.8), (0.05, 0.02, 0.2, 1.3)])
def test_policy(dtype, shape, kl, bonus, masked, T):
    rows, vocab, stride, offset = shape
    x, g = logits_at(rows, vocab, stride, dtype, seed=2 * rows + vocab, offset=offset)
    y, w, old, ref, adv = inputs(rows, vocab, g, x, masked, T)
    scale = (1024.0 if dtype == torch.float16 else 1.0) / rows
    kw = dict(weights=w, kl_coef=kl, entropy_coef=bonus, temperature=T, clip_high=0.3)
    want = R.policy64(x, y, old, adv, scale, ref=ref, **kw)
    kw["ref_logp"] = ref if kl else None
    ent = bonus != 0 or T > 1
    names = ("loss", "loss_rows", "logp", "entropy")
    loss = ce.policy_loss(x, y, old, adv, scale, entropy=ent, **kw)
    check(dict(zip(names, loss)), want, f"loss {shape}")
    step = ce.policy_step(x, y, old, adv, scale, entropy=ent, **kw)
    check(dict(zip(("grad",) + names, step)), want, f"step {shape}")
    # a gradient in rows of its own, its padding left alone; and in place
    buf = torch.full((rows, vocab + 9), 7.0, dtype=dtype, device=DEV)
    other = ce.policy_step(x, y, old, adv, scale, entropy=ent, grad=buf[:, 1:], **kw)
    check({"grad": buf[:, 1:vocab + 1]}, want, f"strided {shape}")
    assert other[0].data_ptr() == buf[:, 1:].data_ptr()
    assert bool((buf[:, 0] == 7).all()) and bool((buf[:, vocab + 1:] == 7).all())
    assert torch.equal(buf[:, 1:vocab + 1], step[0])
    there = ce.policy_step(x, y, old, adv, scale, entropy=ent, grad=x, **kw)
    assert torch.equal(there[0], step[0]) and torch.equal(there[1], step[1])


LENGTHS = {
    "one pair": [0, 5, 9],
    "empty": [0, 0, 3, 3, 3, 8, 8],
    "nothing": [2, 2, 2],
    "ragged": [3, 4, 30, 31, 64, 200, 215, 216, 240],
    "no pairs": [4],
}


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
@pytest.mark.parametrize("vocab,stride,offset", [(9, 9, 0), (1000, 1003, 1), (32000, 32000, 0), (50257, 50257, 3)])
@pytest.mark.parametrize("kind,eps,margin,average,masked", [("sigmoid", 0.0, 0.0, False, 0.0),
                                                            ("sigmoid", 0.1, 0.3, True, 0.4),
                                                            ("hinge", 0.0, 0.2, False, 0.2),
                                                            ("squared", 0.0, 0.1, True, 0.0)])
def test_preference(dtype, lengths, vocab, stride, offset, kind, eps, margin, average, masked):
    ends = LENGTHS[lengths]
    rows, pairs = ends[-1] + 6, len(ends) // 2
    x, g = logits_at(rows, vocab, stride, dtype, seed=vocab + rows, offset=offset)
    y, w, *_ = inputs(rows, vocab, g, x, masked)
    outside = torch.ones(rows, dtype=torch.bool, device=DEV)
    outside[ends[0]:ends[-1]] = False
    x[outside] = math.nan
    y[outside] = vocab + 5
    beta = 0.1 if not average else 1.5
    kw = dict(weights=w, kind=kind, beta=beta, label_smoothing=eps, margin=margin, average=average, temperature=0.9)
    seq = R.preference64(x, y, ends, 1.0, **kw)["seq_logp"][0].float()
    ref = seq + (2 if not average else 0.2) * torch.randn(2 * pairs, generator=g, device=DEV)
    scale = 64.0 / max(1, pairs)
    offs = torch.tensor(ends, device=DEV)
    names = ("loss", "loss_pairs", "seq_logp", "logp")
    for r in (None, ref):
        want = R.preference64(x, y, ends, scale, ref=r, **kw)
        loss = ce.preference_loss(x, y, offs, scale, ref_logp=r, **kw)
        check(dict(zip(names, loss)), want, f"loss {lengths}")
        step = ce.preference_step(x, y, offs, scale, ref_logp=r, **kw)
        check(dict(zip(("grad",) + names, step)), want, f"step {lengths}")
    buf = torch.full((rows, vocab + 11), 7.0, dtype=dtype, device=DEV)
    ce.preference_step(x, y, offs, scale, ref_logp=ref, grad=buf[:, 2:], **kw)
    assert torch.equal(buf[:, 2:vocab + 2], step[0])
    assert bool((buf[:, :2] == 7).all()) and bool((buf[:, vocab + 2:] == 7).all())
    there = ce.preference_step(x, y, offs, scale, ref_logp=ref, grad=x, **kw)
    assert torch.equal(there[0], step[0])


# -- values that masks and mistakes leave in logits ----------------------------------

@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("vocab", [40, 4100, 33001])
@pytest.mark.parametrize("fill", ["-inf", "lowest"])
def test_masked_columns(dtype, vocab, fill):
    """Columns masked by -inf or the type's lowest value: all but one, all of a
    thread's, a label's own, all of a row's."""
    rows = 12
    x, g = logits_at(rows, vocab, vocab + 3, dtype, seed=vocab)
    low = -math.inf if fill == "-inf" else torch.finfo(dtype).min
    y = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    x[0, 1:] = low
    y[0] = 0
    x[1, : vocab - 1] = low
    y[1] = vocab - 1
    x[2, vocab // 3:] = low
    x[3, torch.rand(vocab, generator=g, device=DEV) < 0.9] = low
    x[4, y[4]] = low
    x[5, :] = low                      # -inf: no distribution; the lowest value: the uniform one
    x[6, :] = low
    x[6, vocab // 2] = 1.0
    x[7, ::2] = -math.inf
    x[7, 1::2] = torch.finfo(dtype).min
    x[8, :] = 0.0
    x[9, :] = 60000.0
    x[10, :] = -60000.0
    x[10, 3] = -59990.0
    y[3] = int(x[3].float().argmax())
    old = torch.full((rows,), -1.0, device=DEV)
    adv = torch.ones(rows, device=DEV)
    want = R.policy64(x, y, old, adv, 0.5, entropy_coef=0.01)
    logp, ent = ce.logp_rows(x, y, entropy=True)
    check({"logp": logp, "entropy": ent}, R.logp64(x, y), "logp")
    R.assert_near(ce.logp_rows(x, y), want["logp"], "logp alone")
    step = ce.policy_step(x, y, old, adv, 0.5, entropy_coef=0.01, entropy=True)
    check(dict(zip(("grad", "loss", "loss_rows", "logp", "entropy"), step)), want, "step")
    plain = ce.policy_step(x, y, old, adv, 0.5)
    check({"grad": plain[0], "loss_rows": plain[2]}, R.policy64(x, y, old, adv, 0.5), "step without entropy")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("vocab", [5, 1000, 50257])
def test_rows_that_are_no_distribution(dtype, vocab):
    """NaN, +inf, labels out of range: NaN there, counted, and nothing else touched."""
    rows = 9
    x, g = logits_at(rows, vocab, vocab, dtype, seed=vocab + 1)
    y = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    x[1, vocab - 1] = math.nan
    x[2, 0] = math.inf
    x[3, :] = math.nan
    x[4, :] = math.inf
    y[5], y[6] = vocab, -1
    old, adv = torch.full((rows,), -2.0, device=DEV), torch.ones(rows, device=DEV)
    ce.device_error_reset()
    step = ce.policy_step(x, y, old, adv, 1.0, entropy_coef=0.1, entropy=True)
    assert ce.device_error_count()[0] == 2
    want = R.policy64(x, y, old, adv, 1.0, entropy_coef=0.1)
    check(dict(zip(("grad", "loss", "loss_rows", "logp", "entropy"), step)), want, "policy")
    for i in (1, 2, 3, 4, 5, 6):
        assert bool(torch.isnan(step[0][i]).all()) and math.isnan(step[3][i])
    logp, ent = ce.logp_rows(x, y, entropy=True)
    check({"logp": logp, "entropy": ent}, R.logp64(x, y), "logp")
    # a bad row spoils its own pair, and no other
    ends = [0, 1, 2, 8, 9]  # chosen: row 0; row 1 ... rejected: rows 2-7; row 8
    out = ce.preference_step(x, y, torch.tensor(ends, device=DEV), 1.0)
    want = R.preference64(x, y, ends, 1.0)
    check(dict(zip(("grad", "loss", "loss_pairs", "seq_logp", "logp"), out)), want, "preference")
    ce.device_error_reset()


def test_bad_offsets_read_nothing_out_of_range():
    rows, vocab = 20, 64
    x, g = logits_at(rows, vocab, vocab, torch.float32, seed=4)
    y = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    good = ce.preference_step(x, y, torch.tensor([0, 4, 8, 12, 16], device=DEV), 1.0)
    for ends, pair in (([0, 4, 8, 12, 1 << 40], 1), ([0, 4, 8, 12, 21], 1), ([-1, 4, 8, 12, 16], 0),
                       ([-(1 << 62), 4, 8, 12, 16], 0), ([0, 4, 8, 12, 11], 1)):
        ce.device_error_reset()
        grad, loss, pairs, seq, logp = ce.preference_step(x, y, torch.tensor(ends, device=DEV), 1.0)
        assert ce.device_error_count()[0] == 1, ends
        assert math.isnan(loss) and math.isnan(pairs[pair]), ends
        if ends[-1] == 11:
            continue  # a table that decreases: the other pair may have lost rows
        assert torch.equal(pairs[1 - pair], good[2][1 - pair]), ends
        # the other pair's rows have their gradient
        own = slice(4, 8) if pair == 0 else slice(0, 4)
        assert torch.equal(grad[own], good[0][own]), ends
    ce.device_error_reset()


# -- the formulas' corners ------------------------------------------------------------

def test_policy_on_policy_and_at_the_border():
    """old = logp_rows' log-probabilities: the ratio is 1 to within the bounds of
    two log-probabilities t (one per call: the calls add up in their own orders),
    so the loss is -A to within |A| (2 t + 4 U), U = 2^-24 for each of expf's
    result (2), the product and its clamp. old = the same call's: the ratio is
    exactly 1, and with no room to either side the two terms are equal, which
    counts as unclipped."""
    rows, vocab = 64, 3000
    x, g = logits_at(rows, vocab, vocab, torch.bfloat16, seed=1)
    y = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    adv = torch.randn(rows, generator=g, device=DEV)
    old = ce.logp_rows(x, y)
    bound = adv.double().abs() * (2 * R.logp64(x, y)["logp"][1] + 4 * R.U)
    free = ce.policy_step(x, y, old, adv, 1.0 / rows, clip_low=math.inf, clip_high=math.inf)
    tight = ce.policy_step(x, y, old, adv, 1.0 / rows, clip_low=0.0, clip_high=0.0)
    R.assert_near(free[2], (-adv.double(), bound), "free")
    R.assert_near(tight[2], (-adv.double(), bound), "tight")
    old = free[3]
    free = ce.policy_step(x, y, old, adv, 1.0 / rows, clip_low=math.inf, clip_high=math.inf)
    tight = ce.policy_step(x, y, old, adv, 1.0 / rows, clip_low=0.0, clip_high=0.0)
    assert torch.equal(free[2], -adv) and torch.equal(tight[2], -adv)
    assert torch.equal(free[0], tight[0])
    check({"grad": free[0]}, R.policy64(x, y, R.logp64(x, y)["logp"][0], adv, 1.0 / rows), "grad")


def test_policy_clip_sides():
    x = torch.zeros(4, 8, device=DEV)
    y = torch.zeros(4, dtype=torch.int64, device=DEV)
    lp = -math.log(8)
    old = torch.tensor([lp - 1, lp - 1, lp + 1, lp + 1], device=DEV)  # ratios e, e, 1/e, 1/e
    adv = torch.tensor([1.0, -1.0, 1.0, -1.0], device=DEV)
    grad, loss, rows, _, _ = ce.policy_step(x, y, old, adv, 1.0, clip_low=0.1, clip_high=0.3)
    e = math.e
    want = torch.tensor([-1.3, e, -1 / e, 0.9], device=DEV)
    assert torch.allclose(rows, want, rtol=1e-5, atol=0)
    assert bool((grad[0] == 0).all()) and bool((grad[3] == 0).all())  # clipped: no gradient
    assert torch.allclose(grad[1, 0], torch.tensor(e * 7 / 8, device=DEV), rtol=1e-5)
    assert torch.allclose(grad[2, 0], torch.tensor(-1 / e * 7 / 8, device=DEV), rtol=1e-5)


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "squared"])
@pytest.mark.parametrize("z", [-200.0, -30.0, 0.0, 30.0, 200.0])
def test_preference_far_margins(kind, z):
    """Saturated pairs: finite losses, gradients that vanish and do not overflow."""
    rows, vocab = 8, 100
    x, g = logits_at(rows, vocab, vocab, torch.float32, seed=7)
    y = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    kw = dict(kind=kind, beta=1.0, margin=-z, label_smoothing=0.2 if kind == "sigmoid" else 0.0)
    want = R.preference64(x, y, [0, 4, 8], 1.0, **kw)
    got = ce.preference_step(x, y, torch.tensor([0, 4, 8], device=DEV), 1.0, **kw)
    check(dict(zip(("grad", "loss", "loss_pairs", "seq_logp", "logp"), got)), want, f"{kind} {z}")


def test_zero_rows_and_nothing_left():
    for dtype in TYPES:
        x = torch.empty(0, 50, dtype=dtype, device=DEV)
        y, f = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
        assert ce.logp_rows(x, y).shape == (0,)
        assert float(ce.policy_loss(x, y, f, f, 1.0)[0]) == 0.0
        assert float(ce.policy_step(x, y, f, f, 1.0)[1]) == 0.0
        assert float(ce.preference_step(x, y, torch.tensor([0], device=DEV), 1.0)[1]) == 0.0
        # two empty sequences: h = 0
        assert abs(float(ce.preference_step(x, y, torch.tensor([0, 0, 0], device=DEV), 1.0)[1]) - math.log(2)) < 1e-6
        # a batch whose mask leaves nothing
        x = torch.full((5, 50), math.nan, dtype=dtype, device=DEV)
        y, f = torch.full((5,), -100, device=DEV), torch.full((5,), math.nan, device=DEV)
        w = torch.zeros(5, device=DEV)
        grad, loss, rows, logp, ent = ce.policy_step(x, y, f, f, 1.0, weights=w, entropy=True)
        assert float(loss) == 0 and not grad.any() and not rows.any() and not logp.any() and not ent.any()
        grad, loss, pairs, seq, logp = ce.preference_step(x, y, torch.tensor([0, 2, 5], device=DEV), 1.0, weights=w,
                                                          average=True)
        assert not grad.any() and not seq.any() and not logp.any()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_broadcast_rows(dtype):
    """Rows 0 elements apart are refused (they overlap); one row may have any stride."""
    x = torch.randn(1, 77, device=DEV).to(dtype)
    y = torch.zeros(3, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        ce.logp_rows(x.expand(3, 77), y)
    with pytest.raises(ValueError):
        ce.policy_step(x.expand(3, 77).contiguous(), y, torch.zeros(3, device=DEV), torch.zeros(3, device=DEV), 1.0,
                       grad=torch.empty(1, 77, dtype=dtype, device=DEV).expand(3, 77))
    R.assert_near(ce.logp_rows(x.expand(1, 77), y[:1]), R.logp64(x, y[:1])["logp"], "one row")


# -- differences, and the calls as they are used together -----------------------------

def test_gradient_by_differences():
    """The kernel's gradient against central differences of the kernel's own
    loss along random directions: step h = 2^-5, truncation h^2 / 6 of a third
    derivative below 10 (1.6e-3), rounding of an f32 loss of order 1 2^-24 / h
    (2e-6)."""
    rows, vocab, h = 48, 300, 2.0 ** -5
    x, g = logits_at(rows, vocab, vocab, torch.float32, seed=11)
    y, w, old, ref, adv = inputs(rows, vocab, g, x, 0.0)
    old = R.logp64(x, y)["logp"][0].float() + 0.02 * torch.randn(rows, generator=g, device=DEV)  # far from the clips
    ends = torch.tensor([0, 10, 24, 30, 48], device=DEV)

    def policy(v):
        return ce.policy_loss(v, y, old, adv, 1.0, ref_logp=ref, kl_coef=0.1, entropy_coef=0.05)[0]

    def preference(v):
        return ce.preference_loss(v, y, ends, 1.0, beta=0.3)[0]

    gp = ce.policy_step(x, y, old, adv, 1.0, ref_logp=ref, kl_coef=0.1, entropy_coef=0.05)[0]
    gq = ce.preference_step(x, y, ends, 1.0, beta=0.3)[0]
    for f, grad in ((policy, gp), (preference, gq)):
        for _ in range(4):
            v = torch.randn(rows, vocab, generator=g, device=DEV)
            v /= v.norm()
            num = float((f(x + h * v).double() - f(x - h * v).double()) / (2 * h))
            assert abs(num - float((grad.double() * v.double()).sum())) < 2e-3


def test_a_round_of_training():
    """Rollout scoring, a policy step, then a preference step, on the logits of
    one head: log-probabilities from one call are the next one's inputs, and the
    head's weight gradient is the formula's."""
    g = torch.Generator(DEV).manual_seed(3)
    T, D, vocab = 96, 32, 2000
    hid = torch.randn(T, D, generator=g, device=DEV)
    W = (0.3 * torch.randn(vocab, D, generator=g, device=DEV))
    x = hid @ W.t()
    y = ce.argmax_rows(x + 2 * torch.randn(T, vocab, generator=g, device=DEV)).long()  # sampled tokens
    old, ent = ce.logp_rows(x, y, entropy=True)
    frozen = hid @ (W + 0.02 * torch.randn(W.shape, generator=g, device=DEV)).t()
    ref = ce.logp_rows(frozen, y)
    adv = torch.randn(T, generator=g, device=DEV)
    # one step away from the sampling policy
    grad, loss, rows, logp, _ = ce.policy_step(x, y, old, adv, 1.0 / T, ref_logp=ref, kl_coef=0.05)
    exact, bound = R.logp64(x, y)["logp"]
    R.assert_near(logp, (exact, bound), "logp of the step")
    R.assert_near(logp, (old.double(), 2 * bound), "the step's against the rollout's")
    W2 = W - 0.5 * (grad.t() @ hid)
    x2 = hid @ W2.t()
    want = R.policy64(x2, y, old, adv, 1.0 / T, ref=ref, kl_coef=0.05)
    got = ce.policy_step(x2, y, old, adv, 1.0 / T, ref_logp=ref, kl_coef=0.05)
    check(dict(zip(("grad", "loss", "loss_rows", "logp"), got)), want, "second step")
    # the answers as pairs: the reference's sequence log-probabilities are a call on its logits
    ends = torch.tensor([0, 20, 50, 70, 96], device=DEV)
    seq_ref = ce.preference_loss(frozen, y, ends, 1.0)[2]
    want = R.preference64(x2, y, ends.tolist(), 0.5, ref=seq_ref)
    got = ce.preference_step(x2, y, ends, 0.5, ref_logp=seq_ref)
    check(dict(zip(("grad", "loss", "loss_pairs", "seq_logp", "logp"), got)), want, "preference")
    # -ce_rows is the same log-probability in f32 at T = 1
    R.assert_near(-ce.ce_rows(x2, y), R.logp64(x2, y)["logp"], "ce_rows")


# -- streams, graphs, sizes -------------------------------------------------------------

def everything(x, y, w, old, ref, adv, ends):
    rows = x.shape[0]
    out = list(ce.logp_rows(x, y, weights=w, entropy=True))
    out += [t for t in ce.policy_loss(x, y, old, adv, 1.0 / rows, ref_logp=ref, kl_coef=0.1, weights=w) if t is not None]
    out += list(ce.policy_step(x, y, old, adv, 1.0 / rows, ref_logp=ref, kl_coef=0.1, weights=w, entropy_coef=0.01,
                               entropy=True))
    out += list(ce.preference_loss(x, y, ends, 1.0, weights=w))
    out += list(ce.preference_step(x, y, ends, 1.0, weights=w))
    return out


def a_batch(dtype, seed, rows=70, vocab=9001):
    x, g = logits_at(rows, vocab, vocab + 7, dtype, seed)
    y, w, old, ref, adv = inputs(rows, vocab, g, x, 0.2)
    return x, y, w, old, ref, adv, torch.tensor([1, 20, 40, 45, 66], device=DEV)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_streams_and_repeats(dtype):
    """The same bits on every call, on four streams at once."""
    batches = [a_batch(dtype, s) for s in range(4)]
    want = [everything(*b) for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    got = [[] for _ in batches]
    for _ in range(3):
        for k, (s, b) in enumerate(zip(streams, batches)):
            with torch.cuda.stream(s):
                got[k].append(everything(*b))
    torch.cuda.synchronize()
    same = lambda a, b: torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))  # noqa: E731
    for k, w in enumerate(want):
        for r in got[k]:
            assert all(same(a, b) for a, b in zip(w, r))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_graph_replay(dtype):
    """Two graphs captured from the same calls and replayed side by side on new
    inputs give what eager calls on them give."""
    first, second = a_batch(dtype, 5), a_batch(dtype, 6)
    eager = everything(*second)
    held = [t.clone() for t in first]
    held[0] = torch.empty_strided(first[0].shape, first[0].stride(), dtype=dtype, device=DEV)
    held[0].copy_(first[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        everything(*held)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(everything(*held))
        graphs.append(g)
    for h, t in zip(held, second):
        h.copy_(t)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        for s, g in ((s1, graphs[0]), (s2, graphs[1])):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, eager):
            assert torch.equal(torch.nan_to_num(a.float()), torch.nan_to_num(b.float()))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=ids)
def test_past_2_31_elements(dtype):
    """Logits of more than 2^31 elements, in place: the rows around the
    2^31st element and the last ones."""
    vocab = 131073
    rows = (1 << 31) // vocab + 40
    g = torch.Generator(DEV).manual_seed(9)
    x = torch.empty(rows, vocab, dtype=dtype, device=DEV)
    for a in range(0, rows, 1024):
        b = min(rows, a + 1024)
        x[a:b] = 2 * torch.randn(b - a, vocab, generator=g, device=DEV)
    y = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    some = torch.tensor([0, rows // 2, (1 << 31) // vocab - 1, (1 << 31) // vocab, (1 << 31) // vocab + 1, rows - 1],
                        device=DEV)
    xs, ys = x[some].clone(), y[some]
    old, adv = torch.full((rows,), -14.0, device=DEV), torch.ones(rows, device=DEV)
    logp = ce.logp_rows(x, y)
    want = R.policy64(xs, ys, old[some], adv[some], 1.0)
    R.assert_near(logp[some], want["logp"], "logp")
    # every sequence one row long but the last: pairs of neighbours, one factor each
    pairs = rows // 2
    offs = torch.arange(2 * pairs + 1, device=DEV)
    _, _, seq, lp = ce.preference_loss(x, y, offs, 1.0)
    assert torch.equal(lp[:2 * pairs], logp[:2 * pairs]) and torch.equal(seq, logp[:2 * pairs])
    out = ce.policy_step(x, y, old, adv, 1.0, grad=x)
    R.assert_near(out[0][some], want["grad"], "grad")
    R.assert_near(out[3][some], want["logp"], "logp of the step")


def test_rows_longer_than_shared_memory():
    """Rows of up to 2^24 columns."""
    for vocab, rows, dtype in ((1 << 24, 2, torch.float32), ((1 << 21) + 3, 3, torch.bfloat16)):
        x, g = logits_at(rows, vocab, vocab, dtype, seed=2)
        y, w, old, ref, adv = inputs(rows, vocab, g, x, 0.0)
        want = R.policy64(x, y, old, adv, 64.0, entropy_coef=0.01)
        got = ce.policy_step(x, y, old, adv, 64.0, entropy_coef=0.01, entropy=True)
        check(dict(zip(("grad", "loss", "loss_rows", "logp", "entropy"), got)), want, f"{vocab}")
        there = ce.policy_step(x, y, old, adv, 64.0, entropy_coef=0.01, entropy=True, grad=x)
        assert torch.equal(there[0], got[0])


def test_other_device_refused():
    x = torch.zeros(2, 4, device=DEV)
    y = torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        ce.logp_rows(x, y.cpu())
    with pytest.raises(ValueError):
        ce.logp_rows(x, y, weights=torch.ones(2))
    with pytest.raises(ValueError):
        ce.policy_loss(x, y, torch.ones(2), torch.ones(2, device=DEV), 1.0)
    with pytest.raises(ValueError):
        ce.preference_loss(x, y, torch.tensor([0, 1, 2]), 1.0)
