"""The objectives where their constants are far from 1 and their tensors are
used again: temperatures and scales over the accepted range, beside masked
columns. Against the 64-bit definition (tests/objectives_ref.py)."""
import math

import pytest
import torch

import objectives_ref as R
import row_wise_softmax_ce_gb300 as ce
from test_gpu_objectives import DEV, TYPES, check, ids, logits_at

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    ce.device_error_reset()
    yield
    assert ce.device_error_count() == (0, 0)


def wider(want, scale, T, adv, bonus):
    """The gradient's bound with what a flushed probability is worth: p below
    2^-126 counts as 0, which leaves out at most scale / T p (|g| + |bonus|
    |log p + H|) of a column, |g| <= 2 |A| here (the ratio is 1) and |log p + H|
    <= 88 + log 2^24 < 110 at the largest such p (p |log p| falls below it)."""
    value, bound = want["grad"]
    lost = 2.0 ** -126 * abs(scale) / T * (2 * adv.double().abs() + abs(bonus) * 110)
    return dict(want, grad=(value, bound + lost[:, None]))


# a warp per row, rows staged in shared memory, rows read twice
VOCABS = {torch.float32: (1000, 33001, (1 << 20) + 3), torch.bfloat16: (1000, 33001, (1 << 21) + 3),
          torch.float16: (1000, 33001, (1 << 21) + 3)}


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("kernel", range(3), ids=["warp", "staged", "stream"])
@pytest.mark.parametrize("T", [1e-6, 1e-3, 1e3, 1e6])
def test_masked_columns_at_far_temperatures(dtype, kernel, T):
    """Columns of -inf have a gradient of 0 whatever the temperature, the scale
    and the entropy bonus; columns of the lowest value have the formula's."""
    rows, vocab = 4, VOCABS[dtype][kernel]
    x, g = logits_at(rows, vocab, vocab + 1, dtype, seed=vocab)
    ban = torch.rand(vocab, generator=g, device=DEV) < 0.5
    ban[vocab // 2] = False
    x[0, ban] = -math.inf
    x[1, ban] = torch.finfo(dtype).min
    x[2, : vocab // 2] = -math.inf
    x[2, vocab // 2 + 1:] = torch.finfo(dtype).min
    y = x.float().argmax(1)
    adv = torch.tensor([1.0, -0.5, 2.0, 0.25], device=DEV)
    old = R.logp64(x, y, temperature=T)["logp"][0].float()
    # f16 gradients end at 65504: scales whose factor scale / T stays below
    scales = (T, 3e4 * T) if dtype == torch.float16 else (T, 1.0, 65536.0)
    for scale in scales:
        for bonus in (0.0, 0.01, 1.0):
            what = f"{vocab} T={T} scale={scale} bonus={bonus}"
            want = wider(R.policy64(x, y, old, adv, scale, entropy_coef=bonus, temperature=T), scale, T, adv, bonus)
            for entropy in (False, True):
                got = ce.policy_step(x, y, old, adv, scale, entropy_coef=bonus, temperature=T, entropy=entropy)
                check(dict(zip(("grad", "loss", "loss_rows", "logp", "entropy"), got)), want, what)
                assert not got[0][x == -math.inf].any(), what


def bonus64(x, f, bonus, T):
    """f bonus p_j (log p_j + H) in 64 bits, and its bound. With D = (m - x_j) /
    T, log p_j + H = -D - mean, mean = sum of p (x - m) / T:
      p     its relative error, as in objectives_ref.grad64: err_s + (3 D + 8) U
      D     3 U of the exponent, 5 U of the factor and the product
      mean  sum of e D over s: terms of one sign, so err_s for the sum, err_s for
            s, 8 U for the terms, the quotient and the factor
    -- no error of the size of the entropy's own rounding (U log V)."""
    z = x.double() / T
    D = z.amax(1, keepdim=True) - z
    e = (-D).exp()
    p = e / e.sum(1, keepdim=True)
    mean = -(p * D).sum(1, keepdim=True)
    value = abs(f) * bonus * p * (-D - mean)
    err_s = (6 + R.depth(x.shape[1])) * R.U
    rel_p = err_s + (3 * D + 8) * R.U
    bound = abs(f) * bonus * p * (D * (rel_p + 8 * R.U) + mean.abs() * (rel_p + 2 * err_s + 8 * R.U))
    return value, bound + value.abs() * (R.HALF_STEP[x.dtype] + 4 * R.U) + R.LEAST[x.dtype]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("kernel", range(3), ids=["warp", "staged", "stream"])
@pytest.mark.parametrize("T", [1.0, 1e3, 1e5, 1e6])
def test_entropy_gradient_of_flat_rows(dtype, kernel, T):
    """The entropy bonus alone (no advantage): its gradient is as accurate on a
    row that the temperature makes nearly flat as anywhere."""
    rows, vocab = 4, VOCABS[dtype][kernel]
    x, g = logits_at(rows, vocab, vocab, dtype, seed=vocab + 1)
    y = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    old = R.logp64(x, y, temperature=T)["logp"][0].float()
    scale = T * T * vocab  # columns of order x - m, in range of f16
    grad = ce.policy_step(x, y, old, torch.zeros(rows, device=DEV), scale, entropy_coef=1.0, temperature=T)[0]
    R.assert_near(grad, bonus64(x, scale / T, 1.0, T), f"{vocab} T={T}")


@pytest.mark.parametrize("rows", [1, 300, 8192, 8193, 40000])
def test_sum_of_the_pass_before_it(rows):
    """The C call over and over into the same buffers, the losses changing sign
    and size from pass to pass, nothing between the passes: each loss is the sum
    of its own pass's row losses, over one CTA's rows and a cluster's."""
    import ctypes
    vocab, passes = 40, 60
    L, par = ce.lib(), ce.Policy(1.0, 1.0, 0.2, 0.2, 0.0, 0.0)
    x, g = logits_at(rows, vocab, vocab, torch.float32, seed=rows)
    y = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    old = ce.logp_rows(x, y)
    advs = [(-1.0) ** i * (1 + i) * (torch.rand(rows, generator=g, device=DEV) + 0.5) for i in range(passes)]
    loss_rows, logp = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    kept = [torch.empty(rows, device=DEV) for _ in range(passes)]
    losses = torch.full((passes,), math.nan, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    for i, adv in enumerate(advs):
        st = L.policy_loss(x.data_ptr(), 0, rows, vocab, vocab, y.data_ptr(), old.data_ptr(), adv.data_ptr(), None, None,
                           ctypes.byref(par), loss_rows.data_ptr(), logp.data_ptr(), None, losses[i:].data_ptr(), s)
        assert st == ce.CE_OK
        if i % 3 == 2:  # mostly nothing between two passes
            kept[i].copy_(loss_rows)
    for i in range(2, passes, 3):
        # the sum is of at least 48 bits relative to its largest partial sum, then one rounding
        want, size = kept[i].double().sum(), kept[i].double().abs().sum()
        assert abs(float(losses[i]) - float(want)) <= R.U * abs(float(want)) + 2.0 ** -47 * float(size) * rows, i
    for i in range(passes):
        want = -(advs[i].double()).sum()  # ratios of 1 within 1e-5
        assert abs(float(losses[i]) - float(want)) <= 1e-4 * float(advs[i].double().abs().sum()), i


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("kernel", range(3), ids=["warp", "staged", "stream"])
def test_in_place_of_rows_that_share_lines(dtype, kernel):
    """Odd rows without padding, so that neighbouring rows and slices share
    their 128-byte lines, written in place: the bits of a gradient of its own."""
    rows, vocab = (2000, 1000, 9)[kernel], VOCABS[dtype][kernel]
    vocab += vocab % 2 == 0
    rows = min(rows, (1 << 26) // vocab)
    x, g = logits_at(rows, vocab, vocab, dtype, seed=vocab + 2, offset=3)
    y = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
    old, adv = torch.full((rows,), -12.0, device=DEV), torch.randn(rows, generator=g, device=DEV)
    own = ce.policy_step(x, y, old, adv, 1.0, entropy_coef=0.01)
    for _ in range(2):
        z = torch.empty(x.numel() + 3, dtype=dtype, device=DEV)[3:].view(rows, vocab)  # at the phase of x
        z.copy_(x)
        there = ce.policy_step(z, y, old, adv, 1.0, entropy_coef=0.01, grad=z)
        assert all(torch.equal(a, b) for a, b in zip(there[:4], own[:4]))


def test_given_outputs_over_other_tensors_are_refused():
    x, y = torch.randn(6, 50, device=DEV), torch.zeros(6, dtype=torch.int64, device=DEV)
    f, w, two = torch.zeros(6, device=DEV), torch.ones(7, device=DEV), torch.empty(6, device=DEV)
    for kw in (dict(out=two, entropy=two), dict(out=w[1:], weights=w[:6]), dict(entropy=w[:6], weights=w[:6]),
               dict(out=x[2, 10:16])):
        with pytest.raises(ce.CeError):
            ce.logp_rows(x, y, **kw)
    for call in (ce.policy_loss, ce.policy_step):
        for kw in (dict(entropy=f), dict(entropy=w[1:], weights=w[:6]), dict(entropy=x[0, :6])):
            with pytest.raises(ce.CeError):
                call(x, y, f, f, 1.0, **kw)
    assert bool((w == 1).all()) and not f.any()
    wide = torch.randn(6, 60, device=DEV)
    got = ce.logp_rows(wide, y, vocab=50, out=wide[3, 52:58])  # the padding of a row is not the logits'
    assert torch.equal(got, ce.logp_rows(wide[:, :50], y))


def test_writing_to_a_tensor_counts_as_in_place():
    """A caller's tensor that a call writes to has a new version, so that a
    backward pass that saved it refuses; what is only read has not, nor what a
    refused call would have written."""
    head = torch.randn(50, 8, device=DEV, requires_grad=True)
    y, f = torch.zeros(6, dtype=torch.int64, device=DEV), torch.zeros(6, device=DEV)
    ends = torch.tensor([0, 3, 6], device=DEV)
    for call in (lambda z, g: ce.policy_step(z, y, f, f + 1, 1.0, grad=g),
                 lambda z, g: ce.preference_step(z, y, ends, 1.0, grad=g)):
        x = torch.randn(6, 8, device=DEV) @ head.t()
        loss = (x * x).sum()  # saves x
        call(x.detach(), None)
        loss.backward(retain_graph=True)
        call(x.detach(), x.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    x, out, ent = torch.randn(6, 50, device=DEV), torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    ce.logp_rows(x, y, out=out, entropy=ent)
    assert (x._version, y._version, out._version, ent._version) == (0, 0, 1, 1)
    ce.policy_loss(x, y, f, f, 1.0, entropy=ent)
    grad = torch.empty(6, 50, device=DEV)
    ce.policy_step(x, y, f, f, 1.0, entropy=ent, grad=grad)
    assert (x._version, f._version, ent._version, grad._version) == (0, 0, 3, 1)
    with pytest.raises(ce.CeError):
        ce.policy_step(x, y, f, f, 1.0, temperature=0.0, grad=grad)
    assert grad._version == 1
    with torch.inference_mode():
        z, out = torch.randn(6, 50, device=DEV), torch.empty(6, device=DEV)
        want = ce.policy_step(z, y, f, f + 1, 1.0)[0]
        ce.logp_rows(z, y, out=out)
        assert torch.equal(ce.policy_step(z, y, f, f + 1, 1.0, grad=z)[0], want)
    ce.logp_rows(z, y, out=out)  # inference tensors outside the mode: no version to count


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("vocab", [905000, 920000, 920800, 921600])
def test_rows_that_fill_a_cluster(dtype, vocab):
    """Rows around the longest that the shared memory of 16 CTAs holds (about
    3.5 MB), at a phase of their own: staged below it, read twice above."""
    vocab *= 1 if dtype == torch.float32 else 2
    x, g = logits_at(3, vocab, vocab + 1, dtype, seed=7, offset=1)
    y = torch.randint(0, vocab, (3,), generator=g, device=DEV)
    adv = torch.randn(3, generator=g, device=DEV)
    old = R.logp64(x, y)["logp"][0].float() + 0.05
    want = R.policy64(x, y, old, adv, 64.0, entropy_coef=0.01)
    got = ce.policy_step(x, y, old, adv, 64.0, entropy_coef=0.01, entropy=True)
    check(dict(zip(("grad", "loss", "loss_rows", "logp", "entropy"), got)), want, f"{vocab}")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("vocab", [1000, 33001])
@pytest.mark.parametrize("T", [1e-6, 1e-3, 1e3, 1e6])
def test_far_temperatures(dtype, vocab, T):
    """Log-probabilities, entropies, the policy loss with its KL term and the
    preference step over the accepted temperatures, beside masked columns. Labels
    on the row's largest logit (elsewhere (x - m) / T leaves f32's bounds of first
    order) and, from T = 1e3, anywhere."""
    rows = 40
    x, g = logits_at(rows, vocab, vocab + 3, dtype, seed=vocab + 5)
    x[::3, torch.rand(vocab, generator=g, device=DEV) < 0.5] = -math.inf
    x[1::3, torch.rand(vocab, generator=g, device=DEV) < 0.5] = torch.finfo(dtype).min
    y = x.float().argmax(1)
    if T > 1:
        other = torch.randint(0, vocab, (rows,), generator=g, device=DEV)
        kept = x.gather(1, other[:, None])[:, 0] > torch.finfo(dtype).min / 2
        y = torch.where(kept, other, y)
    w = torch.rand(rows, generator=g, device=DEV) + 0.5
    w[::7] = 0.0
    want = R.logp64(x, y, w, T)
    logp, ent = ce.logp_rows(x, y, weights=w, temperature=T, entropy=True)
    check({"logp": logp, "entropy": ent}, want, "logp_rows")
    assert torch.equal(ce.logp_rows(x, y, weights=w, temperature=T), logp)
    old = want["logp"][0].float()
    adv, ref = torch.randn(rows, generator=g, device=DEV), old + 0.1
    want = R.policy64(x, y, old, adv, T, ref=ref, weights=w, kl_coef=0.1, temperature=T)
    step = ce.policy_step(x, y, old, adv, T, ref_logp=ref, weights=w, kl_coef=0.1, temperature=T)
    check(dict(zip(("grad", "loss", "loss_rows", "logp"), step)), wider(want, T, T, adv.abs() + 1, 0.0), "policy")
    ends = [0, 9, 20, 31, 40]
    want = R.preference64(x, y, ends, T, weights=w, temperature=T, beta=0.2)
    got = ce.preference_step(x, y, torch.tensor(ends, device=DEV), T, weights=w, temperature=T, beta=0.2)
    check(dict(zip(("grad", "loss", "loss_pairs", "seq_logp", "logp"), got)),
          wider(want, T, T, torch.ones(rows, device=DEV), 0.0), "preference")
