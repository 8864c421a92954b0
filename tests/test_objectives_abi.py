"""Refusals of the objectives' entry points, answered on the host before any
launch, and the 64-bit reference their GPU tests use: its gradients against
autograd and against differences. CPU only."""
import ctypes
import math

import pytest
import torch

import objectives_ref as R
import row_wise_softmax_ce_gb300 as ce
from row_wise_softmax_ce_gb300 import build as cuda_build

V = ctypes.c_void_p
HUGE = (1 << 24) + 1


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return ce.lib()


def logp(lib, logits=V(256), dtype=1, rows=4, vocab=10, stride=10, labels=V(512), weights=None, t=1.0, out=V(1 << 20),
         entropy=None):
    return lib.logp_rows(logits, dtype, rows, vocab, stride, labels, weights, t, out, entropy, None)


def policy(lib, step, logits=V(4096), dtype=0, rows=4, vocab=10, stride=10, labels=V(512), old=V(1024), adv=V(1040),
           ref=V(1056), weights=None, scale=1.0, t=1.0, low=0.2, high=0.2, kl=0.1, bonus=0.0, grad=V(1 << 16), gs=10,
           loss_rows=V(1 << 20), out=V(1 << 21), entropy=None, loss=V(1 << 22), par=True):
    p = ctypes.byref(ce.Policy(scale, t, low, high, kl, bonus)) if par else None
    if step:
        return lib.policy_step(logits, dtype, rows, vocab, stride, labels, old, adv, ref, weights, p, grad, gs,
                               loss_rows, out, entropy, loss, None)
    return lib.policy_loss(logits, dtype, rows, vocab, stride, labels, old, adv, ref, weights, p, loss_rows, out,
                           entropy, loss, None)


def preference(lib, step, logits=V(4096), dtype=0, rows=4, vocab=10, stride=10, labels=V(512), weights=None,
               offsets=V(1024), pairs=1, ref=None, scale=1.0, t=1.0, beta=0.1, eps=0.0, margin=0.0, kind=0, average=0,
               grad=V(1 << 16), gs=10, out=V(1 << 20), seq=V(1 << 21), loss_pairs=V(1 << 22), loss=V(1 << 23),
               work=V(1 << 24), par=True):
    p = ctypes.byref(ce.Preference(scale, t, beta, eps, margin, kind, average)) if par else None
    if step:
        return lib.preference_step(logits, dtype, rows, vocab, stride, labels, weights, offsets, pairs, ref, p, grad,
                                   gs, out, seq, loss_pairs, loss, work, None)
    return lib.preference_loss(logits, dtype, rows, vocab, stride, labels, weights, offsets, pairs, ref, p, out, seq,
                               loss_pairs, loss, work, None)


CALLS = {
    "logp": logp,
    "policy_loss": lambda lib, **k: policy(lib, False, **k),
    "policy_step": lambda lib, **k: policy(lib, True, **k),
    "preference_loss": lambda lib, **k: preference(lib, False, **k),
    "preference_step": lambda lib, **k: preference(lib, True, **k),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad", [dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(vocab=0), dict(stride=9),
                                 dict(vocab=HUGE, stride=HUGE), dict(logits=None), dict(labels=None), dict(out=None),
                                 dict(rows=1 << 40, stride=1 << 40), dict(t=0.0), dict(t=-1.0), dict(t=math.nan),
                                 dict(t=math.inf), dict(t=1e-7), dict(t=1e7)], ids=str)
def test_shared_arguments_refused(lib, name, bad):
    assert CALLS[name](lib, **bad) == ce.CE_EINVAL


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad", [dict(logits=V(4098)), dict(dtype=1, logits=V(4097)), dict(dtype=2, logits=V(4097)),
                                 dict(labels=V(516)), dict(weights=V(1026)), dict(out=V((1 << 20) + 2))], ids=str)
def test_misaligned_pointers_refused(lib, name, bad):
    assert CALLS[name](lib, **{"dtype": 0, **bad}) == ce.CE_EALIGN


def test_entropy_alignment(lib):
    assert logp(lib, entropy=V(1026)) == ce.CE_EALIGN
    assert policy(lib, True, entropy=V(1026)) == ce.CE_EALIGN


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("bad", [dict(low=-0.1), dict(high=-0.1), dict(low=math.nan), dict(high=math.nan),
                                 dict(kl=math.nan), dict(kl=math.inf), dict(bonus=math.inf), dict(scale=math.inf),
                                 dict(old=None), dict(adv=None), dict(ref=None), dict(loss_rows=None), dict(loss=None),
                                 dict(par=False)], ids=str)
def test_policy_arguments_refused(lib, step, bad):
    assert policy(lib, step, **bad) == ce.CE_EINVAL


@pytest.mark.parametrize("bad", [dict(old=V(1026)), dict(adv=V(1026)), dict(ref=V(1026)), dict(loss_rows=V(1026)),
                                 dict(loss=V(1026)), dict(grad=V((1 << 16) + 2))], ids=str)
def test_policy_alignment_refused(lib, bad):
    assert policy(lib, True, **bad) == ce.CE_EALIGN


@pytest.mark.parametrize("name", ["policy_step", "preference_step"])
def test_gradient_overlap_refused(lib, name):
    call = CALLS[name]
    assert call(lib, grad=None) == ce.CE_EINVAL
    assert call(lib, gs=9) == ce.CE_EINVAL
    assert call(lib, grad=V(4096), gs=12) == ce.CE_EINVAL                    # in place needs the same rows
    assert call(lib, grad=V(4096 + 40)) == ce.CE_EINVAL                      # inside the logits
    assert call(lib, grad=V(4096 - 40)) == ce.CE_EINVAL                      # runs into them
    assert call(lib, dtype=1, grad=V(4096 + 78)) == ce.CE_EINVAL             # the last 16-bit logit
    assert call(lib, rows=2, gs=(1 << 62)) == ce.CE_EINVAL


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("bad", [dict(beta=0.0), dict(beta=-1.0), dict(beta=math.nan), dict(beta=math.inf),
                                 dict(margin=math.nan), dict(eps=-0.1), dict(eps=0.6), dict(eps=math.nan),
                                 dict(eps=0.1, kind=1), dict(eps=0.1, kind=2), dict(kind=3), dict(kind=-1),
                                 dict(scale=math.nan), dict(pairs=-1), dict(pairs=1 << 41), dict(offsets=None),
                                 dict(seq=None), dict(loss_pairs=None), dict(loss=None), dict(work=None),
                                 dict(par=False)], ids=str)
def test_preference_arguments_refused(lib, step, bad):
    assert preference(lib, step, **bad) == ce.CE_EINVAL


@pytest.mark.parametrize("bad", [dict(offsets=V(1028)), dict(ref=V(1026)), dict(seq=V(1026)), dict(loss_pairs=V(1026)),
                                 dict(loss=V(1026)), dict(work=V((1 << 24) + 8))], ids=str)
def test_preference_alignment_refused(lib, bad):
    assert preference(lib, True, **bad) == ce.CE_EALIGN


def test_accepted_calls_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    assert logp(lib, rows=0, logits=None, labels=None, out=None) == ce.CE_OK  # nothing to do
    for name, call in CALLS.items():
        assert call(lib) == ce.CE_EDEVICE, name
    assert policy(lib, True, low=math.inf, high=math.inf, kl=0.0, ref=None) == ce.CE_EDEVICE
    assert policy(lib, True, grad=V(4096)) == ce.CE_EDEVICE                   # in place
    assert preference(lib, True, pairs=0, seq=None, loss_pairs=None) == ce.CE_EDEVICE


def test_binding_refuses():
    x, y, f = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    with pytest.raises(ValueError):
        ce.logp_rows(x, y)
    with pytest.raises(TypeError):
        ce.logp_rows(x.double(), y)
    with pytest.raises(ValueError):
        ce.policy_loss(x, y, f, f, 1.0)
    with pytest.raises(ValueError):
        ce.preference_loss(x, y, torch.tensor([0, 2, 4]), 1.0)


# -- the reference itself ---------------------------------------------------------

def batch(rows, vocab, seed):
    g = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn(rows, vocab, generator=g, dtype=torch.float64)
    y = torch.randint(0, vocab, (rows,), generator=g)
    w = torch.rand(rows, generator=g).float() + 0.5
    w[::5] = 0
    return x, y, w, g


def differences(f, x, points, h=1e-6):
    """df/dx at a few (row, column) points, by central differences."""
    out = []
    for i, j in points:
        a, b = x.clone(), x.clone()
        a[i, j] += h
        b[i, j] -= h
        out.append((f(a) - f(b)) / (2 * h))
    return torch.stack(out)


@pytest.mark.parametrize("kl,bonus,T", [(0.0, 0.0, 1.0), (0.3, 0.0, 0.7), (0.1, 0.05, 1.4)])
def test_reference_policy_gradient(kl, bonus, T, monkeypatch):
    monkeypatch.setitem(R.HALF_STEP, torch.float64, 2.0 ** -53)
    monkeypatch.setitem(R.LEAST, torch.float64, 0.0)
    x, y, w, g = batch(12, 17, 3)
    old = R.logp64(x, y, w, T)["logp"][0].float() + 0.4 * torch.randn(12, generator=g)
    adv, ref = torch.randn(12, generator=g), old + 0.3 * torch.randn(12, generator=g)
    kw = dict(ref=ref, weights=w, kl_coef=kl, entropy_coef=bonus, temperature=T)
    grad = R.policy64(x, y, old, adv, 0.25, **kw)["grad"][0]
    pts = [(i, j) for i in range(12) for j in (int(y[i]), (int(y[i]) + 5) % 17)]
    num = differences(lambda v: R.policy64(v, y, old, adv, 0.25, **kw)["loss"][0], x, pts)
    got = torch.stack([grad[i, j] for i, j in pts])
    # central differences at h = 1e-6 of an f64 loss of order 1: 1e-16 / 1e-6 rounding, h^2 truncation
    assert float((got - num).abs().max()) < 1e-8
    # and against autograd of a separate writing of the loss
    xv = x.clone().requires_grad_()
    lp = torch.log_softmax(xv / T, 1)
    logp = lp.gather(1, y[:, None])[:, 0]
    r = (logp - old).exp()
    l = torch.maximum(-adv * r, -adv * r.clamp(0.8, 1.2)) + kl * ((ref - logp).exp() - 1 - (ref - logp))
    l = l + bonus * (lp.exp() * lp).sum(1)
    auto, = torch.autograd.grad(0.25 * (w * l).sum(), xv)
    assert float((grad - auto).abs().max()) < 1e-12


@pytest.mark.parametrize("kind,eps,margin,average", [("sigmoid", 0.0, 0.0, False), ("sigmoid", 0.1, 0.4, True),
                                                     ("hinge", 0.0, 0.1, False), ("squared", 0.0, 0.2, True)])
def test_reference_preference_gradient(kind, eps, margin, average, monkeypatch):
    monkeypatch.setitem(R.HALF_STEP, torch.float64, 2.0 ** -53)
    monkeypatch.setitem(R.LEAST, torch.float64, 0.0)
    x, y, w, g = batch(20, 11, 5)
    offsets = [1, 4, 9, 9, 13, 14, 18]  # three pairs, one empty sequence, rows at both ends outside
    ref = torch.randn(6, generator=g)
    kw = dict(ref=ref, weights=w, kind=kind, beta=0.7, label_smoothing=eps, margin=margin, average=average,
              temperature=1.2)
    grad = R.preference64(x, y, offsets, 0.5, **kw)["grad"][0]
    pts = [(i, j) for i in range(20) for j in (int(y[i]), (int(y[i]) + 3) % 11)]
    num = differences(lambda v: R.preference64(v, y, offsets, 0.5, **kw)["loss"][0], x, pts)
    got = torch.stack([grad[i, j] for i, j in pts])
    assert float((got - num).abs().max()) < 1e-7  # the squared loss is of order 100
    assert float(grad[0].abs().max()) == 0 and float(grad[18:].abs().max()) == 0


def test_assert_near_rejects():
    one = torch.ones(3, dtype=torch.float64)
    R.assert_near(one + 0.9e-6, (one, one * 1e-6), "inside")
    for got in (one + 1.1e-6, one * math.nan, one * math.inf):
        with pytest.raises(AssertionError):
            R.assert_near(got, (one, one * 1e-6), "outside")
    with pytest.raises(AssertionError):
        R.assert_near(one, (one * math.nan, one), "a number for a NaN")
