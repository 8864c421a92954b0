"""The objectives' binding: what it refuses and with which error, that it keeps
no reference and no memory, and that it shares the library's state."""
import gc
import sys

import pytest
import torch

import row_wise_softmax_ce_gb300 as ce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


def batch(rows=6, vocab=50, dtype=torch.float32):
    x = torch.randn(rows, vocab, device=DEV).to(dtype)
    y = torch.zeros(rows, dtype=torch.int64, device=DEV)
    f = torch.zeros(rows, device=DEV)
    return x, y, f, torch.tensor([0, rows // 2, rows], device=DEV)


def calls(x, y, f, ends, **kw):
    return [lambda: ce.logp_rows(x, y, **kw), lambda: ce.policy_loss(x, y, f, f, 1.0, **kw),
            lambda: ce.policy_step(x, y, f, f, 1.0, **kw), lambda: ce.preference_loss(x, y, ends, 1.0, **kw),
            lambda: ce.preference_step(x, y, ends, 1.0, **kw)]


@pytest.mark.parametrize("which", range(5))
def test_refusals(which):
    x, y, f, ends = batch()

    def refused(error, xx=x, yy=y, ff=f, ee=ends, **kw):
        with pytest.raises(error):
            calls(xx, yy, ff, ee, **kw)[which]()
    refused(TypeError, xx=None)
    refused(TypeError, xx=x.double())
    refused(TypeError, xx=[1.0])
    refused(ValueError, xx=x.cpu())
    refused(ValueError, xx=x[0])
    refused(ValueError, xx=x.t())
    refused(ValueError, xx=x.expand(3, 6, 50))
    refused(ValueError, xx=x[:1].expand(6, 50))
    refused(ValueError, xx=x[:, :0])
    refused(ValueError, vocab=0)
    refused(ValueError, vocab=51)
    refused(TypeError, vocab=2.5)
    refused(TypeError, yy=None)
    refused(ValueError, yy=y[:-1])
    refused(ValueError, yy=y.int())
    refused(ValueError, yy=y.cpu())
    refused(ValueError, yy=y.repeat(2)[::2])
    refused(TypeError, weights=3)
    refused(ValueError, weights=f[1:])
    refused(ValueError, weights=f.double())
    refused(ValueError, weights=f.cpu())
    refused(ValueError, weights=torch.zeros(12, device=DEV)[::2])
    refused(TypeError, temperature="warm")
    for t in (0.0, -1.0, float("nan"), float("inf"), 1e9):
        refused(ce.CeError, temperature=t)


def test_policy_refusals():
    x, y, f, _ = batch()
    for call in (ce.policy_loss, ce.policy_step):
        for bad in (dict(old_logp=None), dict(advantages=None), dict(old_logp=f[1:]), dict(kl_coef=0.1),
                    dict(ref_logp=f.half()), dict(entropy=f[1:])):
            with pytest.raises(ValueError):
                call(**{**dict(logits=x, labels=y, old_logp=f, advantages=f, scale=1.0), **bad})
        for bad in (dict(scale=None), dict(clip_low="no")):
            with pytest.raises(TypeError):
                call(**{**dict(logits=x, labels=y, old_logp=f, advantages=f, scale=1.0), **bad})
        for bad in (dict(scale=float("nan")), dict(clip_low=-0.1), dict(clip_high=float("nan")), dict(entropy_coef=float("inf"))):
            with pytest.raises(ce.CeError):
                call(**{**dict(logits=x, labels=y, old_logp=f, advantages=f, scale=1.0), **bad})


def test_preference_refusals():
    x, y, _, ends = batch()
    for call in (ce.preference_loss, ce.preference_step):
        for bad in (dict(offsets=ends[:2]), dict(offsets=ends.int()), dict(offsets=ends.cpu()), dict(kind="best"),
                    dict(ref_logp=torch.zeros(3, device=DEV)), dict(offsets=ends[:, None])):
            with pytest.raises(ValueError):
                call(**{**dict(logits=x, labels=y, offsets=ends, scale=1.0), **bad})
        for bad in (dict(beta=0.0), dict(beta=float("nan")), dict(label_smoothing=0.7), dict(margin=float("inf")),
                    dict(kind="hinge", label_smoothing=0.1)):
            with pytest.raises(ce.CeError):
                call(**{**dict(logits=x, labels=y, offsets=ends, scale=1.0), **bad})


@pytest.mark.parametrize("which", [2, 4])
def test_gradient_refusals(which):
    x, y, f, ends = batch(6, 50, torch.bfloat16)
    flat = torch.zeros(6 * 50 + 8, dtype=torch.bfloat16, device=DEV)
    for grad in (torch.zeros(6, 50, device=DEV), torch.zeros(5, 50, dtype=x.dtype, device=DEV), x[:, :49],
                 torch.zeros(6, 50, dtype=x.dtype), torch.zeros(50, 6, dtype=x.dtype, device=DEV).t(),
                 torch.zeros(1, 50, dtype=x.dtype, device=DEV).expand(6, 50), flat):
        with pytest.raises(ValueError):
            calls(x, y, f, ends, grad=grad)[which]()
    wide = torch.zeros(6, 60, dtype=x.dtype, device=DEV)
    with pytest.raises(ce.CeError):  # overlaps the logits without being them
        calls(wide[:, :50], y, f, ends, grad=wide[:, 1:51])[which]()


def test_numbers_of_any_kind():
    """Python ints and floats and 0-d tensors as constants."""
    x, y, f, _ = batch()
    a = ce.policy_loss(x, y, f, f + 1, 1, clip_low=torch.tensor(0.25), temperature=1)
    b = ce.policy_loss(x, y, f, f + 1, 1.0, clip_low=0.25, temperature=1.0)
    assert all(torch.equal(u, v) for u, v in zip(a[:3], b[:3]))


def test_given_outputs():
    x, y, f, _ = batch()
    out, ent = torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    got = ce.logp_rows(x, y, entropy=ent, out=out)
    assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == ent.data_ptr()
    want = ce.logp_rows(x, y, entropy=True)
    assert torch.equal(out, want[0]) and torch.equal(ent, want[1])
    assert torch.equal(ce.logp_rows(x, y, out=out), want[0])
    step = ce.policy_step(x, y, f, f, 1.0, entropy=ent)
    assert step[4].data_ptr() == ent.data_ptr()
    with pytest.raises(ValueError):
        ce.logp_rows(x, y, out=out[1:])


def test_nothing_is_kept():
    x, y, f, ends = batch(200, 3000, torch.bfloat16)
    held = [x, y, f, ends]
    for _ in range(3):
        for c in calls(x, y, f, ends):
            c()
    torch.cuda.synchronize()
    gc.collect()
    refs, memory = [sys.getrefcount(t) for t in held], torch.cuda.memory_allocated()
    for _ in range(50):
        for c in calls(x, y, f, ends):
            c()
        for bad in (dict(weights=f[1:]), dict(temperature=0.0), dict(vocab=5000)):
            for c in calls(x, y, f, ends, **bad):
                with pytest.raises((ValueError, ce.CeError)):
                    c()
    torch.cuda.synchronize()
    gc.collect()
    assert [sys.getrefcount(t) for t in held] == refs
    assert torch.cuda.memory_allocated() == memory


def test_one_library():
    """The binding and the ctypes calls are of one loaded library: its counters count both."""
    x, y, f, ends = batch()
    ce.device_error_reset()
    ce.logp_rows(x, y + 50)
    ce.ce_rows(x, y + 50)
    assert ce.device_error_count()[0] == 12
    ce.device_error_reset()
    assert ce.device_error_count()[0] == 0


def test_leaves_that_require_grad():
    """Logits that require a gradient are read as they are; the results do not."""
    x, y, f, ends = batch()
    leaf = x.clone().requires_grad_()
    for a, b in zip(calls(leaf, y, f, ends), calls(x, y, f, ends)):
        u, v = a(), b()
        for p, q in zip(u if isinstance(u, tuple) else (u,), v if isinstance(v, tuple) else (v,)):
            if p is not None:
                assert torch.equal(p, q) and not p.requires_grad
    grad = ce.policy_step(leaf.detach(), y, f, f + 1, 1.0)[0]
    leaf.grad = grad
    assert leaf.grad is grad


def test_entropy_not_wanted():
    """False and None alike: the log-probabilities alone."""
    x, y, f, _ = batch()
    assert torch.equal(ce.logp_rows(x, y, entropy=None), ce.logp_rows(x, y))
    assert ce.policy_loss(x, y, f, f, 1.0, entropy=None)[3] is None
