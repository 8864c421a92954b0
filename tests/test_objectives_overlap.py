"""Outputs of the objectives that share memory with an input or with one
another are refused on the host, before any launch. CPU only: the addresses are
made up."""
import pytest
import torch

import row_wise_softmax_ce_gb300 as ce
from test_objectives_abi import CALLS, V, lib, logp, policy, preference  # noqa: F401  (lib: a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses beside a CUDA device")

# where the calls of test_objectives_abi put what they pass: 4 rows of 10 f32 logits, 1 pair
LOGITS, LABELS, WEIGHTS, GRAD = 4096, 512, 2048, 1 << 16
AT = dict(logits=V(LOGITS), dtype=0, weights=V(WEIGHTS))


@pytest.mark.parametrize("where", [LABELS, LABELS + 28, LABELS - 12, WEIGHTS, WEIGHTS + 4, WEIGHTS - 4, LOGITS - 12,
                                   LOGITS + 156, LOGITS + 80])
@pytest.mark.parametrize("name", ["out", "entropy"])
def test_logp_outputs_over_inputs(lib, name, where):  # noqa: F811
    assert logp(lib, **AT, **{name: V(where)}) == ce.CE_EINVAL


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("name", ["out", "entropy", "loss_rows", "loss"])
@pytest.mark.parametrize("where", [LABELS + 4, WEIGHTS + 12, 1024, 1040 + 8, 1056 + 12, LOGITS + 8])
def test_policy_outputs_over_inputs(lib, step, name, where):  # noqa: F811
    assert policy(lib, step, **AT, **{name: V(where)}) == ce.CE_EINVAL


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("name", ["out", "seq", "loss_pairs", "loss", "work"])
@pytest.mark.parametrize("where", [LABELS + 16, WEIGHTS, 1024 + 16, 8192, LOGITS + 16])
def test_preference_outputs_over_inputs(lib, step, name, where):  # noqa: F811
    assert preference(lib, step, **AT, ref=V(8192), **{name: V(where)}) == ce.CE_EINVAL


def test_outputs_over_one_another(lib):  # noqa: F811
    assert logp(lib, **AT, entropy=V(1 << 20)) == ce.CE_EINVAL
    assert logp(lib, **AT, entropy=V((1 << 20) + 12)) == ce.CE_EINVAL
    for step in (False, True):
        assert policy(lib, step, **AT, entropy=V(1 << 21)) == ce.CE_EINVAL
        assert policy(lib, step, **AT, out=V((1 << 20) - 4)) == ce.CE_EINVAL
        assert policy(lib, step, **AT, loss=V((1 << 20) + 8)) == ce.CE_EINVAL
        assert preference(lib, step, **AT, seq=V((1 << 20) + 12)) == ce.CE_EINVAL
        assert preference(lib, step, **AT, loss=V(1 << 22)) == ce.CE_EINVAL
        assert preference(lib, step, **AT, loss=V((1 << 24) + 12)) == ce.CE_EINVAL
    # the work buffer of a step is 16 (rows + 1) bytes, of a loss 16
    assert preference(lib, True, **AT, loss=V((1 << 24) + 76)) == ce.CE_EINVAL
    assert preference(lib, True, **AT, loss=V((1 << 24) + 80)) == ce.CE_EDEVICE
    assert preference(lib, False, **AT, loss=V((1 << 24) + 16)) == ce.CE_EDEVICE


@pytest.mark.parametrize("name", ["policy_step", "preference_step"])
def test_gradient_over_the_rest(lib, name):  # noqa: F811
    call = CALLS[name]
    assert call(lib, **AT, grad=V(WEIGHTS - 156)) == ce.CE_EINVAL
    assert call(lib, **AT, grad=V(LABELS + 8)) == ce.CE_EINVAL
    assert call(lib, **AT, grad=V(1024 - 100)) == ce.CE_EINVAL
    assert call(lib, **AT, grad=V((1 << 20) - 100)) == ce.CE_EINVAL


@pytest.mark.parametrize("name", CALLS)
def test_side_by_side_is_accepted(lib, name):  # noqa: F811
    """Neighbours without a shared byte, the padding of rows, and what a call does not read."""
    call = CALLS[name]
    assert call(lib, **AT) == ce.CE_EDEVICE
    assert call(lib, **AT, out=V(LOGITS + 160)) == ce.CE_EDEVICE       # behind the last logit
    assert call(lib, **AT, out=V(LOGITS - 16)) == ce.CE_EDEVICE
    assert call(lib, **AT, out=V(WEIGHTS + 16)) == ce.CE_EDEVICE
    assert call(lib, **AT, stride=20, out=V(LOGITS + 80 + 40)) == ce.CE_EDEVICE   # in the padding of row 1
    assert call(lib, **AT, stride=20, out=V(LOGITS + 80 + 64)) == ce.CE_EDEVICE   # up to row 2
    assert call(lib, **AT, stride=20, out=V(LOGITS + 80 + 36)) == ce.CE_EINVAL    # row 1's last logit
    assert call(lib, **AT, stride=20, out=V(LOGITS + 80 + 68)) == ce.CE_EINVAL    # row 2's first
    if name.startswith("policy"):
        assert call(lib, **AT, kl=0.0, ref=V(1 << 21)) == ce.CE_EDEVICE  # a reference that is not read
    if name.endswith("step"):
        assert call(lib, **AT, grad=V(LOGITS)) == ce.CE_EDEVICE          # in place


def test_no_rows_share_nothing(lib):  # noqa: F811
    assert policy(lib, True, rows=0, loss=V(LABELS)) == ce.CE_EDEVICE
    assert preference(lib, True, rows=0, pairs=0, loss=V(LABELS)) == ce.CE_EDEVICE
    assert preference(lib, True, rows=0, pairs=0, loss=V(1024)) == ce.CE_EINVAL  # offsets[0] is read
