"""The places that draws_ref.py allows a drawn column: the right one and its
rounding, not one a lane or a warp away. CPU only."""
import math

import pytest
import torch

import draws_ref as D

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def right(w, u):
    c = w.cumsum(0)
    return min(int((c <= u * c[-1]).sum()), len(w) - 1)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab,away", [(700, 1), (50257, 2), (200001, 8), (200001, 64)])
def test_own_places(dtype, vocab, away):
    g = torch.Generator().manual_seed(vocab)
    x = (0.5 * torch.randn(vocab, generator=g)).to(TYPES[dtype])
    w = torch.softmax(x.double(), 0)
    for u in (0.03, 0.25, 0.5, 0.77, 0.96):
        token = right(w, u)
        assert D.check_own(x, 1.0, u, token) == 0.0
        for wrong in (token - away, token + away):
            with pytest.raises(AssertionError):
                D.check_own(x, 1.0, u, wrong)
    with pytest.raises(AssertionError):
        D.check_own(x, 1.0, 0.5, -1)


def test_place_without_a_column():
    """Measured in what is drawn from, whatever the column that is left out holds."""
    g = torch.Generator().manual_seed(1)
    x = 0.5 * torch.randn(50176, generator=g)
    x[777] = 80.0
    w = torch.exp(x.double())
    w[777] = 0.0
    for u in (0.2, 0.8):
        token = right(w, u)
        assert D.check_own(x, 1.0, u, token, leave=777) == 0.0
        for wrong in (token - 4, token + 4, 777):
            with pytest.raises(AssertionError):
                D.check_own(x, 1.0, u, wrong, leave=777)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab,away", [(700, 2), (50257, 64)])
def test_rest_places(dtype, vocab, away):
    g = torch.Generator().manual_seed(vocab)
    x = 0.5 * torch.randn(vocab, generator=g)
    y = (x + 0.5 * torch.randn(vocab, generator=g)).to(TYPES[dtype])
    x = x.to(TYPES[dtype])
    w = (torch.softmax(x.double(), 0) - torch.softmax(y.double(), 0)).clamp(min=0)
    for u in (0.1, 0.5, 0.9):
        token = right(w, u)
        assert D.check_rest(x, y, 1.0, u, token) == 0.0
        for wrong in (token - away, token + away):
            with pytest.raises(AssertionError):
                D.check_rest(x, y, 1.0, u, wrong)
    assert D.check_rest(x, x.clone(), 1.0, 0.5, 3) is None  # nothing but rounding


def test_steps():
    for size in (2, 4):
        n = 16 // size
        for vocab in (1, 2, 256 * n - n + 1, 256 * n - n + 2, 50257, 1 << 24):
            most = max(-(-(phase + vocab) // n) for phase in range(n))
            assert D.steps_of(vocab, size) == -(-most // 256)
    assert math.isclose(2.0 ** float(D.exponents(torch.tensor([0.0, 1.0]), 0.5)[0]), math.exp(-2.0), rel_tol=1e-15)
