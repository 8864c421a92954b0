"""choice_work refuses what sample_rows and verify_drafts refuse. CPU only."""
import ctypes

import pytest

import row_wise_softmax_ce_gb300 as ce
from row_wise_softmax_ce_gb300 import build as cuda_build

V = ctypes.c_void_p
MOST = (1 << 31) - 1


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return ce.lib()


@pytest.mark.parametrize("rows,vocab", [(MOST + 1, 10), (1 << 40, 10), (MOST + 1, 1 << 24), (4, (1 << 24) + 1)])
def test_refused_by_all(lib, rows, vocab):
    assert lib.sample_rows(V(4096), 0, rows, vocab, vocab, V(512), 1.0, None, V(1 << 50), None, V(1 << 60), None) == ce.CE_EINVAL
    for requests in (-1, 0, 2):
        assert lib.choice_work(0, rows, vocab, requests) == ce.CE_EINVAL


def test_most_rows(lib):
    """8 bytes for a step of 256 vectors, of each row, and of each draft row."""
    assert lib.choice_work(0, MOST, 1, -1) == 8 * MOST
    assert lib.choice_work(1, MOST, 1 << 24, MOST) == 16 * MOST * 8193
