"""The first calls of a process: a function of the library loads and prepares
its own kernels, not the objectives' as well; an objective's first call may be
one that a graph captures; the counters of a process count what it launched."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

START = """
import time, torch
import row_wise_softmax_ce_gb300 as ce
x = torch.randn(40, 30000, device="cuda:0")
y = torch.zeros(40, dtype=torch.int64, device="cuda:0")
f = torch.full((40,), -10.0, device="cuda:0")
ce.lib()
torch.cuda.synchronize()
"""

TIMED = START + """
t = time.perf_counter()
ce.ce_rows(x, y)
torch.cuda.synchronize()
ce.device_error_count()
print(1e3 * (time.perf_counter() - t))
"""

CAPTURED = START + """
ends = torch.tensor([0, 20, 40], device="cuda:0")
def everything(x):
    out = []
    for v in (x, x.bfloat16(), x.half()):
        for ent in (False, True):
            out += [ce.logp_rows(v, y, entropy=True)[ent]]
            out += [t for t in ce.policy_loss(v, y, f, f, 1.0, entropy=ent) if t is not None]
            out += [t for t in ce.policy_step(v, y, f, f, 1.0, entropy=ent) if t is not None]
        out += list(ce.preference_loss(v, y, ends, 1.0)) + list(ce.preference_step(v, y, ends, 1.0))
    return out
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = everything(x)
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, everything(x)))
print("same")
"""


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def run(program):
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout.strip()


def test_first_row_losses():
    """With the counters read: 1.0 ms without the objectives' kernels, 11.4 ms
    with all of them loaded beside; the best of a few processes."""
    times = []
    while len(times) < 4 and min(times, default=1e9) > 4.0:
        times.append(float(run(TIMED)))
    assert min(times) <= 4.0, times


def test_counters_before_and_after():
    """Nothing counted before the first objective, its bad labels after it."""
    assert run(START + """
print(*ce.device_error_count())
ce.device_error_reset()
ce.logp_rows(x, y - 1)
print(*ce.device_error_count())
ce.device_error_reset()
print(*ce.device_error_count())
""").split() == ["0", "0", "40", "0", "0", "0"]


def test_first_calls_captured():
    """No call before the capture: the graph's results are the eager calls'."""
    assert run(CAPTURED) == "same"
