"""Refusals of the choices' entry points, answered on the host before any
launch, and the 64-bit reference their GPU tests use. CPU only."""
import ctypes
import math

import pytest
import torch

import choices_ref as R
import row_wise_softmax_ce_gb300 as ce
from row_wise_softmax_ce_gb300 import build as cuda_build

V = ctypes.c_void_p
HUGE = (1 << 24) + 1


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return ce.lib()


def sample(lib, logits=V(4096), dtype=0, rows=4, cols=10, stride=10, uniforms=V(512), t=1.0, temps=None,
           tokens=V(1 << 20), logp=None, work=V(1 << 22)):
    return lib.sample_rows(logits, dtype, rows, cols, stride, uniforms, t, temps, tokens, logp, work, None)


def verify(lib, logits=V(4096), dtype=0, rows=4, cols=10, stride=10, drafts=V(512), q=V(8192), qs=10, offsets=V(1024),
           requests=2, uniforms=V(2048), t=1.0, temps=None, accepted=V(1 << 20), tokens=V(1 << 21), logp=None,
           work=V(1 << 22)):
    return lib.verify_drafts(logits, dtype, rows, cols, stride, drafts, q, qs, offsets, requests, uniforms, t, temps,
                             accepted, tokens, logp, work, None)


def how(score=0, k=2, groups=1, top_groups=1, group_top=2, renormalise=1, scale=1.0):
    return ctypes.byref(ce.Route(score, k, groups, top_groups, group_top, renormalise, scale))


def route(lib, logits=V(4096), dtype=0, rows=4, cols=12, stride=12, par=True, bias=None, weights=None,
          chosen=V(1 << 20), gates=V(1 << 21), counts=None, **kw):
    return lib.route_rows(logits, dtype, rows, cols, stride, how(**kw) if par else None, bias, weights, chosen, gates,
                          counts, None)


def grad(lib, logits=V(4096), dtype=0, rows=4, cols=12, stride=12, par=True, weights=None, chosen=V(512),
         gates_grad=V(1024), out=V(1 << 20), gs=12, **kw):
    return lib.route_grad(logits, dtype, rows, cols, stride, how(**kw) if par else None, weights, chosen, gates_grad,
                          out, gs, None)


CALLS = {"sample": sample, "verify": verify, "route": route, "grad": grad}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad", [dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(cols=0), dict(stride=9),
                                 dict(cols=HUGE, stride=HUGE), dict(logits=None), dict(rows=1 << 40, stride=1 << 40)],
                         ids=str)
def test_shared_arguments_refused(lib, name, bad):
    assert CALLS[name](lib, **bad) == ce.CE_EINVAL


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("bad", [dict(logits=V(4098)), dict(dtype=1, logits=V(4097)), dict(dtype=2, logits=V(4097))],
                         ids=str)
def test_misaligned_rows_refused(lib, name, bad):
    assert CALLS[name](lib, **bad) == ce.CE_EALIGN


@pytest.mark.parametrize("call", [sample, verify])
def test_temperatures(lib, call):
    for t in (-1.0, 1e-7, 1e7, math.nan, math.inf):
        assert call(lib, t=t) == ce.CE_EINVAL
    assert call(lib, temps=V(514)) == ce.CE_EALIGN
    if not torch.cuda.is_available():
        assert call(lib, t=0.0) == ce.CE_EDEVICE


@pytest.mark.parametrize("bad", [dict(uniforms=None), dict(tokens=None), dict(work=None)], ids=str)
def test_sample_arguments_refused(lib, bad):
    assert sample(lib, **bad) == ce.CE_EINVAL


@pytest.mark.parametrize("bad", [dict(uniforms=V(514)), dict(tokens=V((1 << 20) + 4)), dict(logp=V(1026)), dict(work=V(1032))],
                         ids=str)
def test_sample_alignment_refused(lib, bad):
    assert sample(lib, **bad) == ce.CE_EALIGN


def test_scratch(lib):
    """Enough for a row's steps of 256 vectors of 16 bytes at any phase, 8 bytes each."""
    for dtype, n in ((0, 4), (1, 8), (2, 8)):
        for vocab in (1, n, 256 * n, 256 * n + 1, 50257, 1 << 24):
            steps = -(-((vocab + n - 1 + n - 1) // n) // 256)
            assert lib.choice_work(dtype, 3, vocab, -1) >= 24 * steps
            assert lib.choice_work(dtype, 3, vocab, 5) >= 48 * steps
    assert lib.choice_work(1, 0, 10, -1) == 0
    for bad in ((3, 1, 10, 0), (0, -1, 10, 0), (0, 1, 0, 0), (0, 1, HUGE, 0), (0, 1, 10, -2), (0, 1 << 61, 1 << 20, 0)):
        assert lib.choice_work(*bad) == ce.CE_EINVAL


@pytest.mark.parametrize("bad", [dict(drafts=None), dict(offsets=None), dict(uniforms=None), dict(accepted=None),
                                 dict(tokens=None), dict(work=None), dict(requests=-1), dict(requests=1 << 41),
                                 dict(qs=9), dict(rows=2, qs=1 << 62)], ids=str)
def test_verify_arguments_refused(lib, bad):
    assert verify(lib, **bad) == ce.CE_EINVAL


@pytest.mark.parametrize("bad", [dict(drafts=V(516)), dict(offsets=V(1028)), dict(uniforms=V(2050)),
                                 dict(accepted=V((1 << 20) + 4)), dict(tokens=V((1 << 21) + 4)), dict(logp=V(1026)),
                                 dict(q=V(8194)), dict(work=V(1032))], ids=str)
def test_verify_alignment_refused(lib, bad):
    assert verify(lib, **bad) == ce.CE_EALIGN


@pytest.mark.parametrize("bad", [dict(par=False), dict(score=2), dict(score=-1), dict(k=0), dict(k=13), dict(k=33, cols=64, stride=64),
                                 dict(scale=math.nan), dict(scale=math.inf), dict(scale=-1e39), dict(cols=1025, stride=1025)], ids=str)
@pytest.mark.parametrize("call", [route, grad])
def test_router_refused(lib, call, bad):
    assert call(lib, **{"gs": 1025, **bad} if call is grad else bad) == ce.CE_EINVAL


@pytest.mark.parametrize("bad", [dict(groups=0), dict(groups=5), dict(groups=-2), dict(top_groups=0), dict(top_groups=2),
                                 dict(groups=4, top_groups=5), dict(group_top=0), dict(group_top=3),
                                 dict(groups=4, top_groups=1, k=4), dict(groups=33, cols=66, stride=66),
                                 dict(chosen=None), dict(gates=None)], ids=str)
def test_route_arguments_refused(lib, bad):
    assert route(lib, **bad) == ce.CE_EINVAL


@pytest.mark.parametrize("bad", [dict(bias=V(1026)), dict(weights=V(1026)), dict(chosen=V((1 << 20) + 4)),
                                 dict(gates=V((1 << 21) + 2)), dict(counts=V(1028))], ids=str)
def test_route_alignment_refused(lib, bad):
    assert route(lib, **bad) == ce.CE_EALIGN


@pytest.mark.parametrize("bad", [dict(chosen=None), dict(gates_grad=None), dict(out=None), dict(gs=11),
                                 dict(out=V(4096), gs=14), dict(out=V(4096 + 48)), dict(out=V(4096 - 40)),
                                 dict(rows=2, gs=1 << 62)], ids=str)
def test_grad_arguments_refused(lib, bad):
    assert grad(lib, **bad) == ce.CE_EINVAL


@pytest.mark.parametrize("bad", [dict(chosen=V(516)), dict(gates_grad=V(1026)), dict(out=V((1 << 20) + 2)),
                                 dict(weights=V(1026))], ids=str)
def test_grad_alignment_refused(lib, bad):
    assert grad(lib, **bad) == ce.CE_EALIGN


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses beside a CUDA device")
def test_outputs_over_the_rest_refused(lib):
    for where in (512, 512 + 12, 1024, 4096, 4096 + 152):
        assert sample(lib, temps=V(1024), logp=V(where)) == ce.CE_EINVAL
    for where in (512, 1024 + 8, 4096 + 144):
        assert sample(lib, temps=V(1024), tokens=V(where)) == ce.CE_EINVAL
    assert sample(lib, logp=V((1 << 20) + 16)) == ce.CE_EINVAL
    for name in ("accepted", "tokens", "logp", "work"):
        for where in (512 + 16, 1024 + 16, 2048 + 16, 4096 + 80, 8192 + 80, 16384):
            assert verify(lib, temps=V(16384), **{name: V(where)}) == ce.CE_EINVAL, (name, where)
    assert verify(lib, logp=V((1 << 21) + 16)) == ce.CE_EINVAL
    assert verify(lib, work=V((1 << 20) - 16)) == ce.CE_EINVAL
    assert sample(lib, work=V((1 << 20) - 16)) == ce.CE_EINVAL and sample(lib, work=V(4096 + 160 - 16)) == ce.CE_EINVAL
    for name in ("chosen", "gates", "counts"):
        for where in (512 + 8, 1024 + 8, 4096 + 96):
            assert route(lib, bias=V(512), weights=V(1024), **{name: V(where)}) == ce.CE_EINVAL, (name, where)
    assert route(lib, gates=V((1 << 20) + 32)) == ce.CE_EINVAL
    assert route(lib, counts=V((1 << 20) + 32)) == ce.CE_EINVAL
    for where in (512 - 100, 1024 + 16, 2048 - 100):
        assert grad(lib, weights=V(2048), out=V(where)) == ce.CE_EINVAL


def test_accepted_calls_reach_the_device_check(lib):
    if torch.cuda.is_available():
        pytest.skip("a CUDA device is present")
    for name, call in CALLS.items():
        assert call(lib) == ce.CE_EDEVICE, name
    assert grad(lib, out=V(4096)) == ce.CE_EDEVICE                                    # in place
    assert sample(lib, stride=20, logp=V(4096 + 48)) == ce.CE_EDEVICE                 # in the padding of row 0
    assert verify(lib, q=None, qs=0) == ce.CE_EDEVICE                                 # drafts that were looked up
    assert route(lib, groups=4, top_groups=2, k=6) == ce.CE_EDEVICE
    # nothing to do
    assert sample(lib, rows=0, logits=None, uniforms=None, tokens=None, work=None) == ce.CE_OK
    assert verify(lib, rows=0, requests=0, logits=None, drafts=None, q=None, uniforms=None, accepted=None, tokens=None,
                  work=None) == ce.CE_OK
    assert verify(lib, rows=0, logits=None, drafts=None, q=None, uniforms=None, tokens=None, work=None) == ce.CE_EDEVICE
    assert route(lib, rows=0, logits=None, chosen=None, gates=None) == ce.CE_OK
    assert route(lib, rows=0, logits=None, chosen=None, gates=None, counts=V(1024)) == ce.CE_EDEVICE
    assert grad(lib, rows=0, logits=None, chosen=None, gates_grad=None, out=None) == ce.CE_OK


def test_binding_refuses():
    x, u = torch.zeros(4, 12), torch.zeros(4)
    with pytest.raises(ValueError):
        ce.sample_rows(x, u)  # not on a CUDA device
    with pytest.raises(TypeError):
        ce.sample_rows(x.double(), u)
    with pytest.raises(ValueError):
        ce.route_rows(x, 2, score="tanh")
    with pytest.raises(ValueError):
        ce.route_grad(x, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2))


# -- the C structure and argument lists ---------------------------------------------

def test_layout(tmp_path):
    import os
    import re
    import subprocess
    fields = [f for f, _ in ce.Route._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "ce_rows.h"\nint main(void)\n{\nprintf("%zu", '
                   'sizeof(ce_route));\n' + "\n".join(f'printf(" %zu", offsetof(ce_route, {f}));' for f in fields)
                   + "\nreturn 0;\n}\n")
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(ce.HEADER), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    assert out.split() == [str(ctypes.sizeof(ce.Route))] + [str(getattr(ce.Route, f).offset) for f in fields]
    header = re.sub(r"/\*.*?\*/", " ", open(ce.HEADER).read(), flags=re.S)
    scores = dict(re.findall(r"CE_ROUTE_(\w+) = (\d+)", header))
    assert {k.lower(): int(v) for k, v in scores.items()} == ce.ROUTE_SCORES


@pytest.mark.parametrize("name", ["sample_rows", "verify_drafts", "route_rows", "route_grad"])
def test_arguments(lib, name):
    import re
    header = re.sub(r"/\*.*?\*/", " ", open(ce.HEADER).read(), flags=re.S)
    args = re.search(r"CE_API int %s\((.*?)\);" % name, header, re.S).group(1).split(",")

    def kind(arg):
        if "*" in arg or "ce_stream_t" in arg:
            return ctypes.c_void_p
        return {"int64_t": ctypes.c_int64, "int": ctypes.c_int, "double": ctypes.c_double}[arg.split()[0]]
    assert [kind(a) for a in args] == list(getattr(lib, name).argtypes)


# -- the reference itself ------------------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_reference_route_gradient(score, renormalise):
    g = torch.Generator().manual_seed(4)
    x = 2 * torch.randn(5, 9, generator=g, dtype=torch.float64)
    chosen = torch.tensor([[3, 1, 8], [0, -1, -1], [5, 5, 2], [-1, -1, -1], [7, 0, 4]])
    G = torch.randn(5, 3, generator=g)
    weights = torch.tensor([1.0, 2.0, 1.0, 1.0, 0.0])

    def total(v):
        s = torch.sigmoid(v) if score == "sigmoid" else torch.softmax(v, 1)
        on = (chosen >= 0).double()
        p = s.gather(1, chosen.clamp(min=0)) * on
        if renormalise:
            p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
        return 1.5 * (p * G * (weights != 0)[:, None]).sum()
    got, _ = R.route_grad64(x, chosen, G, score, renormalise, 1.5, weights)
    v = x.clone().requires_grad_()
    auto, = torch.autograd.grad(total(v), v)
    assert float((got - auto).abs().max()) < 1e-14
    h = 1e-6
    for r, j in [(0, 3), (0, 2), (1, 0), (2, 5), (2, 2), (3, 1), (4, 7)]:
        a, b = x.clone(), x.clone()
        a[r, j] += h
        b[r, j] -= h
        # central differences of an f64 sum of order 1: 1e-16 / 1e-6 of rounding, h^2 of truncation
        assert abs(float((total(a) - total(b)) / (2 * h)) - float(got[r, j])) < 1e-8


def test_reference_rejects():
    """Each check lets the right answer pass and not the one beside it."""
    x = torch.tensor([0.0, 1.0, -math.inf, 2.0, 0.5])
    p = torch.softmax(x.double(), 0)
    u = float(p[0] + 0.5 * p[1])
    R.check_sampled(x, u, 1.0, 1, float(p[1].log()), "right")
    for token, lp in ((0, float(p[0].log())), (2, 0.0), (3, float(p[3].log())), (-1, 0.0), (1, float(p[1].log()) + 1e-5)):
        with pytest.raises(AssertionError):
            R.check_sampled(x, u, 1.0, token, lp, "wrong")
    R.check_sampled(x, u, 0.0, 3, 0.0, "greedy")
    with pytest.raises(AssertionError):
        R.check_sampled(x, u, 0.0, 1, 0.0, "greedy")
    rows, y = torch.stack([x, x, x]), torch.stack([x.flip(0).nan_to_num(neginf=-3.0)] * 3)
    q = torch.softmax(y[0].double(), 0)
    ratio = float(p[0] / q[0])
    un = [[0.99 * ratio, 0.3], [0.9, 0.1], [0.5, 0.5]]
    rest = (p - q).clamp(min=0)
    t = int((rest.cumsum(0) > 0.1 * rest.sum()).nonzero()[0])
    last = 1
    assert float(p[last] / q[last]) < 0.9
    good = ([1], [0, t, -1])
    args = (rows, [0, last, -1], [0, 3], un, y, [1.0] * 3)
    R.check_verified(*args, *good, None)
    for bad in (([0], [last, -1, -1]), ([2], [0, last, 1]), ([1], [0, t, 1]), ([1], [0, (t + 1) % 5, -1])):
        with pytest.raises(AssertionError):
            R.check_verified(*args, *bad, None)
    z = torch.tensor([[0.0, 3.0, 1.0, 3.0]])
    s = torch.softmax(z.double(), 1)[0]
    R.check_routed(z, 2, torch.tensor([[1, 3]]), torch.tensor([[0.5, 0.5]]), None)
    R.check_routed(z, 2, torch.tensor([[1, 3]]), s[[1, 3]][None].float(), None, renormalise=False)
    for chosen, gates in (([[3, 1]], [[0.5, 0.5]]), ([[1, 2]], [[0.88, 0.12]]), ([[1, 3]], [[0.5, 0.501]])):
        with pytest.raises(AssertionError):
            R.check_routed(z, 2, torch.tensor(chosen), torch.tensor(gates), None)
