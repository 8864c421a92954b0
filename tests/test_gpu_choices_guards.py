"""Sentinels around every output and the work buffer of the choices (C ABI):
sample_rows, verify_drafts, route_rows and route_grad write nothing beside them,
whatever the offsets of the requests hold.

A work buffer has exactly the bytes that choice_work asks for. Outputs start at
every phase of 16 bytes that their alignment allows, rows at every phase."""
import ctypes
import math

import pytest
import torch

import row_wise_softmax_ce_gb300 as ce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": (0, torch.float32), "bf16": (1, torch.bfloat16), "f16": (2, torch.float16)}
MARGIN = 512  # bytes to either side
SENTINEL = 0xA5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)


class Guarded:
    """An output inside sentinels, `phase` bytes behind a 16-byte boundary."""

    def __init__(self, shape, dtype, phase=0):
        self.shape, self.dtype = shape, dtype
        n = math.prod(shape) * dtype.itemsize
        self.lo, self.hi = MARGIN + phase, MARGIN + phase + n
        self.buf = torch.full((self.hi + MARGIN,), SENTINEL, dtype=torch.uint8, device=DEV)

    @property
    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr() + self.lo)

    def get(self):
        """The output; its margins have been left alone."""
        torch.cuda.synchronize()
        assert bool((self.buf[:self.lo] == SENTINEL).all()) and bool((self.buf[self.hi:] == SENTINEL).all())
        return self.buf[self.lo:self.hi].clone().view(self.dtype).view(self.shape)


def p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def rows_of(rows, vocab, dtype, stride, lead, g):
    buf = torch.full((lead + rows * stride + 16,), 1e4)
    buf[::2] = math.nan
    buf[lead:lead + rows * stride].view(rows, stride)[:, :vocab] = 2 * torch.randn(rows, vocab, generator=g)
    return buf.to(dtype).to(DEV)[lead:lead + rows * stride].view(rows, stride)[:, :vocab]


def same(a, b):
    """Bit for bit."""
    bits = {8: torch.int64, 4: torch.int32, 2: torch.int16}[a.element_size()]
    return torch.equal(a.contiguous().view(bits), b.contiguous().view(bits))


def stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def scratch(code, rows, vocab, requests):
    return Guarded((ce.lib().choice_work(code, rows, vocab, requests),), torch.uint8)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 5), (7, 33), (5, 1017), (5, 1024), (5, 1025), (4, 2041), (4, 2048), (4, 2049),
                                        (3, 20011), (5003, 37), (601, 9001), (1, 300007)])
def test_sample(kind, rows, vocab):
    code, dtype = TYPES[kind]
    g = torch.Generator().manual_seed(rows + vocab)
    lead = vocab % 8
    x = rows_of(rows, vocab, dtype, vocab + rows % 3, lead, g)
    u = torch.rand(rows, generator=g).to(DEV)
    tokens, logp = Guarded((rows,), torch.int64, 8 * (lead & 1)), Guarded((rows,), torch.float32, 4 * (lead & 3))
    work = scratch(code, rows, vocab, -1)
    st = ce.lib().sample_rows(p(x), code, rows, vocab, x.stride(0), p(u), 0.9, None, tokens.ptr, logp.ptr, work.ptr, stream())
    assert st == ce.CE_OK
    want = ce.sample_rows(x, u, temperature=0.9, logp=True)
    work.get()
    assert same(tokens.get(), want[0]) and same(logp.get(), want[1])


TABLES = [[0, 3, 4, 9], [0, 9], [2, 2, 5, 5, 8], list(range(10)), [4], [0, 5, 3, 9], [-4, 2, 9], [0, 4, 900], [0, 1 << 40, 9],
          [9, 0], [3, -(1 << 50), 9], [9, 0, 9, 0, 9]]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("lookup", [False, True])
@pytest.mark.parametrize("vocab", [1, 5, 1024, 2041, 2049, 20011])
def test_verify(kind, lookup, vocab):
    code, dtype = TYPES[kind]
    g = torch.Generator().manual_seed(vocab)
    rows, lead = 9, vocab % 8
    x = rows_of(rows, vocab, dtype, vocab + 1, lead, g)
    y = None if lookup else rows_of(rows, vocab, dtype, vocab + 2, lead // 2, g)
    drafts = torch.randint(-1, vocab + 1, (rows,), generator=g).to(DEV)  # none, and one that is no token, among them
    u = torch.rand(rows, 2, generator=g).to(DEV)
    u[::2, 0] *= 1e-3
    for table in TABLES:
        ends, requests = torch.tensor(table, device=DEV), len(table) - 1
        accepted = Guarded((requests,), torch.int64, 8 * (lead & 1))
        tokens, logp = Guarded((rows,), torch.int64, 8 * (lead & 1)), Guarded((rows,), torch.float32, 4 * (lead & 3))
        work = scratch(code, rows, vocab, requests)
        st = ce.lib().verify_drafts(p(x), code, rows, vocab, x.stride(0), p(drafts), p(y), 0 if lookup else y.stride(0), p(ends),
                                    requests, p(u), 1.0, None, accepted.ptr, tokens.ptr, logp.ptr, work.ptr, stream())
        assert st == ce.CE_OK
        work.get()
        got, emitted, lp = accepted.get().tolist(), tokens.get(), logp.get()
        for n, a, b in zip(got, table, table[1:]):
            assert 0 <= n <= b - a if 0 <= a <= b <= rows else n == -1, (table, got)
        assert bool(((emitted >= -1) & (emitted < vocab)).all())
        for r in range(rows):  # a row in no request
            if not any(0 <= a <= r < b <= rows for a, b in zip(table, table[1:])):
                assert int(emitted[r]) == -1 and float(lp[r]) == 0, (table, r)
        if table == sorted(table) and 0 <= table[0] and table[-1] <= rows:
            want = ce.verify_drafts(x, drafts, ends, u, draft_logits=y, logp=True)
            assert got == want[0].tolist() and same(emitted, want[1]) and same(lp, want[2])
            # each request emits what it accepted and one token more, unless all its rows accepted
            for n, a, b in zip(got, table, table[1:]):
                assert bool((emitted[a + min(n + 1, b - a):b] == -1).all()) and bool((emitted[a:a + n] >= 0).all())


def router(score, k, renormalise, groups=1, top_groups=1):
    return ctypes.byref(ce.Route(ce.ROUTE_SCORES[score], k, groups, top_groups, 2, renormalise, 1.5))


SHAPES = [(1, 1, 1), (5, 7, 3), (33, 60, 4), (2003, 60, 4), (2003, 128, 9), (17, 256, 8), (4001, 256, 8), (9, 257, 17),
          (2501, 384, 8), (2501, 511, 20), (5, 1000, 32), (2001, 1024, 6)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("score,renormalise", [("softmax", 1), ("softmax", 0), ("sigmoid", 1), ("sigmoid", 0)])
@pytest.mark.parametrize("rows,E,k", SHAPES)
def test_route(kind, score, renormalise, rows, E, k):
    code, dtype = TYPES[kind]
    g = torch.Generator().manual_seed(rows + E)
    lead = E % 8
    x = rows_of(rows, E, dtype, E + lead % 3, lead, g)
    bias, w = (0.1 * torch.randn(E, generator=g)).to(DEV), (torch.rand(rows, generator=g) > 0.1).float().to(DEV)
    kw = dict(score=score, renormalise=bool(renormalise), scale=1.5, weights=w)
    chosen, gates = Guarded((rows, k), torch.int64, 8 * (lead & 1)), Guarded((rows, k), torch.float32, 4 * (lead & 3))
    counts = Guarded((E,), torch.int64, 8)
    st = ce.lib().route_rows(p(x), code, rows, E, x.stride(0), router(score, k, renormalise), p(bias), p(w), chosen.ptr, gates.ptr,
                             counts.ptr, stream())
    assert st == ce.CE_OK
    want = ce.route_rows(x, k, bias=bias, counts=True, **kw)
    chosen = chosen.get()
    assert same(chosen, want[0]) and same(gates.get(), want[1]) and same(counts.get(), want[2])
    G = torch.randn(rows, k, generator=g).to(DEV)
    grad = ce.route_grad(x, chosen, G, **kw)
    for pad, phase in ((0, 0), (0, 1), (3, 2)):  # rows side by side on 16 bytes, off them, and apart
        stride = E + pad
        out = Guarded((rows * stride,), dtype, phase * dtype.itemsize)
        st = ce.lib().route_grad(p(x), code, rows, E, x.stride(0), router(score, k, renormalise), p(w), p(chosen), p(G), out.ptr,
                                 stride, stream())
        assert st == ce.CE_OK
        got = out.get().view(rows, stride)
        assert same(got[:, :E], grad)
        assert bool((got[:, E:].contiguous().view(torch.uint8) == SENTINEL).all())
