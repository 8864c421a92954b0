"""The objectives across the shapes that choose their kernels: rows a warp
holds, rows of one CTA, of a cluster, longer than shared memory; grids smaller
than the rows; gradients of another 16-byte phase than the logits'; guard bands;
drawn cases. Against the 64-bit definition, within the bounds of
tests/objectives_ref.py."""
import math
import random
import threading

import pytest
import torch

import objectives_ref as R
import row_wise_softmax_ce_gb300 as ce
from test_gpu_objectives import DEV, TYPES, check, ids, inputs, logits_at

pytestmark = pytest.mark.gpu
SENTINEL = 7.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    ce.device_error_reset()
    yield
    ce.debug_grid_cap(0)
    assert ce.device_error_count()[1] == 0, "a bounded wait gave up"
    ce.device_error_reset()


def guarded(rows, vocab, dtype, before, pad):
    """A [rows, vocab] view of rows `pad` wider inside a SENTINEL-filled buffer, and a check of the rest."""
    stride = vocab + pad
    buf = torch.full((before + rows * stride + 70,), SENTINEL, dtype=dtype, device=DEV)
    view = buf[before:before + rows * stride].view(rows, stride)[:, :vocab]

    def untouched():
        view.fill_(SENTINEL)
        return bool((buf == SENTINEL).all())
    return view, untouched


def run_all(x, y, w, old, ref, adv, ends, T, kl, bonus, what, before=0, pad=0, kind="sigmoid"):
    rows, vocab = x.shape
    scale = 512.0 / rows
    kw = dict(weights=w, kl_coef=kl, entropy_coef=bonus, temperature=T)
    want = R.policy64(x, y, old, adv, scale, ref=ref, **kw)
    got = ce.logp_rows(x, y, weights=w, temperature=T)
    check({"logp": got}, want, f"{what}: logp_rows")
    kw["ref_logp"] = ref if kl else None
    names = ("loss", "loss_rows", "logp", "entropy")
    check(dict(zip(names, ce.policy_loss(x, y, old, adv, scale, **kw))), want, f"{what}: policy_loss")
    grad, untouched = guarded(rows, vocab, x.dtype, before, pad)
    got = ce.policy_step(x, y, old, adv, scale, grad=grad, **kw)
    check(dict(zip(("grad",) + names, got)), want, f"{what}: policy_step")
    assert untouched(), f"{what}: policy_step wrote outside its rows"
    if ends is None:
        return
    offs = torch.tensor(ends, device=DEV)
    kw = dict(weights=w, kind=kind, beta=0.3, temperature=T)
    want = R.preference64(x, y, ends, scale, **kw)
    names = ("loss", "loss_pairs", "seq_logp", "logp")
    check(dict(zip(names, ce.preference_loss(x, y, offs, scale, **kw))), want, f"{what}: preference_loss")
    grad, untouched = guarded(rows, vocab, x.dtype, before, pad)
    got = ce.preference_step(x, y, offs, scale, grad=grad, **kw)
    check(dict(zip(("grad",) + names, got)), want, f"{what}: preference_step")
    assert untouched(), f"{what}: preference_step wrote outside its rows"


def sequences(rows, pairs, rng):
    cuts = sorted(rng.randint(0, rows) for _ in range(2 * pairs + 1))
    return cuts


def a_case(rows, vocab, stride, dtype, offset, masked, T, kl, bonus, seed, pairs, before, pad, kind="sigmoid"):
    x, g = logits_at(rows, vocab, stride, dtype, seed, offset=offset)
    y, w, old, ref, adv = inputs(rows, vocab, g, x, masked, T)
    ends = sequences(rows, pairs, random.Random(seed)) if pairs else None
    what = f"{rows} x {vocab} of {stride} {ids(dtype)} +{offset}, grad +{before} of {vocab + pad}, seed {seed}"
    run_all(x, y, w, old, ref, adv, ends, T, kl, bonus, what, before, pad, kind)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("edge", [512, 2048, 4096, 8192, 32768])
@pytest.mark.parametrize("by", [-1, 0, 1, 5])
def test_where_kernels_change(dtype, edge, by):
    """Row lengths around the bytes at which another kernel takes over."""
    vocab = edge // (4 if dtype == torch.float32 else 2) + by
    a_case(37, vocab, vocab + 3, dtype, 1, 0.2, 0.9, 0.1, 0.01, vocab, 3, 2, 5)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,vocab", [(2000, 9000), (1300, 40000), (1, 151936), (2, 151936), (20, 151936), (152, 70001),
                                        (460, 20000)])
def test_splits(dtype, rows, vocab):
    """Few rows over clusters, more than one wave of rows, whole rows."""
    a_case(rows, vocab, vocab, dtype, 0, 0.1, 1.0, 0.05, 0.0, rows, 2 if rows > 1 else 0, 0, 0)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cap", [1, 2, 5])
@pytest.mark.parametrize("rows,vocab", [(40, 700), (23, 3001), (17, 20001), (9, 100003), (4, 1 << 21)])
def test_fewer_clusters_than_rows(dtype, cap, rows, vocab):
    """Every kernel looping over rows, some of them masked; the same bits as without a cap."""
    x, g = logits_at(rows, vocab, vocab + 1, dtype, seed=cap + vocab)
    y, w, old, ref, adv = inputs(rows, vocab, g, x, 0.4)
    args = (x, y, old, adv, 1.0)
    kw = dict(weights=w, ref_logp=ref, kl_coef=0.1, entropy_coef=0.01, entropy=True)
    want = R.policy64(x, y, old, adv, 1.0, ref=ref, weights=w, kl_coef=0.1, entropy_coef=0.01)
    free = ce.policy_step(*args, **kw)
    ce.debug_grid_cap(cap)
    try:
        step, loss = ce.policy_step(*args, **kw), ce.policy_loss(*args, **kw)
        pref = ce.preference_step(x, y, torch.tensor([0, rows // 2, rows], device=DEV), 1.0, weights=w)
    finally:
        ce.debug_grid_cap(0)
    names = ("loss", "loss_rows", "logp", "entropy")
    check(dict(zip(("grad",) + names, step)), want, "step")
    check(dict(zip(names, loss)), want, "loss")
    for a, b in zip(step, free):
        assert torch.equal(a, b)
    wantp = R.preference64(x, y, [0, rows // 2, rows], 1.0, weights=w)
    check(dict(zip(("grad", "loss", "loss_pairs", "seq_logp", "logp"), pref)), wantp, "preference")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("vocab", [1, 3, 17, 31, 250, 2040, 4000, 30011])
@pytest.mark.parametrize("offset,before,pad", [(0, 1, 0), (1, 0, 1), (3, 6, 2), (7, 2, 7), (5, 5, 3)])
def test_phases(dtype, vocab, offset, before, pad):
    """Logits and gradients that start at every pair of phases, rows shifting by their strides."""
    a_case(11, vocab, vocab + (offset % 3), dtype, offset, 0.0, 1.0, 0.0, 0.0, vocab + offset, 2, before, pad)


def test_zero_rows_of_a_wide_vocabulary():
    for dtype in TYPES:
        for vocab in (50257, 151936, 1 << 22):
            x = torch.empty(0, vocab, dtype=dtype, device=DEV)
            y, f = torch.empty(0, dtype=torch.int64, device=DEV), torch.empty(0, device=DEV)
            assert float(ce.policy_step(x, y, f, f, 1.0)[1]) == 0.0
            out = ce.preference_step(x, y, torch.tensor([0, 0, 0], device=DEV), 1.0)
            assert abs(float(out[1]) - math.log(2)) < 1e-6
            assert float(ce.preference_loss(x, y, torch.tensor([0], device=DEV), 1.0)[0]) == 0.0


def test_entropy_bonus_without_the_entropies():
    x, g = logits_at(33, 1000, 1000, torch.bfloat16, seed=8)
    y, w, old, ref, adv = inputs(33, 1000, g, x, 0.2)
    a = ce.policy_step(x, y, old, adv, 1.0, weights=w, entropy_coef=0.02)
    b = ce.policy_step(x, y, old, adv, 1.0, weights=w, entropy_coef=0.02, entropy=True)
    assert a[4] is None and b[4] is not None
    for u, v in zip(a[:4], b[:4]):
        assert torch.equal(u, v)


def test_one_row_of_any_stride():
    """A single row's stride is not its own: a slice of a wider tensor, and an expanded row."""
    big = torch.randn(5, 4096, device=DEV)
    y, f = torch.tensor([7], device=DEV), torch.zeros(1, device=DEV)
    for x in (big[2:3, 100:1300], big[:1].expand(1, 4096), big[3:4, :1]):
        yy = y.clamp(max=x.shape[1] - 1)
        want = R.policy64(x, yy, f, f + 1, 1.0)
        got = ce.policy_step(x, yy, f, f + 1, 1.0)
        check(dict(zip(("grad", "loss", "loss_rows", "logp"), got)), want, "one row")


def test_one_row_in_place_of_a_wider_one():
    """The first columns of a single wider row, in place: the rest of it is left alone."""
    for dtype in TYPES:
        x = torch.randn(1, 900, device=DEV).to(dtype)
        y, f = torch.tensor([3], device=DEV), torch.zeros(1, device=DEV)
        want, pref = R.policy64(x[:, :700], y, f, f + 1, 1.0), R.preference64(x[:, :700], y, [0, 1, 1], 1.0)
        z = x.clone()
        ce.policy_step(z, y, f, f + 1, 1.0, vocab=700, grad=z)
        R.assert_near(z[:, :700], want["grad"], "policy")
        assert torch.equal(z[:, 700:], x[:, 700:])
        z = x.clone()
        ce.preference_step(z, y, torch.tensor([0, 1, 1], device=DEV), 1.0, vocab=700, grad=z)
        R.assert_near(z[:, :700], pref["grad"], "preference")
        assert torch.equal(z[:, 700:], x[:, 700:])


def test_sums_that_overflow():
    """A weighted loss beyond f32 is infinite, not NaN; beyond f32 before the scale only, likewise."""
    x, y, f = torch.zeros(3, 8, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV), torch.zeros(3, device=DEV)
    w = torch.full((3,), 3e38, device=DEV)
    old = torch.full((3,), -math.log(8) - 10, device=DEV)  # a ratio of e^10, unclipped at a negative advantage
    loss = ce.policy_loss(x, y, old, f - 1, 1.0, weights=w)[0]
    assert float(loss) == math.inf
    seq = ce.preference_loss(x, y, torch.tensor([0, 2, 3], device=DEV), 1.0, weights=w)[2]
    assert float(seq[0]) == -math.inf and float(seq[1]) == -math.inf


def test_large_weights_and_long_sums():
    """A loss summed over more rows than one CTA takes, of both signs."""
    rows = 20011
    x, g = logits_at(rows, 64, 64, torch.float32, seed=12)
    y, w, old, ref, adv = inputs(rows, 64, g, x, 0.3)
    w = w * 1000.0 * torch.where(torch.rand(rows, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    want = R.policy64(x, y, old, adv, 1e-3, weights=w)
    got = ce.policy_step(x, y, old, adv, 1e-3, weights=w)
    check(dict(zip(("grad", "loss", "loss_rows", "logp"), got)), want, "long sum")
    ends = [0, 9000, 12000, 12001, 12001, 20011, 20011]
    want = R.preference64(x, y, ends, 1.0, weights=w / 1000, average=True, beta=0.05)
    got = ce.preference_step(x, y, torch.tensor(ends, device=DEV), 1.0, weights=w / 1000, average=True, beta=0.05)
    check({"seq_logp": got[3], "logp": got[4]}, want, "long sequences")


def test_many_pairs():
    """More pairs than the join has CTAs."""
    pairs, vocab = 3000, 40
    rows = 2 * pairs + 11
    x, g = logits_at(rows, vocab, vocab, torch.bfloat16, seed=13)
    y, *_ = inputs(rows, vocab, g, x, 0.0)
    ends = list(range(2 * pairs + 1))
    want = R.preference64(x, y, ends, 1.0 / pairs, beta=0.5)
    got = ce.preference_step(x, y, torch.tensor(ends, device=DEV), 1.0 / pairs, beta=0.5)
    check(dict(zip(("grad", "loss", "loss_pairs", "seq_logp", "logp"), got)), want, "many pairs")


def test_host_threads():
    """Four host threads, each on its own stream and batch: the bits of a call alone."""
    batches = []
    for s in range(4):
        x, g = logits_at(90 + s, 5000 + 4001 * s, 5000 + 4001 * s, torch.bfloat16, seed=s)
        y, w, old, ref, adv = inputs(x.shape[0], x.shape[1], g, x, 0.1)
        batches.append((x, y, w, old, adv, torch.tensor([0, 20, 40, 60, 80], device=DEV)))

    def work(b):
        x, y, w, old, adv, ends = b
        return list(ce.policy_step(x, y, old, adv, 1.0, weights=w)[:4]) + list(ce.preference_step(x, y, ends, 1.0, weights=w))
    want = [work(b) for b in batches]
    torch.cuda.synchronize()
    bad = []

    def thread(k):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = work(batches[k])
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                    bad.append(k)
    threads = [threading.Thread(target=thread, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_beside_the_cross_entropy_in_one_graph():
    """A captured step of both kinds, replayed on new logits: the cross-entropy
    step's results are what they are without the objectives beside it."""
    rows, vocab = 128, 8000
    x, g = logits_at(rows, vocab, vocab, torch.float32, seed=21)
    y, w, old, ref, adv = inputs(rows, vocab, g, x, 0.0)
    z, _ = logits_at(rows, vocab, vocab, torch.float32, seed=22)

    def step():
        return list(ce.ce_grad_step(x, y, 1.0 / rows)) + list(ce.policy_step(x, y, old, adv, 1.0 / rows)[:4]) + \
            [ce.argmax_rows(x)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(z)
    want = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("seed", range(60))
def test_drawn(seed):
    rng = random.Random(seed)
    dtype = rng.choice(TYPES)
    vocab = int(round(math.exp(rng.uniform(0, math.log(160000)))))
    rows = max(1, min(int(round(math.exp(rng.uniform(0, math.log(3000))))), 12_000_000 // vocab))
    a_case(rows, vocab, vocab + rng.choice([0, 0, 1, 7, 64]), dtype, rng.choice([0, 0, 1, 4, 7]), rng.choice([0.0, 0.3, 0.9]),
           rng.choice([1.0, 0.5, 1.7]), rng.choice([0.0, 0.2]), rng.choice([0.0, 0.03]), seed, rng.choice([1, 2, 9]),
           rng.choice([0, 0, 1, 3]), rng.choice([0, 0, 2, 5]), rng.choice(["sigmoid", "squared"]))


def c_output(n, dtype=torch.float32):
    """n elements between sentinels, and a check that the sentinels are whole."""
    buf = torch.full((n + 96,), SENTINEL, dtype=dtype, device=DEV)

    def whole():
        return bool((buf[:48] == SENTINEL).all()) and bool((buf[48 + n:] == SENTINEL).all())
    return buf[48:48 + n], whole


@pytest.mark.parametrize("rows,vocab", [(1, 5), (37, 900), (130, 9000), (5, 100003)])
def test_c_calls_write_their_outputs_only(rows, vocab):
    """The C ABI: every output between sentinels, the work buffer of a preference
    call used by two calls in a row, a reference that is not wanted never read."""
    import ctypes
    L, par = ce.lib(), ce.Policy(1.0, 1.0, 0.2, 0.2, 0.0, 0.01)
    x, g = logits_at(rows, vocab, vocab, torch.bfloat16, seed=rows)
    y, w, old, ref, adv = inputs(rows, vocab, g, x, 0.3)
    bad_ref = torch.full((rows,), math.nan, device=DEV)
    s = torch.cuda.current_stream().cuda_stream
    outs = [c_output(rows) for _ in range(3)] + [c_output(1)]
    grad = c_output(rows * vocab, torch.bfloat16)
    (loss_rows, _), (logp, _), (ent, _), (loss, _) = outs
    st = L.policy_step(x.data_ptr(), 1, rows, vocab, vocab, y.data_ptr(), old.data_ptr(), adv.data_ptr(),
                       bad_ref.data_ptr(), w.data_ptr(), ctypes.byref(par), grad[0].data_ptr(), vocab,
                       loss_rows.data_ptr(), logp.data_ptr(), ent.data_ptr(), loss.data_ptr(), s)
    assert st == ce.CE_OK and all(whole() for _, whole in outs + [grad])
    want = R.policy64(x, y, old, adv, 1.0, weights=w, entropy_coef=0.01)
    check({"loss": loss[0], "loss_rows": loss_rows, "logp": logp, "entropy": ent, "grad": grad[0].view(rows, vocab)}, want,
          "policy_step")
    st = L.policy_loss(x.data_ptr(), 1, rows, vocab, vocab, y.data_ptr(), old.data_ptr(), adv.data_ptr(), None,
                       w.data_ptr(), ctypes.byref(par), loss_rows.data_ptr(), logp.data_ptr(), None, loss.data_ptr(), s)
    assert st == ce.CE_OK and all(whole() for _, whole in outs)
    check({"loss": loss[0], "loss_rows": loss_rows, "logp": logp}, want, "policy_loss")
    assert L.logp_rows(x.data_ptr(), 1, rows, vocab, vocab, y.data_ptr(), w.data_ptr(), 1.0, logp.data_ptr(),
                       ent.data_ptr(), s) == ce.CE_OK
    assert all(whole() for _, whole in outs)
    check({"logp": logp, "entropy": ent}, want, "logp_rows")

    ends = [0, rows // 3, rows // 2, rows // 2, rows]
    offs, pp = torch.tensor(ends, device=DEV), ce.Preference(0.5, 1.0, 0.2, 0.0, 0.1, 0, 0)
    seq, pairs, work = c_output(4), c_output(2), c_output(4 * (rows + 1))
    for _ in range(2):
        st = L.preference_step(x.data_ptr(), 1, rows, vocab, vocab, y.data_ptr(), w.data_ptr(), offs.data_ptr(), 2, None,
                               ctypes.byref(pp), grad[0].data_ptr(), vocab, logp.data_ptr(), seq[0].data_ptr(),
                               pairs[0].data_ptr(), loss.data_ptr(), work[0].data_ptr(), s)
        assert st == ce.CE_OK and all(whole() for _, whole in outs + [grad, seq, pairs, work])
        want = R.preference64(x, y, ends, 0.5, weights=w, beta=0.2, margin=0.1)
        check({"loss": loss[0], "loss_pairs": pairs[0], "seq_logp": seq[0], "logp": logp,
               "grad": grad[0].view(rows, vocab)}, want, "preference_step")
        loss.fill_(SENTINEL)
    small = c_output(4)
    st = L.preference_loss(x.data_ptr(), 1, rows, vocab, vocab, y.data_ptr(), w.data_ptr(), offs.data_ptr(), 2, None,
                           ctypes.byref(pp), logp.data_ptr(), seq[0].data_ptr(), pairs[0].data_ptr(), loss.data_ptr(),
                           small[0].data_ptr(), s)
    assert st == ce.CE_OK and all(whole() for _, whole in outs + [seq, pairs, small])
    check({"loss": loss[0], "loss_pairs": pairs[0], "seq_logp": seq[0], "logp": logp}, want, "preference_loss")


@pytest.mark.parametrize("which", ["old_logp", "advantages", "ref_logp"])
def test_numbers_that_are_not(which):
    """A NaN among a row's numbers makes that row NaN, and no other."""
    rows, vocab = 9, 300
    x, g = logits_at(rows, vocab, vocab, torch.float32, seed=2)
    y, w, old, ref, adv = inputs(rows, vocab, g, x, 0.0)
    kw = {"old_logp": old, "advantages": adv, "ref_logp": ref}
    kw[which] = kw[which].clone()
    kw[which][4] = math.nan
    grad, loss, rows_, logp, _ = ce.policy_step(x, y, scale=1.0, kl_coef=0.1, **kw)
    want = R.policy64(x, y, kw["old_logp"], kw["advantages"], 1.0, ref=kw["ref_logp"], kl_coef=0.1)
    check({"grad": grad, "loss": loss, "loss_rows": rows_, "logp": logp}, want, which)
    assert math.isnan(rows_[4]) and bool(torch.isnan(grad[4]).all()) and not math.isnan(logp[4])
    assert int(torch.isnan(rows_).sum()) == 1
