"""The objectives over sampled answers and pairs of answers in 64 bits, from
their definitions (include/ce_rows.h), with a bound of each output's rounding
error beside it. Works on any device; used with torch tensors.

Rounding, counted in U = 2^-24 (half a step of f32 at 1) of the value named:
  exp((x - m) / T)   the subtraction, the factor log2(e) / T and its product
                     round the exponent y by 3 U |y|, ex2.approx adds 4 U of
                     the result: e (3 |y| + 4) U
  s                  its terms' errors (|y| e <= 1/e: 3/e + 4 < 6 U of s), and
                     one U of s per addition on the way of a term: at most
                     DEPTH, the additions in one thread's chain, its warp's,
                     CTA's and cluster's joins, each with a rescaling
  log s              the relative error of s, and 2 U of its value
  (x_y - m) / T      3 U of its value
Everything after is carried through the formulas to first order and counted
with the same factors (expf, expm1f, logf, log1pf: 4 U of their value).
"""
import math

import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# below these a result may be flushed or rounded to a denormal of its type
LEAST = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def depth(vocab):
    """Additions on the way of one term: 32 threads at least share a row, 16
    pairs a push and then one addition each; 5 levels in each of warp, CTA and
    cluster."""
    return vocab / 32 / 16 + 16 + 2 * 15


def rows64(x, labels, live, T):
    """f64 row quantities of rows that count; elsewhere zeros."""
    z = x.double() / T
    m = z.amax(1, keepdim=True)
    nan = ~torch.isfinite(m[:, 0]) | torch.isnan(z).any(1)
    d = z - m
    e = d.exp()
    s = e.sum(1)
    V = x.shape[1]
    good = (labels >= 0) & (labels < V)
    at = labels.clamp(0, V - 1)
    dy = d.gather(1, at[:, None])[:, 0]
    logp = dy - s.log()
    H = s.log() - torch.where(e > 0, e * d, 0.0).sum(1) / s
    logp = torch.where(nan | ~good, math.nan, logp)
    H = torch.where(nan, math.nan, H)
    err_s = (6 + depth(V)) * U  # relative
    t_logp = err_s + 2 * U * s.log() + 3 * U * dy.abs() + U * logp.abs() + 2 * U
    # u / (T s): its terms e d carry the relative errors of e and of d, its sum one U per addition of sum |e d|
    t_H = t_logp.nan_to_num(0.0) * 0 + err_s + 2 * U * s.log() + (2 * err_s + 8 * U) * (s.log() - H).abs() + 2 * U * H.abs()
    zero = torch.zeros_like(logp)
    pick = lambda v: torch.where(live, v, zero)  # noqa: E731
    p = e / s[:, None]
    p = torch.where((nan & live)[:, None], math.nan, p)
    return {"d": d, "p": p, "s": s, "at": at, "logp": pick(logp), "H": pick(H), "t_logp": pick(t_logp).nan_to_num(0.0),
            "t_H": pick(t_H).nan_to_num(0.0), "err_s": err_s}


def live_rows(weights, rows, device):
    w = torch.ones(rows, dtype=torch.float64, device=device) if weights is None else weights.double()
    return w, w != 0


def grad64(r, g, t_g, f, dtype, bonus=0.0):
    """f (g ([y] - p) + bonus p (log p + H)) and a bound of its error (bound t_g of g)."""
    p, d = r["p"], r["d"]
    y = torch.zeros_like(p)
    y.scatter_(1, r["at"][:, None], 1.0)
    grad = g[:, None] * (y - p)
    rel_p = r["err_s"] + (3 * d.abs() + 8) * U
    rel_p = torch.where(p > 0, rel_p, 0.0)
    tol = t_g[:, None] * (y + p) + g.abs()[:, None] * (p * (rel_p + 4 * U) + 4 * U * y)
    if bonus:
        lp = torch.where(p > 0, d - r["s"].log()[:, None], 0.0)
        term = p * (lp + r["H"][:, None])
        grad = grad + bonus * term
        tol = tol + abs(bonus) * p * ((lp.abs() + r["H"][:, None].abs()) * (rel_p + 8 * U) + r["t_H"][:, None]
                                      + r["err_s"] + 4 * U * (d.abs() + r["s"].log()[:, None]).nan_to_num(0.0, posinf=0.0))
    grad, tol = grad * f[:, None], tol * f.abs()[:, None]
    dead = (f == 0)[:, None]
    grad = torch.where(dead, 0.0, grad)
    # two roundings of the f32 factors, one to the type
    tol = torch.where(dead, 0.0, tol.nan_to_num(0.0) + grad.abs().nan_to_num(0.0) * (HALF_STEP[dtype] + 4 * U) + LEAST[dtype])
    return grad, tol


def policy64(x, labels, old, adv, scale, ref=None, weights=None, clip_low=0.2, clip_high=0.2, kl_coef=0.0,
             entropy_coef=0.0, temperature=1.0):
    """{name: (value, bound)} of loss, loss_rows, logp, entropy, grad."""
    w, live = live_rows(weights, x.shape[0], x.device)
    x = torch.where(live[:, None], x, torch.zeros_like(x))
    labels = torch.where(live, labels, 0)
    r = rows64(x, labels, live, temperature)
    zero = torch.zeros_like(w)
    A, o = torch.where(live, adv.double(), zero), torch.where(live, old.double(), zero)
    ratio = (r["logp"] - o).exp()
    t_ratio = ratio * (r["t_logp"] + U * (r["logp"] - o).abs() + 4 * U)
    held = ratio.clamp(1 - clip_low, 1 + clip_high)
    plain, clipped = -A * ratio, -A * held
    rows = torch.where(plain < clipped, clipped, plain)
    rows = torch.where(torch.isnan(plain), plain, rows)
    g = torch.where(plain < clipped, 0.0, plain)
    t_rows = A.abs() * (t_ratio + 2 * U * ratio)
    t_g = torch.where(plain < clipped, 0.0, A.abs() * (t_ratio + 2 * U * ratio))
    if kl_coef:
        far = torch.where(live, ref.double(), zero) - r["logp"]
        t_far = r["t_logp"] + U * far.abs()
        rows = rows + kl_coef * (torch.expm1(far) - far)
        g = g - kl_coef * torch.expm1(far)
        t_rows = t_rows + abs(kl_coef) * (torch.expm1(far).abs() * (t_far + 8 * U) + 4 * U * far.abs())
        t_g = t_g + abs(kl_coef) * (far.exp() * t_far + 8 * U * torch.expm1(far).abs())
    rows = rows - entropy_coef * r["H"]
    t_rows = t_rows + abs(entropy_coef) * (r["t_H"] + 2 * U * r["H"].abs())
    rows, g = torch.where(live, rows, zero), torch.where(live, g, zero)
    t_rows = torch.where(live, t_rows.nan_to_num(0.0) + 4 * U * rows.abs().nan_to_num(0.0) + LEAST[torch.float32], zero)
    weighted = torch.where(live, w * rows, zero)
    loss = scale * weighted.sum()
    t_loss = abs(scale) * (w.abs() * t_rows).sum() + U * loss.abs() + LEAST[torch.float32]
    grad, t_grad = grad64(r, g, t_g.nan_to_num(0.0), scale * w / temperature, x.dtype, entropy_coef)
    return {"loss": (loss, t_loss), "loss_rows": (rows, t_rows), "logp": (r["logp"], r["t_logp"]),
            "entropy": (r["H"], r["t_H"]), "grad": (grad, t_grad)}


def preference64(x, labels, offsets, scale, ref=None, weights=None, kind="sigmoid", beta=0.1, label_smoothing=0.0,
                 margin=0.0, average=False, temperature=1.0):
    """{name: (value, bound)} of loss, loss_pairs, seq_logp, logp, grad; `offsets` a list."""
    R, P = x.shape[0], len(offsets) // 2
    w, live = live_rows(weights, R, x.device)
    seq_of = torch.full((R,), -1, dtype=torch.int64, device=x.device)
    for s, (a, b) in enumerate(zip(offsets, offsets[1:])):
        seq_of[a:b] = s
    live = live & (seq_of >= 0)
    x = torch.where(live[:, None], x, torch.zeros_like(x))
    labels = torch.where(live, labels, 0)
    r = rows64(x, labels, live, temperature)
    zero = torch.zeros_like(w)
    w = torch.where(live, w, zero)
    wl, t_wl = torch.where(live, w * r["logp"], zero), w.abs() * r["t_logp"]
    seg = lambda v: torch.stack([v[a:b].sum() for a, b in zip(offsets, offsets[1:])]) if P else v[:0]  # noqa: E731
    L, t_L, count = seg(wl), seg(t_wl), seg(w)
    per = torch.where(count != 0, 1 / count, 0.0) if average else torch.ones_like(count)
    L, t_L = L * per, t_L * per.abs()
    h, t_h = L[:P] - L[P:], t_L[:P] + t_L[P:]
    if ref is not None:
        h = h - (ref[:P].double() - ref[P:].double())
    if kind == "squared":
        off = h - margin - 0.5 / beta
        pairs, dh = off * off, 2 * off
        t_pairs, t_dh = 2 * off.abs() * t_h + t_h * t_h, 2 * t_h
    else:
        z = beta * h - margin
        t_z = beta * t_h + U * z.abs()
        if kind == "hinge":
            pairs = torch.where(z < 1, 1 - z, torch.where(torch.isnan(z), z, 0.0))
            dh = torch.where(z < 1, -beta, torch.where(torch.isnan(z), z, 0.0))
            t_pairs, t_dh = t_z, t_z * 0
        else:
            eps = label_smoothing
            sp = lambda v: torch.clamp(v, min=0) + torch.log1p((-v.abs()).exp())  # noqa: E731
            sg = torch.sigmoid
            pairs = (1 - eps) * sp(-z) + (eps * sp(z) if eps else 0.0)
            dh = beta * (eps * sg(z) - (1 - eps) * sg(-z))
            t_pairs = t_z + 8 * U * pairs
            # sigma' <= sigma(z) sigma(-z)
            t_dh = beta * ((t_z + 12 * U) * (eps * sg(z) + (1 - eps) * sg(-z)))
    least = LEAST[torch.float32]
    t_pairs = t_pairs.nan_to_num(0.0, posinf=0.0) + 2 * U * pairs.abs().nan_to_num(0.0, posinf=0.0) + least
    t_dh = t_dh.nan_to_num(0.0, posinf=0.0) + 2 * U * dh.abs().nan_to_num(0.0, posinf=0.0)
    loss = scale * pairs.sum()
    t_loss = abs(scale) * t_pairs.sum() + U * loss.abs().nan_to_num(0.0, posinf=0.0) + least
    sign = torch.cat([dh, -dh]) * per
    t_sign = torch.cat([t_dh, t_dh]) * per.abs()
    inside = seq_of.clamp(min=0)
    g = torch.where(live, sign[inside], zero) if P else zero
    t_g = torch.where(live, t_sign[inside] + 4 * U * g.abs(), zero) if P else zero
    grad, t_grad = grad64(r, g, t_g.nan_to_num(0.0), scale * w / temperature, x.dtype)
    t_seq = t_L.nan_to_num(0.0) + 2 * U * L.abs().nan_to_num(0.0, neginf=0.0, posinf=0.0) + least
    return {"loss": (loss, t_loss), "loss_pairs": (pairs, t_pairs), "seq_logp": (L, t_seq),
            "logp": (r["logp"], r["t_logp"]), "grad": (grad, t_grad)}


def logp64(x, labels, weights=None, temperature=1.0):
    w, live = live_rows(weights, x.shape[0], x.device)
    x = torch.where(live[:, None], x, torch.zeros_like(x))
    r = rows64(x, torch.where(live, labels, 0), live, temperature)
    return {"logp": (r["logp"], r["t_logp"]), "entropy": (r["H"], r["t_H"])}


def assert_near(got, want, what):
    """Every element of `got` within its bound; NaN where NaN, infinities equal."""
    value, bound = want
    got = got.double()
    assert got.shape == value.shape, f"{what}: shape {tuple(got.shape)} != {tuple(value.shape)}"
    bad = torch.isnan(got) != torch.isnan(value)
    inf = torch.isinf(value) | torch.isinf(got)
    bad |= inf & (got != value) & ~torch.isnan(value)
    off = torch.where(inf | torch.isnan(value), 0.0, (got - value).abs())
    bad |= off > bound
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside their bound; first at {i}: got "
                             f"{float(got[i])!r}, want {float(value[i])!r} +- {float(torch.as_tensor(bound).expand_as(value)[i])!r}")
