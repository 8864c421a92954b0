"""The choices made from a row's softmax in 64 bits, from their definitions
(include/ce_rows.h): what a given output must satisfy. Works on any device.

A drawn column is right where the number that drew it lies in the column's
share of the row, widened by the rounding of the border; an accepted draft
where a q < p, to the rounding of the two; a choice of experts where it is
sorted and complete to the rounding of the scores.

Rounding, counted in U = 2^-24 as in objectives_ref.py. A weight
exp((x - m) / T) carries (3 |y| + 4) U of its value, y = (x - m) / T log2(e),
and U of it more for every addition on its way into a running sum (at most
ADDS), so the sum of a row's first weights is off by at most
    border = sum_j e_j (3 |y_j| + 4 + ADDS) U
and the target u S by as much again; the fixed point numbers that the sums are
held in add 2^-36 for each of a row's at most 16 * 4 * 33 * 3 segments, less
than U of the largest weight, which is 1.
"""
import math

import torch

from objectives_ref import U, depth


def adds(vocab):
    """Additions on the way of a weight: a lane's chain (at most the row / 32 / 2
    pairs' sums of one CTA's warp; lanes' runs are shorter), then the joins."""
    return vocab / 32 + 64


def softmax64(x, t):
    """p and the bound of its error, beside the row's weights' border error (per row, relative to S)."""
    z = x.double() / t
    d = z - z.max()
    e = d.exp()
    y = d.clamp(min=-200).abs() * 1.4426950408889634
    S = e.sum()
    p = e / S
    border = float((e * (3 * y + 4 + adds(len(x)))).sum() * U / S) + float(U / S)
    each = (3 * y + 4 + 6 + depth(len(x))) * U * p  # its own rounding and the sum's
    return p, each, border


COLDEST = float(torch.tensor(1e-6))  # as a temperature tensor holds it


def good_temperature(t):
    return t == 0 or COLDEST <= t <= 1e6


def is_distribution(x):
    return bool(torch.isfinite(x.max())) and not bool(torch.isnan(x).any())


def held(u):
    return 0.0 if math.isnan(u) else min(max(u, 0.0), 1 - 2.0 ** -24)


def check_drawn(w, error, border, u, token, what):
    """`token` may be drawn by u from the weights w >= 0 (their errors `error`), borders off by `border`."""
    assert 0 <= token < len(w), (what, token)
    assert float(w[token] + error[token]) > 0, (what, token, "has no weight")
    total = float(w.sum())
    end = float(w[:token + 1].sum())
    start = end - float(w[token])
    at = held(u) * total
    assert start - 2 * border <= at <= end + 2 * border, (what, token, start, at, end, border)


def check_sampled(x, u, T, token, logp, what):
    """One row of sample_rows: x its columns, logp None if not asked for."""
    if not good_temperature(T) or not is_distribution(x):
        assert token == -1, (what, token)
        assert logp is None or math.isnan(logp), (what, logp)
        return
    if T == 0:
        assert token == int((x == x.max()).nonzero()[0]), (what, token)
        assert logp is None or logp == 0, (what, logp)
        return
    p, each, border = softmax64(x, T)
    check_drawn(p, each, border, u, token, what)
    check_logp(x, T, token, logp, what)


def check_logp(x, T, token, logp, what):
    if logp is None:
        return
    z = x.double() / T
    d = z - z.max()
    log_s = float(d.exp().sum().log())
    want = float(d[token]) - log_s
    bound = (6 + depth(len(x))) * U + 2 * U * log_s + 4 * U * abs(float(d[token])) + U * abs(want) + 2 * U
    assert abs(logp - want) <= bound, (what, token, logp, want, bound)


def check_verified(logits, drafts, offsets, uniforms, draft_logits, temperatures, accepted, tokens, logp):
    """verify_drafts on the whole: lists or CPU tensors; a list of how each row ended (for the tests' own use)."""
    rows, V = logits.shape
    offsets, drafts = [int(v) for v in offsets], [int(v) for v in drafts]
    seen = [False] * rows
    ends = []
    for s, (a, b) in enumerate(zip(offsets, offsets[1:])):
        n, stopped = int(accepted[s]), False
        assert 0 <= n <= b - a, (s, n)
        for r in range(a, b):
            seen[r] = True
            what, x, T, d = (s, r), logits[r], float(temperatures[r]), drafts[r]
            token, lp = int(tokens[r]), None if logp is None else float(logp[r])
            if stopped:
                assert token == -1 and (lp is None or lp == 0), what
                continue
            took = r - a < n
            stopped = not took
            if not good_temperature(T) or not is_distribution(x):
                assert not took and token == -1 and (lp is None or math.isnan(lp)), what
                ends.append("bad")
                continue
            has = 0 <= d < V
            if T == 0:
                top = int((x == x.max()).nonzero()[0])
                assert token == top and took == (has and d == top), what
                assert lp is None or lp == 0, what
                ends.append("greedy")
                continue
            p, each, border = softmax64(x, T)
            w, error = p, each
            if has:
                q, q_each, q_border = torch.zeros_like(p), torch.zeros_like(p), 0.0
                q[d] = 1.0
                drawn = True
                if draft_logits is not None:
                    drawn = is_distribution(draft_logits[r])
                    if drawn:
                        q, q_each, q_border = softmax64(draft_logits[r], T)
                side = float(uniforms[r][0]) * float(q[d]) - float(p[d])
                slack = abs(float(uniforms[r][0])) * float(q_each[d]) + float(each[d]) + 4 * U * float(p[d])
                if not drawn or float(p[d]) == 0:
                    assert not took, what
                elif abs(side) > slack:
                    assert took == (side < 0), (what, side)
                if took:
                    assert token == d, what
                    check_logp(x, T, token, lp, what)
                    ends.append("accepted")
                    continue
                if drawn:
                    # p - q: both errors, the sums over the row twice
                    w, error = (p - q).clamp(min=0), each + q_each + U * (p + q)
                    border = float((each + q_each + adds(V) * U * (p + q)).sum()) + 2.0 ** -40
                    if draft_logits is None:
                        border = 2 * border  # the drafted column is left out of a sum that held it
                    if float(w.sum()) <= 2 * border:  # nothing left to the rounding: from p, or what rounding left
                        assert 0 <= token < V and float(p[token]) > 0, what
                        ends.append("nothing left")
                        continue
            check_drawn(w, error, border, float(uniforms[r][1]), token, what)
            check_logp(x, T, token, lp, what)
            ends.append("rest" if w is not p else "drawn")
        if not stopped:
            assert n == b - a
    for r in range(rows):
        if not seen[r]:
            assert int(tokens[r]) == -1 and (logp is None or float(logp[r]) == 0), r
    return ends


# -- routing ----------------------------------------------------------------------

def scores64(x, score):
    """Scores and the bounds of their errors. sigmoid: e^-z by base 2, its exponent's product and constant
    rounded (2 U |z| of e^-z, of which the score has its part 1 - s), ex2 (4 U), a sum, a reciprocal (2 U);
    softmax, (3 |y| + 4) U, the sum's (6 + 32 + 5) U, a reciprocal and the product."""
    z = x.double()
    if score == "sigmoid":
        s = torch.sigmoid(z)
        return s, s * (8 + 2 * z.clamp(-1e4, 1e4).abs() * (1 - s)) * U
    d = z - z.amax(1, keepdim=True)
    s = torch.softmax(z, 1)
    y = d.clamp(min=-200).abs() * 1.4426950408889634
    return s, s * (3 * y + 52) * U


def check_routed(x, k, chosen, gates, counts, score="softmax", bias=None, groups=1, top_groups=None, group_top=2,
                 renormalise=True, scale=1.0, weights=None):
    """All rows of route_rows; CPU tensors. Every row's choice is sorted, complete and of kept groups to the
    rounding of what it goes by, its equals in order of their columns, its gates right."""
    rows, E = x.shape
    top_groups = groups if top_groups is None else top_groups
    s, es = scores64(x, score)
    by = s if bias is None else s + bias.double()
    eby = es if bias is None else es + U * by.abs()
    out = (x == -math.inf) | torch.isnan(by) | (by == -math.inf)
    per = E // groups
    tally = torch.zeros(E, dtype=torch.int64)
    for r in range(rows):
        c, g = [int(v) for v in chosen[r]], gates[r].double()
        if weights is not None and float(weights[r]) == 0:
            assert c == [-1] * k and float(g.abs().sum()) == 0, r
            continue
        if bool(torch.isnan(x[r]).any()) or float(x[r].max()) == math.inf:
            assert c == [-1] * k and bool(torch.isnan(g).all()), r
            continue
        ok = ~out[r]
        real = [e for e in c if e >= 0]
        assert c == real + [-1] * (k - len(real)) and len(set(real)) == len(real), (r, c)
        assert all(bool(ok[e]) for e in real), (r, c)
        # where the choice goes by the logits (no bias) it is exact
        key, ekey = (by[r], eby[r]) if bias is not None else (x[r].double(), torch.zeros(E, dtype=torch.float64))
        # equals in all that they go by keep the order of their columns; others may be within a rounding
        near = lambda i, j: float(x[r, i]) != float(x[r, j]) or (bias is not None and float(bias[i]) != float(bias[j]))  # noqa: E731
        allowed = torch.ones(E, dtype=torch.bool)
        if top_groups < groups:
            sums, errors = [], []
            for i in range(groups):
                v = [(float(by[r, j]), float(eby[r, j])) for j in range(i * per, (i + 1) * per) if bool(ok[j])]
                v.sort(reverse=True)
                v = v[:group_top]
                sums.append(sum(a for a, _ in v) if v else -math.inf)
                errors.append(sum(b for _, b in v) + U * abs(sums[-1]) if v else 0.0)
            order = sorted(range(groups), key=lambda i: (-sums[i], i))
            kept, edge = order[:top_groups], order[top_groups:]
            clear = all(sums[a] - errors[a] > sums[b] + errors[b] or (sums[a] == sums[b] and errors[a] == 0)
                        or (sums[a] == sums[b] and _same_members(x[r], a, b, per))
                        for a in kept for b in edge)
            if not clear:
                continue  # the groups may change places, and with them everything else
            for i in edge:
                allowed[i * per:(i + 1) * per] = False
        live = allowed & ok
        assert all(bool(live[e]) for e in real), (r, c, "not of a kept group")
        assert len(real) == min(k, int(live.sum())), (r, c)
        for a, b in zip(real, real[1:]):
            gap = float(key[a] - key[b])
            assert gap > 0 or (gap == 0 and a < b) or (near(a, b) and -gap <= float(ekey[a] + ekey[b])), (r, a, b, gap)
        if real:
            last = real[-1]
            rest = live.clone()
            rest[real] = False
            for e in rest.nonzero()[:, 0].tolist():
                gap = float(key[last] - key[e])
                assert gap > 0 or (gap == 0 and last < e) or (near(last, e) and -gap <= float(ekey[last] + ekey[e])), \
                    (r, last, e, gap)
        # gates: a score (es), or its part of the chosen's sum (es of both, 5 levels of a sum, a division)
        want, err = gates64(x[r], real, score, renormalise)
        want, err = want * scale, err * abs(scale) + (want * scale).abs() * 2 * U + 2.0 ** -126 * (1 + abs(scale))
        assert bool(((g[:len(real)] - want).abs() <= err).all()), (r, g, want)
        assert float(g[len(real):].abs().sum()) == 0, r
        tally[real] += 1
    if counts is not None:
        taken = chosen[chosen >= 0]
        assert torch.equal(counts, torch.bincount(taken.flatten(), minlength=E)), "counts of the choice returned"
    return tally


def _same_members(x, a, b, per):
    return torch.equal(x[a * per:(a + 1) * per].sort()[0], x[b * per:(b + 1) * per].sort()[0])


def gates64(x, chosen, score, renormalise):
    """Gates of one row (scale 1) and their error bounds."""
    z = x.double()
    s, es = scores64(x[None], score)
    s, es = s[0][chosen], es[0][chosen]
    if not renormalise or not chosen:
        return s, es
    # exp(z - top) by base 2: 2 U |z - top| for the exponent's roundings and U |z - top| for the difference's, ex2
    # 4 U; 1 / (1 + e^-|z|): at most 7 U, since |z| e^-|z| < 1; the sum's 5 levels and a division
    zc = z[chosen]
    ls = torch.nn.functional.logsigmoid(zc) if score == "sigmoid" else zc
    f = torch.softmax(ls, 0)
    d = (zc - zc.max()).clamp(min=-200).abs()
    rel = (3 * d + 20) * U
    return f, f * (rel + (f * rel).sum() + 8 * U)


def route_grad64(x, chosen, gates_grad, score="softmax", renormalise=True, scale=1.0, weights=None):
    """The gradient in f64 by the formulas, and a bound of its error before the last rounding."""
    rows, E = x.shape
    grad = torch.zeros(rows, E, dtype=torch.float64)
    err = torch.zeros(rows, E, dtype=torch.float64)
    for r in range(rows):
        if weights is not None and float(weights[r]) == 0:
            continue
        at = [(int(c), i) for i, c in enumerate(chosen[r]) if 0 <= int(c) < E]
        if not at:
            continue
        cols = [c for c, _ in at]
        G = gates_grad[r].double()[[i for _, i in at]] * scale
        eG = G.abs() * U
        s, es = scores64(x[r][None], score)
        sc, esc, zc = s[0][cols], es[0][cols], x[r].double()[cols].clamp(-1e4, 1e4)
        if renormalise:
            f, ef = gates64(x[r], cols, score, True)
            D = (f * G).sum()
            eD = (ef * G.abs() + f * eG + 6 * U * f * G.abs()).sum()
            v = f * (G - D)
            ev = ef * (G - D).abs() + f * (eG + eD + U * (G - D).abs()) + 2 * U * v.abs()
            if score == "sigmoid":
                ev = ev * (1 - sc) + v.abs() * (1 - sc) * (10 + 2 * zc.abs()) * U
                v = v * (1 - sc)
        elif score == "sigmoid":
            v = sc * (1 - sc) * G
            ev = v.abs() * (20 + 4 * zc.abs()) * U
        else:
            v = sc * G
            ev = esc * G.abs() + sc * eG + 2 * U * v.abs()
            D = v.sum()
            eD = ev.sum() + 6 * U * v.abs().sum()
            grad[r] -= s[0] * D
            err[r] += es[0] * D.abs() + s[0] * eD + 3 * U * s[0] * D.abs()
        for i, c in enumerate(cols):
            grad[r, c] += v[i]
            err[r, c] += ev[i] + 2 * U * (v[i].abs() + grad[r, c].abs())
    return grad, err + 2.0 ** -126
