"""Where a drawn column may lie, to the additions that a drawn column really
waits for. Works on any device.

The weights of the columns drawn from are e_j = 2^y_j, y_j <= 0 the exponent
beside the largest of them. Rounding in U = 2^-24 as in objectives_ref.py:

  a step's sum   a column's weight is formed beside its lane's largest, raised
                 once more by each end of the row (a column each), then to its
                 warp's largest and to the row's: 3 U |y_j| over all of them,
                 since their exponents add up to y_j, and five times 4 U of ex2
                 and U of the product, 24 U with the last product exact. At most
                 32 pairs are added in a lane, the pair's two, the two ends and 5
                 levels of the warp, 41 U
  a step's draw  weights anew, (3 |y_j| + 4) U, and at most 10 additions
  segments       held as whole numbers of 2^-36 of the largest weight, rounded
                 down: one for each step, and 256 vectors or 8 warps, 32 lanes and
                 8 columns of the step that is drawn from

and nothing else depends on the row's length. The number's place u S is off by
the error of S, the token's borders by those of the columns before it, and
inside its step, which lies within a step's columns to either side, by that
step's second look. A row's sum s, which only max(0, p - q) takes, adds the
steps of a lane of one warp, and 5 levels.
"""
import math

import torch

from choices_ref import held
from objectives_ref import U

STEP = 32 * 8 * 16  # bytes of a row that a step holds


def steps_of(vocab, size):
    n = 16 // size
    return -(-((vocab + 2 * n - 2) // n) // 256)


def exponents(x, T, leave=None):
    """Base 2, beside the largest; column `leave` is not drawn from."""
    z = x.double() / float(torch.tensor(T, dtype=torch.float32))
    if leave is not None:
        z[leave] = -math.inf
    return (z - z.max()) * 1.4426950408889634


def _least(vocab, size):
    return (2 * steps_of(vocab, size) + 300) * 2.0 ** -36


def check_place(w, error, again, least, u, token, size, what):
    """`token` may be drawn by u from weights w: the columns' errors in the steps' sums `error`, in the draw from
    a step `again`, and of the whole `least`. Returns how far off its share the number lies, over the weights' sum."""
    assert 0 <= token < len(w) and float(w[token]) > 0, (what, token)
    upto, wrong = w.cumsum(0), error.cumsum(0)
    end = float(upto[token])
    start, at = end - float(w[token]), held(u) * float(upto[-1])
    near = again[max(0, token - STEP // size):token + STEP // size].sum()
    bound = held(u) * float(wrong[-1]) + float(wrong[token]) + float(near) + least
    off = max(0.0, start - at, at - end)
    assert off <= bound, (what, token, start, at, end, bound)
    return off / float(upto[-1])


def check_own(x, T, u, token, leave=None, what=None):
    """A token drawn from a row's softmax, or from what is left of it without the column `leave`."""
    y = exponents(x, T, leave)
    e = torch.exp2(y)
    y = y.clamp(min=-200).abs()
    size = x.element_size()
    return check_place(e, e * (3 * y + 65) * U, e * (3 * y + 14) * U, _least(len(x), size), u, token, size, what)


def softmax_error(x, T):
    """p and its error as max(0, p - q) takes it: 2^(y_j - log2 s), the exponent's sum rounded by U of its own and
    log2 s by 2 U of its value and by the error of s."""
    y = exponents(x, T)
    e = torch.exp2(y)
    s = float(e.sum())
    y = y.clamp(min=-200).abs()
    lane = -(-steps_of(len(x), x.element_size()) // 32)
    of_s = float((e * (3 * y + 65 + 5)).sum()) / s + lane + 5
    p = e / s
    return p, p * (4 * y + 4 + 3 * math.log2(s) + of_s) * U


def check_rest(x, draft, T, u, token, what=None):
    """A token drawn from max(0, p - q). Its sums: 20 additions in a half step, 10 in the draw."""
    p, ep = softmax_error(x, T)
    q, eq = softmax_error(draft, T)
    w, error = (p - q).clamp(min=0), ep + eq + U * (p + q)
    size = x.element_size()
    if float(w.sum()) <= float(error.sum()):  # what is left is rounding
        assert 0 <= token < len(x) and float(p[token]) > 0, (what, token)
        return None
    # a column that has nothing left may be drawn where rounding leaves it something
    shown = torch.where(w > 0, w, torch.where(error > 0, 1e-300, 0.0))
    return check_place(shown, error + 20 * U * w, error + 10 * U * w, _least(len(x), size) * 2.0 ** -20, u, token, size, what)
