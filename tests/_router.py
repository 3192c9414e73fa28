"""The routing row by row in plain Python and 64 bits, from its definition.

Not collected by pytest (no test_ prefix). Shares no code with the library.
"""
import math

import numpy as np

MOST = float(np.finfo(np.float32).max)


def _counted(x):
    """A logit or bias as it counts: None leaves its expert out."""
    x = float(x)
    if math.isnan(x) or x == -math.inf:
        return None
    return min(x, MOST)


def _log_sigmoid(x):
    return -math.log1p(math.exp(-x)) if x >= 0 else x - math.log1p(math.exp(x))


def route_row(logits, bias, topk, sigmoid, groups, topk_groups, best, renormalize, scale):
    """(idx, weights) of one row, lists of topk."""
    n = len(logits)
    l = [_counted(x) for x in logits]
    there = [e for e in range(n) if l[e] is not None]
    s = {}
    if sigmoid:
        for e in there:
            s[e] = math.exp(_log_sigmoid(l[e]))
    elif there:
        m = max(l[e] for e in there)
        z = math.fsum(math.exp(l[e] - m) for e in there)
        for e in there:
            s[e] = math.exp(l[e] - m) / z
    if bias is None:
        value, order = dict(s), {e: l[e] for e in there}
    else:
        b = [_counted(x) for x in bias]
        value = {e: s[e] + b[e] for e in there if b[e] is not None}
        order = value
    if groups > 1:
        per = n // groups
        of = []
        for g in range(groups):
            # without a bias the order of single scores is that of the logits
            by = order if best == 1 else value
            v = sorted((by[e] for e in range(g * per, (g + 1) * per) if e in by), reverse=True)
            of.append(sum(v[:best]) if len(v) >= best else -math.inf)
        kept = sorted(range(groups), key=lambda g: (-of[g], g))[:topk_groups]
        order = {e: v for e, v in order.items() if e // per in kept}
    picks = sorted(order, key=lambda e: (-order[e], e))[:topk]
    if renormalize and picks:
        logs = [_log_sigmoid(l[e]) if sigmoid else l[e] for e in picks]
        top = max(logs)
        w = [math.exp(x - top) for x in logs]
        total = math.fsum(w)
        w = [x / total for x in w]
    else:
        w = [s[e] for e in picks]
    pad = topk - len(picks)
    return picks + [-1] * pad, [x * float(np.float32(scale)) for x in w] + [0.0] * pad


def check(got_idx, got_w, logits, bias, valid, topk, sigmoid, groups, topk_groups, best, renormalize, scale, what=""):
    """Picks equal; weights off by their own rounding to fp32 (half a step,
    2^-24, or half the smallest subnormal) and 64-bit arithmetic's: exp and
    the argument's difference to the largest, each some steps of 2^-53 of
    values up to 2^10 here, far below 2^-30 of the weight."""
    for t in range(len(logits)):
        if t < valid:
            idx, w = route_row(logits[t], bias, topk, sigmoid, groups, topk_groups, best, renormalize, scale)
        else:
            idx, w = [-1] * topk, [0.0] * topk
        assert got_idx[t].tolist() == idx, (what, t, got_idx[t].tolist(), idx)
        for g, x in zip(got_w[t].tolist(), w):
            assert abs(g - x) <= abs(x) * (2.0 ** -24 + 2.0 ** -30) + 2.0 ** -149, (what, t, g, x)
