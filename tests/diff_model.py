"""Differential attention in 64 bits, from the definition, one query row at a time over contiguous keys; and the
bounds that a kernel's outputs are held to."""
import numpy as np

import rules_model


def weights(q, k, i, scale, window=0, softcap=0.0, slope=0.0, doc_start=0, prefix=0):
    """The softmax weights of one map over k [L, d] (zeros for unseen keys; all zeros where none is seen)."""
    L = k.shape[0]
    t = np.arange(L)
    lo = max(0, doc_start, i - window + 1 if window > 0 else 0)
    see = ((t >= lo) & (t <= i)) | (t < min(max(prefix, 0), L))
    p = np.zeros(L)
    if see.any():
        x = scale * (k[see] @ q)
        if softcap > 0:
            x = softcap * np.tanh(x / softcap)
        x = x - slope * np.abs(i - t[see])
        w = np.exp(x - x.max())
        p[see] = w / w.sum()
    return p


def row(q, k, v, i, scale, lam, norm_weight, norm_eps, weight_eps, **rules):
    """Output [d] of a query q [d] (both halves) and the error that it may have.  The error of y = o_1 - lam o_2 is that
    of each map's quotient (rules_model.bound without its output rounding) and the fp32 difference; a norm r = (mean
    y^2 + eps)^-1/2 then lies between its values for the largest and the least sum of squares; the output is rounded
    by at most half a bf16 step."""
    d = q.shape[0]
    half = d // 2
    y, err = 0.0, 0.0
    for m in range(2):
        at = slice(m * half, (m + 1) * half)
        o, mass, size = rules_model.row(q[at], k[:, at], v, i, scale, **rules)
        e = rules_model.bound(np.zeros(d), mass, size, half, weight_eps)
        f = 1.0 if m == 0 else -lam
        y = y + f * o
        err = err + abs(f) * (e + 4 * 2.0 ** -24 * np.abs(o))
    if norm_weight is None:
        out, far = y, err
    else:
        s, more = np.mean(y * y), np.mean(2 * np.abs(y) * err + err * err)
        r, up, down = ((x + norm_eps) ** -0.5 for x in (s, max(s - more, 0.0), s + more))
        out = y * r * norm_weight
        far = np.abs(norm_weight) * np.maximum((np.abs(y) + err) * up - np.abs(y) * r, np.abs(y) * r - (np.abs(y) - err) * down)
        far = far + np.abs(out) * (d + 16) * 2.0 ** -24
    return out, (np.abs(out) + far) * 2.0 ** -8 + far + 1e-37


def score(qs, k, i, scale, lams, rules):
    """Sum over the group's query heads of |a_1 - lam a_2| for each key, and the error that it may have; `rules` has a dict a
    head.  A weight is off by what its logit is, twice (itself and the sum), as in rules_model.bound."""
    half = k.shape[1] // 2
    total, err = np.zeros(k.shape[0]), np.zeros(k.shape[0])
    for q, lam, r in zip(qs, lams, rules):
        w = 0.0
        for m in range(2):
            at = slice(m * half, (m + 1) * half)
            p = weights(q[at], k[:, at], i, scale, **r)
            size = max(1.0, float((abs(scale) * (np.abs(k[:, at]) @ np.abs(q[at]))).max(initial=0.0)),
                       abs(r.get("slope", 0.0)) * k.shape[0])
            f = 1.0 if m == 0 else -lam
            w = w + f * p
            err += abs(f) * p * 2.1 * ((half + 16) * 2.0 ** -24 * size + 2.0 ** -20)
        total += np.abs(w)
    return total, err + total * 8 * 2.0 ** -24
