"""Attention with score rules in 64 bits, from the definition, one query row at a time over contiguous
keys; and the bound that a kernel's bf16 output is held to."""
import numpy as np


def row(q, k, v, i, scale, window=0, softcap=0.0, slope=0.0, doc_start=0, prefix=0):
    """Output [d] of a query at position i over k, v [L, d] (float64), its sum of p |v| (the size that
    errors of the weights scale with) and the largest |scale q k| sum of its keys."""
    L = k.shape[0]
    t = np.arange(L)
    lo = max(0, doc_start, i - window + 1 if window > 0 else 0)
    see = ((t >= lo) & (t <= i)) | (t < min(max(prefix, 0), L))
    if not see.any():
        return np.zeros(v.shape[1]), np.zeros(v.shape[1]), 0.0
    k, v, t = k[see], v[see], t[see]
    x = scale * (k @ q)
    size = float((abs(scale) * (np.abs(k) @ np.abs(q))).max())
    if softcap > 0:
        x = softcap * np.tanh(x / softcap)
    x = x - slope * np.abs(i - t)
    p = np.exp(x - x.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v), max(size, float(np.abs(x).max()))


def bound(ref, mass, size, d, weight_eps):
    """Half a bf16 step of the value, plus what weights off by e carry into the quotient (twice e, once in
    the sum of p v and once in the sum of p): e is the weights' own rounding (`weight_eps`) and the
    logits' fp32 error, d + 16 roundings of sums and products no larger than `size`; 2^-20 for the
    hardware's power of two (2^-22 relative) over sums in another order."""
    e = weight_eps + (d + 16) * 2.0 ** -24 * max(size, 1.0) + 2.0 ** -20
    return np.abs(ref) * 2.0 ** -8 + 2.1 * e * mass + 1e-37
