"""Host model of the FP8 cache with one scale per (block, kv head): the E4M3 grid, the scale rule and
the append, in 64 bits, from their definitions."""
import numpy as np

MIN_EXP, MAX_EXP = -120, 119


def round_e4m3(x):
    """The E4M3 value nearest to each x (ties to the even code), saturated at 448, in float64."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    with np.errstate(divide="ignore"):
        e = np.maximum(np.floor(np.log2(np.where(a > 0, a, 1.0))), -6)
    step = np.exp2(e - 3)  # a / step <= 16; np.rint rounds ties to even
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), x)


def needed_scale(amax):
    e = MIN_EXP
    while e < MAX_EXP and amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(codes, scales, rows, slots):
    """codes [NB, Hkv, 16, d] values, scales [NB, Hkv], rows [T, Hkv, d], valid slots: copies after the append."""
    codes, scales = codes.astype(np.float64).copy(), scales.astype(np.float64).copy()
    by_block = {}
    for i, s in enumerate(slots):
        if s >= 0:
            by_block.setdefault(int(s) // 16, []).append((i, int(s) % 16))
    for blk, items in by_block.items():
        offs = [o for _, o in items]
        for g in range(codes.shape[1]):
            need = needed_scale(max(np.abs(rows[i, g]).max() for i, _ in items))
            old = scales[blk, g]
            new = need if 0 in offs else max(old, need)
            if 0 not in offs and new != old:
                for o in range(16):
                    if o not in offs:
                        codes[blk, g, o] = round_e4m3(codes[blk, g, o] * (old / new))
            for i, o in items:
                codes[blk, g, o] = round_e4m3(rows[i, g] / new)
            scales[blk, g] = new
    return codes, scales
