"""Eviction by accumulated weight on the host, from its definition: plain lists, one (sequence, kv head) at a time."""
import numpy as np


def order(scores, pos, L, seen, n_sink, n_recent):
    """The slots [0, L) from the first to be kept to the last: protected ones by slot, then by descending score (NaN
    last, -0.0 as 0.0), equal ones by slot."""
    def key(i):
        if pos[i] < n_sink or pos[i] >= seen - n_recent:
            return (0, 0.0, i)
        s = float(scores[i])
        return (2, 0.0, i) if s != s else (1, -s + 0.0, i)
    return sorted(range(L), key=key)


def evict(k, v, bt, lens, scores, slot_pos, dropped, n_sink, k_top, n_recent, trigger, stack=None):
    """All arrays as numpy; pools [NB, Hkv, 16, ...] of any type (a list of them in `k` and `v`'s place is fine too).
    Returns copies after the call: (pools, lens, scores, slot_pos, dropped, stack)."""
    pools = [p.copy() for p in list(k) + list(v)]
    lens, scores, slot_pos, dropped = lens.copy(), scores.copy(), slot_pos.copy(), dropped.copy()
    budget = n_sink + k_top + n_recent
    stack = None if stack is None else list(stack)
    for b, L in enumerate(lens.tolist()):
        if L <= max(trigger, budget):
            continue
        seen = L + int(dropped[b])
        for g in range(scores.shape[1]):
            pos = [int(p) if p >= 0 else i + int(dropped[b]) for i, p in enumerate(slot_pos[b, g, :L])]
            keep = set(order(scores[b, g], pos, L, seen, n_sink, n_recent)[:budget])
            holes = [i for i in range(budget) if i not in keep]
            moved = [i for i in range(budget, L) if i in keep]
            assert len(holes) == len(moved)
            slot_pos[b, g, :budget] = pos[:budget]
            for to, at in zip(holes, moved):
                for p in pools:
                    p[bt[b, to // 16], g, to % 16] = p[bt[b, at // 16], g, at % 16]
                scores[b, g, to] = scores[b, g, at]
                slot_pos[b, g, to] = pos[at]
            scores[b, g, budget:L] = 0
            slot_pos[b, g, budget:L] = -1
        if stack is not None:
            stack += [int(x) for x in bt[b, (budget + 15) // 16:(L + 15) // 16]]
        dropped[b] += L - budget
        lens[b] = budget
    return pools, lens, scores, slot_pos, dropped, stack
