"""The rows' side of an eviction in its forms, against the exact host model: both head sizes of both pool types where kept rows
lie close (tables of up to four budgets), a few (sequence, kv head) pairs whose moves many CTAs share, and as many pairs as leave
one CTA to each, whose warps copy more than one batch of moves."""
import numpy as np
import pytest

import test_gpu_evict as evict

RULES = (4, 512, 1024)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_prompts_cut_to_half_and_steady_states(d, q8, inplace):
    s = evict._state([2900, 1540, 1541, 2011], 3, d, 182, 41, q8=q8)
    assert s["bt"].shape[1] * 16 <= 4 * sum(RULES)
    evict._check(s, evict._call(s, *RULES, inplace=inplace), *RULES, inplace=inplace)
    s = evict._state([1800, 1796, 1700], 3, d, 113, 42, q8=q8, dropped=[300, 5, 1], budget=sum(RULES), scores="few")
    evict._check(s, evict._call(s, *RULES, trigger=1795, inplace=inplace), *RULES, trigger=1795, inplace=inplace)


# a CTA's eight warps take 4096 bytes of K and of V a turn each, of rows of d elements: 64 to 256 moves
@pytest.mark.gpu
@pytest.mark.parametrize("q8,d,rules,most", [
    (False, 128, (4, 6, 78), 170),
    (False, 64, (4, 6, 150), 318),
    (True, 128, (4, 6, 150), 318),
    (True, 64, (4, 6, 290), 596),
])
def test_more_moves_than_a_turn(q8, d, rules, most):
    """2449 pairs: more than sixteen for each of 152 SMs."""
    lens = np.random.default_rng(43).integers(most - 9, most + 1, 31)
    s = evict._state(lens.tolist(), 79, d, (most + 15) // 16, 43, q8=q8)
    assert s["bt"].shape[1] * 16 <= 4 * sum(rules)
    # the recent window lies past the budget and fills what is evicted below it, more than a turn's moves
    turn = 8 * 4 * 32 * 16 // (d if q8 else 2 * d)
    assert min(sum(rules), most - 9 - sum(rules)) > turn and rules[2] - 9 > turn
    evict._check(s, evict._call(s, *rules), *rules)
