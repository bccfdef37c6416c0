"""Differential attention where a sum or a parameter is no number: a NaN or an infinite logit in one map of a key that the
query sees reaches the scores of every key of its heads, and no others; a row that sees no key is zero whatever the norm's
weights and the factor."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
import test_gpu_diff_decode as decode
import test_gpu_diff_prefill as prefill
from paged_kv_cache_mapped_gb300 import header_constants

C = header_constants()
DEV = torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[9, 12, 16], [2500, 700, 1900]], ids=["whole rows", "rows in shares"])
@pytest.mark.parametrize("hq,d", [(4, 64), (8, 128), (12, 64), (10, 128)])
@pytest.mark.parametrize("half", [0, 1])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), "q"])
def test_a_sum_that_is_no_number_reaches_the_scores(lens, hq, d, half, bad):
    """Up to four heads a kv head (pairs) and five and six (wide).  A logit of NaN or +infinity in either map leaves no
    weight |a_1 - lambda a_2| of the keys that the row sees a number; keys that it does not see, the other kv head and the
    other sequences keep their values, bit for bit."""
    c = decode._case(lens, hq, 2, d, 31, fill=0.0)
    r = dict(window=300, prefix_lens=[3, 0, 20])
    g, at = hq // 2, d // 2 * half + 5
    c["q"][:, :, at] = 1.0
    before = torch.rand((3, 2, 2512), device=DEV)
    clean = before.clone()
    out = decode._call(c, scores=clean, **r)
    if bad == "q":
        c["q"][0, :g, at] = float("nan")
    else:
        t = lens[0] - 2
        c["pools"][0][int(c["bt"][0, t // 16]), 0, t % 16, at] = bad
    got, err = before.clone(), pkv.new_error_word(DEV)
    again = decode._call(c, scores=got, error_word=err, **r)
    assert pkv.read_error(err) == 0
    L = lens[0]
    t = torch.arange(2512, device=DEV)
    seen = (t < L) & ((t >= L - 300) | (t < 3))
    assert torch.isnan(got[0, 0, seen]).all()
    assert torch.equal(got[0, 0, ~seen], before[0, 0, ~seen])
    assert torch.equal(got[0, 1], clean[0, 1]) and torch.equal(got[1:], clean[1:])
    assert not torch.isfinite(again[0, :g].float()).any()
    assert torch.equal(again[0, g:], out[0, g:]) and torch.equal(again[1:], out[1:])


@pytest.mark.gpu
def test_eviction_reports_the_scores_that_are_no_numbers():
    """The weights of a step whose logits are no numbers, handed on: the eviction says so."""
    c = decode._case([90, 40], 4, 2, 64, 32, fill=0.0)
    c["pools"][0][int(c["bt"][0, 1]), 0, 3, 40] = float("nan")
    scores, pos = torch.zeros((2, 2, 96), device=DEV), torch.full((2, 2, 96), -1, dtype=torch.int32, device=DEV)
    decode._call(c, scores=scores)
    err = pkv.new_error_word(DEV)
    pkv.kv_evict(*c["pools"], c["bt"], torch.tensor(c["lens"], dtype=torch.int32, device=DEV), scores, pos,
                 torch.zeros(2, dtype=torch.int32, device=DEV), 2, 20, 10, error_word=err)
    assert pkv.read_error(err) == C["PKV_DEV_BAD_SCORE"]


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq", [4, 12], ids=["pairs", "wide"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_that_see_nothing_are_zero_whatever_the_norm(hq, d, bad):
    """A weight of the norm that is no number makes that column of the rows that see a key none, and no other; a
    factor that is no number besides leaves a row zero whose blocks are all outside the pool."""
    lens, docs = [300, 40, 0, 2500, 33], [0, 41, 0, 2500, 0]
    c = decode._case(lens, hq, 2, d, 33)
    want = decode._call(c, doc_starts=docs).float()
    c["w"][7] = bad
    got = decode._call(c, doc_starts=docs).float()
    others = [i for i in range(d) if i != 7]
    assert not got[1:4].any() and torch.equal(got[:, :, others], want[:, :, others])
    assert not torch.isfinite(got[[0, 4], :, 7]).any()
    c["lam"][:] = bad
    c["bt"][[0, 3]] = -1
    err = pkv.new_error_word(DEV)
    got = decode._call(c, error_word=err, doc_starts=[0, 41, 0, 0, 0]).float()
    assert pkv.read_error(err) == C["PKV_DEV_BAD_BLOCK_ID"]
    assert not got[:4].any() and not torch.isfinite(got[4]).any()
    # of many tokens: some rows of an item see nothing, all rows of one, and shares of keys
    for lens, new in (([100, 64], [100, 3]), ([3000, 700], [2, 200])):
        c = prefill._case(lens, new, hq, 2, d, 34)
        pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)])
        docs = np.where(np.arange(len(pos)) % 2 == 0, pos + 1, np.maximum(pos - 5, 0))
        want = prefill._call(c, doc_starts=docs).float()
        c["w"][7] = bad
        got = prefill._call(c, doc_starts=docs).float()
        assert not got[::2].any() and torch.equal(got[:, :, others], want[:, :, others])
        assert not torch.isfinite(got[1::2, :, 7]).any()
        assert not prefill._call(c, doc_starts=pos + 1).any()
        # NaN in V rows past every row's keys, in the blocks that they share, has rows computed again
        c["pools"][1][int(c["bt"][0, (lens[0] - 1) // 16]), :, (lens[0] - 1) % 16] = float("nan")
        last = new[0] - 1
        docs2 = np.where(np.arange(len(pos)) == last, pos + 1, docs)
        got = prefill._call(c, doc_starts=docs2).float()
        assert not got[::2].any() and not got[last].any()
