"""The decode that emits scores (bf16 and INT8 pools) where a key's logit is no number, and where a block is outside the
pool: what the attended keys get, and that every other score stays."""
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
from helpers import paged_from_contiguous, rand_bf16, rand_code_pool
from paged_kv_cache_mapped_gb300 import header_constants

pytestmark = pytest.mark.gpu
C = header_constants()
DEV = torch.device("cuda:0")
LENS = {"whole rows": [9, 12, 16], "rows in shares": [2500, 700, 1900]}


def _case(lens, hq, d, q8, seed):
    g = torch.Generator().manual_seed(seed)
    k, v = (rand_bf16((len(lens), max(lens), 2, d), g) for _ in range(2))
    nb = sum((L + 15) // 16 for L in lens) + 3
    kc, vc, bt = paged_from_contiguous(k, v, lens, nb, g)
    pools = [kc.to(DEV), vc.to(DEV)]
    if q8:
        pools = [rand_code_pool((nb, 2, 16, d), g).to(DEV) for _ in range(2)]
        pools += [(torch.rand((nb, 2, 16), generator=g) * 0.02).to(DEV) for _ in range(2)]
    return dict(q=rand_bf16((len(lens), hq, d), g).to(DEV), pools=pools, bt=bt.to(DEV), scale=d ** -0.5,
                lens=torch.tensor(lens, dtype=torch.int32, device=DEV), q8=q8)


def _call(c, scores, logits, window=0, err=None):
    fn = pkv.paged_decode_attention_scores_q8 if c["q8"] else pkv.paged_decode_attention_scores
    return fn(c["q"], *c["pools"], c["bt"], c["lens"], c["scale"], scores, window, logits=logits, error_word=err)


@pytest.mark.parametrize("lens", LENS.values(), ids=LENS)
@pytest.mark.parametrize("hq,d,q8", [(2, 64, False), (8, 128, False), (16, 64, False), (8, 128, True)])
@pytest.mark.parametrize("where", ["k", "q"])
def test_a_sum_that_is_no_number_reaches_the_scores(lens, hq, d, q8, where):
    """Its log-sum-exp is NaN, not that of a row which attends to nothing, and so are the scores of the attended keys."""
    c = _case(lens, hq, d, q8, 41)
    g, window, L = hq // 2, 300, lens[0]
    before, logits = torch.rand((3, 2, 2512), device=DEV), torch.zeros((3, hq, 2512), device=DEV)
    clean = before.clone()
    out, lse = (t.clone() for t in _call(c, clean, logits, window))
    if where == "q":
        c["q"][0, :g, 5] = float("nan")
    else:
        t = L - 2
        blk = int(c["bt"][0, t // 16])
        (c["pools"][2][blk, 0] if q8 else c["pools"][0][blk, 0, :, 5])[t % 16] = float("nan")
    got, err = before.clone(), pkv.new_error_word(DEV)
    again, lse2 = _call(c, got, logits, window, err)
    assert pkv.read_error(err) == 0
    first = max(0, L - window)
    assert torch.isnan(lse2[0, :g]).all() and torch.isnan(again[0, :g].float()).all()
    assert torch.isnan(got[0, 0, first:L]).all()
    assert torch.equal(got[0, 0, :first], before[0, 0, :first]) and torch.equal(got[0, 0, L:], before[0, 0, L:])
    assert torch.equal(got[0, 1], clean[0, 1]) and torch.equal(got[1:], clean[1:])
    assert torch.equal(again[0, g:], out[0, g:]) and torch.equal(again[1:], out[1:])
    assert torch.equal(lse2[0, g:], lse[0, g:]) and torch.equal(lse2[1:], lse[1:])


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("window", [0, 250])
@pytest.mark.parametrize("stride", [320, 321])
def test_keys_of_a_bad_block_get_no_score(q8, window, stride):
    """Over the logits of another call, whose keys there had weights: those scores stay, bit for bit."""
    c = _case([300, 77], 8, 64, q8, 42)
    err = pkv.new_error_word(DEV)
    before, logits = torch.rand((2, 2, stride), device=DEV), torch.full((2, 8, stride), 1e3, device=DEV)
    for x in (-1, c["pools"][0].shape[0]):
        c["bt"][0, 5] = x
        after = before.clone()
        _, lse = _call(c, after, logits, window, err)
        assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_BLOCK_ID"] and torch.isfinite(lse).all()
        start = max(0, 300 - window) if window else 0
        assert torch.equal(after[0, :, 80:96], before[0, :, 80:96]) and torch.equal(after[0, :, :start], before[0, :, :start])
        add = after - before
        assert (add[0, :, start:80] > 0).all() and (add[0, :, 96:300] > 0).all() and (add[1, :, :77] > 0).all()
        # each row's probabilities sum to 1: four heads a kv head, fp32 sums of 300 steps of at most half 2^-23 of 5
        assert torch.allclose(add.sum(2), torch.full((2, 2), 4.0, device=DEV), rtol=0, atol=300 * 5 * 2.0 ** -24 + 1e-4)
