"""Differential attention of many tokens: the weights of the nearest steps of a long row are two bf16 terms (2^-16) and
not one (2^-8), in shares and whole, for every set of rules.

Every key of a kv head has the same V, so each map's output is that V whatever the logits and under equal factors of 1 the
difference is 0; what is left is the rounding of the weights, which the sums of the weights (of unrounded ones) do not share.
With the weight on the nearest keys an output may be off, for each map, by two terms' 2^-16 of |V| and by fp32 roundings: those of
the products and sums of some hundred keys and of a rescale a step, fewer than 256 of 2^-24, 2^-16 as well.  One term is off by
up to 2^-9 a weight."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
import test_gpu_diff_prefill as prefill

DEV = torch.device("cuda:0")
BOUND = 2 * (2.0 ** -16 + 2.0 ** -16)   # both maps, of |V|


def _equal_values(c):
    """One V for all keys of a kv head, of both signs."""
    g = torch.Generator().manual_seed(5)
    v = (torch.rand((c["hkv"], c["d"]), generator=g) + 1).bfloat16() * (torch.randint(0, 2, (c["hkv"], c["d"]), generator=g) * 2 - 1)
    c["pools"][1][:] = v.bfloat16()[None, :, None].to(DEV)
    c["lam"][:] = 1.0
    return v.double().abs()


def _off(c, v, **r):
    err = pkv.new_error_word(DEV)
    got = prefill._call(c, error_word=err, **r).double().cpu().abs()
    assert pkv.read_error(err) == 0
    g = c["hq"] // c["hkv"]
    return (got / v.repeat_interleave(g, 0)).amax(-1)   # [rows, heads], of |V|


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("lens,new", [([3000, 2500], [2, 1]), ([1900, 700], [400, 130]), ([6000], [1500])],
                         ids=["in shares", "chunks", "a long chunk"])
@pytest.mark.parametrize("d", [64, 128])
def test_near_keys_under_a_distance_bias(d, lens, new, softcap):
    """Slopes of 0.5 and 0.3: beyond 100 keys the weights are below 2^-40."""
    c = prefill._case(lens, new, 8, 2, d, 71, norm=False)
    v = _equal_values(c)
    off = _off(c, v, alibi_slopes=[0.5, 0.3] * 4, softcap=softcap)
    assert off.max() <= BOUND * (1 + 2.0 ** -8), float(off.max())


def _aim(c, blocks):
    """Logits of some 30 above the others' at the keys of block `blocks[b]` of each sequence, apart by fractions."""
    half, g = c["d"] // 2, torch.Generator().manual_seed(6)
    c["pools"][0][:] = 0
    for b, blk in enumerate(blocks):
        own = int(c["bt"][b, blk])
        for m in range(2):
            x = 1 + 0.5 * torch.rand((c["hkv"], 16, half), generator=g)
            c["pools"][0][own, :, :, m * half:(m + 1) * half] = x.bfloat16().to(DEV)
    c["q"] = ((1 + 0.1 * torch.rand(c["q"].shape, generator=g)) * 30.0 * half ** -0.5).bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [0.0, 200.0])
@pytest.mark.parametrize("lens,new", [([3000, 2500], [2, 1]), ([1900, 1700], [60, 33])], ids=["in shares", "chunks"])
@pytest.mark.parametrize("d", [64, 128])
def test_near_keys_that_the_query_points_at(d, lens, new, softcap):
    """No bias: the last whole block that every row sees carries the weight, within the nearest sixth of the steps.  (The
    others' logits are 30 * half / sqrt(half) * scale = 30 below, 4000 of them 2^-31.)"""
    c = prefill._case(lens, new, 8, 2, d, 72, norm=False)
    v = _equal_values(c)
    _aim(c, [(L - n + 1) // 16 - 1 for L, n in zip(lens, new)])
    off = _off(c, v, softcap=softcap)
    assert off.max() <= BOUND * (1 + 2.0 ** -8), float(off.max())


@pytest.mark.parametrize("d", [64, 128])
def test_one_term_is_past_the_bound(d):
    """The same rows with weights of one bf16 term, worked out here: most rows are past the bound."""
    rng = np.random.default_rng(d)
    past = 0
    for _ in range(200):
        off = 0.0
        for m in range(2):
            n = np.arange(120)
            x = rng.standard_normal(120) - 0.4 * n
            p = np.exp2((x - x.max()) * 1.4426950408889634).astype(np.float32)
            one = torch.from_numpy(p).bfloat16().double().numpy()
            off += (1 - 2 * m) * one.sum() / p.astype(np.float64).sum()
        past += abs(off) > 2 * BOUND
    assert past > 150, past
