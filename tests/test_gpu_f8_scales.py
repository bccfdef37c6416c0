"""The FP8 cache's block scales where they decide: a refused row at the start of a block in the append, and
decodes over blocks of far apart weights and scales."""
import numpy as np
import pytest
import torch

import f8_model
import paged_kv_cache_mapped_gb300 as pkv
import rules_model
import test_gpu_decode_rules as decode
import test_gpu_f8_append as append
from paged_kv_cache_mapped_gb300 import header_constants

C = header_constants()
DEV = torch.device("cuda:0")


def _append(pools, k, v, slots):
    dev = [t.to(DEV) for t in pools]
    err = pkv.new_error_word(DEV)
    pkv.kv_append_f8(dev[0], dev[2], dev[1], dev[3], k.to(DEV), v.to(DEV), torch.tensor(slots, device=DEV), error_word=err)
    return dev, pkv.read_error(err)


@pytest.mark.gpu
@pytest.mark.parametrize("in_k", [False, True], ids=["V", "K"])
@pytest.mark.parametrize("spread", [0.0, 5.0], ids=["alike", "apart"])
@pytest.mark.parametrize("slots", [[32], [32, 33], [32, 35, 47], list(range(32, 48)), [16, 17, 32, 33]], ids=str)
def test_a_refused_row_at_offset_0_does_not_start_the_block(slots, spread, in_k):
    """Head 0's row at the block's offset 0 is not finite: it is not written, so the block keeps its scale or
    moves to a larger one with all that it holds; head 1's block starts anew."""
    nb, hkv, d = 4, 2, 64
    k, v = append._rows(len(slots), hkv, d, 21, spread)
    first = slots.index(32)
    (k if in_k else v)[first, 0, 5] = float("nan")
    pools = append._pools(nb, hkv, d, 22)
    dev, code = _append(pools, k, v, slots)
    assert code == C["PKV_DEV_BAD_VALUE"]
    for codes, scales, rows, gc, gs in ((pools[0], pools[1], k, dev[0], dev[1]), (pools[2], pools[3], v, dev[2], dev[3])):
        for h in (0, 1):
            at = [-1 if h == 0 and i == first else s for i, s in enumerate(slots)]
            r = np.nan_to_num(rows[:, h:h + 1].double().numpy())
            wc, ws = f8_model.append(append._vals(codes[:, h:h + 1]), scales[:, h:h + 1].numpy(), r, at)
            assert np.array_equal(gs[:, h:h + 1].cpu().double().numpy(), ws), h
            assert np.array_equal(append._vals(gc[:, h:h + 1]), wc), h


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1.0, float("nan"), float("inf")])
def test_a_refused_row_at_offset_0_leaves_the_old_scale_to_be_checked(bad):
    """The block does not start anew, so an old scale that is no scale refuses the block's other rows."""
    k, v = append._rows(2, 1, 128, 23)
    k[0, 0, 0] = float("inf")
    pools = append._pools(4, 1, 128, 24)
    pools[3][2, 0] = bad
    dev, code = _append(pools, k, v, [32, 33])
    assert code == C["PKV_DEV_BAD_VALUE"]
    assert all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8)) for a, b in zip(dev, pools))


@pytest.mark.gpu
@pytest.mark.parametrize("slots,written", [([9, 12, 11, 13, 40], [9, 12, -1, -1, 40]), ([16, 17, 17, 18, 19], [16, 17, -1, -1, -1]),
                                           ([3, 2, 1, 0, 16], [3, -1, -1, -1, 16]), ([40, 41, 40, -1, 9], [40, 41, -1, -1, 9])])
def test_tokens_after_a_descending_one_are_left_out(slots, written):
    """What a block's tokens before the refused one write stands, with the scale of those alone."""
    k, v = append._rows(len(slots), 2, 128, 25)
    pools = append._pools(4, 2, 128, 26)
    dev, code = _append(pools, k, v, slots)
    assert code == C["PKV_DEV_BAD_SLOT"]
    for codes, scales, rows, gc, gs in ((pools[0], pools[1], k, dev[0], dev[1]), (pools[2], pools[3], v, dev[2], dev[3])):
        wc, ws = f8_model.append(append._vals(codes), scales.numpy(), rows.double().numpy(), written)
        assert np.array_equal(gs.cpu().double().numpy(), ws) and np.array_equal(append._vals(gc), wc)


@pytest.mark.gpu
@pytest.mark.parametrize("a", [1.703125, 1.6953125])
@pytest.mark.parametrize("d", [64, 128])
def test_light_keys_keep_their_digits_beside_heavy_ones(d, a):
    """The first block's keys weigh 2^19.6 times the others' and have V = 0, so the others, all alike, make the
    output; 2000 copies, so that most lie whole in one warp's share, where fp16's smallest step of 2^-24 is not to be
    counted from the heavy keys' weight (it would be 1.5 % of a light one)."""
    c = decode._case([64], 8, 2, d, 51, True)
    kc, ks, vc, vs = c["pools"]
    first = int(c["bt"][0, 0])
    c["q"] = torch.full((1, 8, d), a).bfloat16()
    c["scale"] = 8.0 / d  # logits 8 a in the first block, 0 in the others
    for t, x in ((kc, 0.0), (vc, 3.0), (ks, 1.0), (vs, 0.25)):
        t.copy_(torch.full(t.shape, x).to(t.dtype))
    kc[first] = torch.ones_like(kc[first].float()).to(kc.dtype)
    vc[first] = torch.zeros_like(vc[first].float()).to(vc.dtype)
    n = 2000
    many = dict(c, q=c["q"].repeat(n, 1, 1), bt=c["bt"].repeat(n, 1), lens=c["lens"] * n)
    err = pkv.new_error_word(DEV)
    got = decode._call(many, err=err).double().cpu().numpy()
    assert pkv.read_error(err) == 0
    k, v = np.zeros((64, d)), np.full((64, d), 0.75)
    k[:16], v[:16] = 1.0, 0.0
    ref, mass, size = rules_model.row(np.full(d, a), k, v, 63, c["scale"])
    far = np.abs(got - ref) - rules_model.bound(ref, mass, size, d, 2.0 ** -11)
    assert float(far.max()) <= 0


ENDS = [(-120, 40, -9.0), (-100, 60, -6.07), (-120, 119, -9.0), (-120, 119, -7.0), (0, 119, -6.0), (-30, 119, -9.5), (119, -120, -9.0),
        (-100, 100, -0.1)]


def _far_scales(e0, e1, slope, zero, d):
    """Two sequences whose first block has V scale 2^e0 and the largest weights, the others 2^e1 and weights of
    2^(23 slope) a block less, so that either may carry the row; as all zeros the first block is what the append
    makes of a block of zero rows.  Also each row's exact output, its bound, and Σ |v|.  The bound takes, beside
    the half step of 2^-11 of each weight, that of fp16's smallest numbers: 2^-25 in units of 2^-6 of the largest weight
    times scale (no scale counting less than 2^-100 there), for each code."""
    c = decode._case([64, 41], 8, 2, d, 50, True)
    c["q"].zero_()  # the logits are the distance bias alone
    vc, vs = c["pools"][2], c["pools"][3]
    vs.fill_(2.0 ** e1)
    first = c["bt"][:, 0].long()
    vs[first] = 2.0 ** e0
    if zero:
        vc.view(torch.uint8)[first] = 0
    x = vc.float().cpu().double().numpy() * vs.cpu().double().numpy()[:, :, None, None]
    ref, bound, size = (np.zeros((2, 8, d)) for _ in range(3))
    for b, L in enumerate(c["lens"]):
        for t in range(L):
            c["v"][b, t] = x[int(c["bt"][b, t // 16]), :, t % 16]
        for h in range(8):
            v = c["v"][b, :L, h // 4]
            ref[b, h], mass, top = rules_model.row(np.zeros(d), c["k"][b, :L, h // 4], v, L - 1, 1.0, slope=float(np.float32(slope)))
            bound[b, h] = rules_model.bound(ref[b, h], mass, top, d, 2.0 ** -11)
            size[b, h] = np.abs(v).sum(0)
            s = np.array([float(vs[int(c["bt"][b, t // 16]), h // 4]) for t in range(L)])
            p = np.exp(slope * np.arange(L) - max(0.0, slope * (L - 1)))
            bound[b, h] += 2.0 ** -31 * (p * np.maximum(s, 2.0 ** -100)).max() * (np.abs(v) / s[:, None]).sum(0)
    return c, ref, bound, size


@pytest.mark.gpu
@pytest.mark.parametrize("e0,e1,slope", ENDS)
@pytest.mark.parametrize("zero", [False, True], ids=["values", "zeros"])
@pytest.mark.parametrize("d", [64, 128])
def test_v_scales_at_both_ends_of_their_range(d, zero, e0, e1, slope):
    """Two sequences, every block in a share of its own.  Shares are joined by fp32 weights relative to the
    largest: one is off by up to 2^-148 (two steps of the smallest numbers), and a share holds its keys by
    weights of up to 2^8 in that unit, over a sum of at least 1: 2^-140 of Σ |v|."""
    c, ref, bound, size = _far_scales(e0, e1, slope, zero, d)
    err = pkv.new_error_word(DEV)
    got = decode._call(c, err=err, alibi_slopes=[slope] * 8).double().cpu().numpy()
    assert pkv.read_error(err) == 0
    assert float((np.abs(got - ref) - bound - 2.0 ** -140 * size).max()) <= 0


@pytest.mark.gpu
@pytest.mark.parametrize("e0,e1,slope", ENDS)
@pytest.mark.parametrize("zero", [False, True], ids=["values", "zeros"])
@pytest.mark.parametrize("d", [64, 128])
def test_v_scales_far_apart_within_a_share(d, zero, e0, e1, slope):
    """2000 copies of each sequence, 14000 units and more for some 1800 warps: shares of 8 units and more, in which
    most sequences (of 3 and 4 units) lie whole.  Each key's weight is an fp32 number relative to the largest, off
    by up to 2^-148 where it is one of the smallest, 2^-148 of Σ |v|: half of the copies at least meet that."""
    c, ref, bound, size = _far_scales(e0, e1, slope, zero, d)
    n = 2000
    many = dict(c, q=c["q"].repeat(n, 1, 1), bt=c["bt"].repeat(n, 1), lens=c["lens"] * n)
    err = pkv.new_error_word(DEV)
    got = decode._call(many, err=err, alibi_slopes=[slope] * 8).double().cpu().numpy().reshape(n, 2, 8, d)
    assert pkv.read_error(err) == 0
    far = np.abs(got - ref) - bound
    assert float((far - 2.0 ** -140 * size).max()) <= 0
    assert float(np.mean(far <= 2.0 ** -148 * size, axis=0).min()) >= 0.5
