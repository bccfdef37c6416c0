"""pkv_kv_append_f8 against the host model, exactly: fresh blocks and blocks whose scale stays or
grows, runs that start and end inside a block, single tokens, zero rows, the ends of the exponent
range, scales that are no powers of two, skipped and refused tokens, and untouched blocks."""
import numpy as np
import pytest
import torch

import f8_model
import paged_kv_cache_mapped_gb300 as pkv
from paged_kv_cache_mapped_gb300 import header_constants

C = header_constants()
DEV = torch.device("cuda:0")


def test_grid_of_the_model_is_torchs():
    """The model's rounding against torch's own conversion: every E4M3 value, the midpoints between
    neighbours and the values beside them."""
    v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mid = (v[1:] + v[:-1]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), [447.9]])
    x = np.concatenate([x, -x]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(f8_model.round_e4m3(x), want)


def test_scale_of_the_model():
    for amax, e in [(448.0, 0), (448.1, 1), (0.0, -120), (224.0, -1), (1.75 * 2.0 ** 127, 119), (1e-40, -120)]:
        assert f8_model.needed_scale(amax) == 2.0 ** e, amax


def _pools(nb, hkv, d, seed, pow2=True):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        codes = (torch.randn((nb, hkv, 16, d), generator=g) * 120).clamp(-448, 448).to(torch.float8_e4m3fn)
        e = torch.randint(-9, -4, (nb, hkv), generator=g).float()
        scales = torch.exp2(e if pow2 else e + torch.rand((nb, hkv), generator=g))
        out += [codes, scales]
    return out  # k codes, k scales, v codes, v scales


def _rows(T, hkv, d, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    amp = torch.exp2(torch.randn((T, hkv, 1), generator=g) * spread)
    return [(torch.randn((T, hkv, d), generator=g) * amp).bfloat16() for _ in range(2)]


def _vals(codes):
    return codes.cpu().float().double().numpy()


def _check(pools, k, v, slots, err_code=0, model_slots=None):
    kc, ks, vc, vs = pools
    dev = [t.to(DEV) for t in pools]
    err = pkv.new_error_word(DEV)
    pkv.kv_append_f8(dev[0], dev[2], dev[1], dev[3], k.to(DEV), v.to(DEV), torch.tensor(slots, dtype=torch.int64, device=DEV),
                     error_word=err)
    assert pkv.read_error(err) == err_code
    at = slots if model_slots is None else model_slots
    for codes, scales, rows, gc, gs in ((kc, ks, k, dev[0], dev[1]), (vc, vs, v, dev[2], dev[3])):
        wc, ws = f8_model.append(_vals(codes), scales.numpy(), rows.double().numpy(), at)
        assert np.array_equal(gs.cpu().double().numpy(), ws)
        assert np.array_equal(_vals(gc), wc)
    return dev


LAYOUTS = {
    "one token at 0": [32],
    "one token inside": [37],
    "last of a block": [47],
    "whole block": list(range(48, 64)),
    "all but the first": list(range(49, 64)),
    "across blocks": list(range(26, 32)) + list(range(96, 112)) + list(range(112, 115)),
    "gaps": [65, 67, 68, 79, 3, 9],
    "with skips": [-1, 33, 34, -1, -1, 80, -1],
}


@pytest.mark.gpu
@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 128), (2, 64), (8, 128)])
@pytest.mark.parametrize("name", LAYOUTS)
def test_append_matches_the_model(name, hkv, d, pow2):
    slots = LAYOUTS[name]
    _check(_pools(8, hkv, d, 1, pow2), *_rows(len(slots), hkv, d, 2), slots)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_token_by_token_equals_the_model_step_by_step(d):
    """Forty decode steps of three sequences, one token each: scales grow as larger rows arrive."""
    hkv = 2
    pools = _pools(12, hkv, d, 3)
    for step in range(40):
        k, v = _rows(3, hkv, d, 100 + step)
        slots = [(step // 16) * 16 + step % 16 + 64 * b for b in range(3)]
        dev = _check(pools, k, v, slots)
        pools = [t.cpu() for t in dev]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 7, 16, 333, 5000])
def test_long_calls(T):
    hkv, d, nb = 2, 128, 400
    perm = np.random.default_rng(T).permutation(nb)
    at = np.arange(5, 5 + T)
    _check(_pools(nb, hkv, d, 4), *_rows(T, hkv, d, 5), [int(s) for s in perm[at // 16] * 16 + at % 16])


@pytest.mark.gpu
def test_extreme_rows():
    """Zeros, the smallest and largest bf16 numbers, values on the 448 edge of a scale and ties."""
    d, hkv = 64, 1
    tiny, big = torch.finfo(torch.bfloat16).smallest_normal, torch.finfo(torch.bfloat16).max
    rows = torch.zeros((7, hkv, d))
    rows[1, 0, 3] = tiny
    rows[2, 0, :2] = torch.tensor([big, -big])
    rows[3, 0, 0] = 448.0
    rows[4, 0, 0] = 450.0
    rows[5, 0] = torch.arange(d) * 0.5 + 16.5
    rows[6, 0, 0] = 2.0 ** -133
    k = rows.bfloat16()
    _check(_pools(8, hkv, d, 6), k, k.flip(0), [0, 16, 32, 48, 64, 80, 96])
    _check(_pools(8, hkv, d, 6), k, k.flip(0), [1, 18, 35, 52, 69, 86, 103])


@pytest.mark.gpu
def test_zero_scale_pools_and_empty_call():
    pools = _pools(4, 2, 128, 7)
    pools[1].zero_()
    pools[3].zero_()
    _check(pools, *_rows(3, 2, 128, 8), [5, 6, 33])
    _check(pools, *_rows(0, 2, 128, 8), [])
    _check(pools, *_rows(2, 2, 128, 8), [-1, -5])


@pytest.mark.gpu
def test_refused_tokens():
    nb, hkv, d = 8, 2, 128
    k, v = _rows(4, hkv, d, 9)
    # a slot outside the pool: the other tokens are written
    _check(_pools(nb, hkv, d, 10), k, v, [3, nb * 16, 40, 41], C["PKV_DEV_BAD_SLOT"], [3, -1, 40, 41])
    # descending and equal slots of one block: reported, the first of the run stands
    _check(_pools(nb, hkv, d, 10), k, v, [9, 8, 40, 41], C["PKV_DEV_BAD_SLOT"], [9, -1, 40, 41])
    _check(_pools(nb, hkv, d, 10), k, v, [9, 9, 40, 41], C["PKV_DEV_BAD_SLOT"], [9, -1, 40, 41])


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_rows_are_left_out(bad):
    """Token 1's V row of head 0 holds the value: its head-0 rows of K and V stay as they were and do
    not count for the scale; head 1 is written whole."""
    nb, hkv, d = 4, 2, 64
    k, v = _rows(3, hkv, d, 11)
    v[1, 0, 7] = bad
    pools = _pools(nb, hkv, d, 12)
    dev = [t.to(DEV) for t in pools]
    err = pkv.new_error_word(DEV)
    pkv.kv_append_f8(dev[0], dev[2], dev[1], dev[3], k.to(DEV), v.to(DEV), torch.tensor([20, 21, 22], device=DEV), error_word=err)
    assert pkv.read_error(err) == C["PKV_DEV_BAD_VALUE"]
    for codes, scales, rows, gc, gs in ((pools[0], pools[1], k, dev[0], dev[1]), (pools[2], pools[3], v, dev[2], dev[3])):
        for h, at in ((0, [20, -1, 22]), (1, [20, 21, 22])):
            r = rows[:, h:h + 1].double().numpy()
            r = np.where(np.isfinite(r), r, 0.0)
            wc, ws = f8_model.append(_vals(codes[:, h:h + 1]), scales[:, h:h + 1].numpy(), r, at)
            assert np.array_equal(gs[:, h:h + 1].cpu().double().numpy(), ws)
            assert np.array_equal(_vals(gc[:, h:h + 1]), wc)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1.0, float("nan"), float("inf")])
def test_bad_old_scale_is_refused_unless_the_block_starts_anew(bad):
    nb, hkv, d = 4, 1, 128
    k, v = _rows(1, hkv, d, 13)
    pools = _pools(nb, hkv, d, 14)
    pools[3][2, 0] = bad
    dev = [t.to(DEV) for t in pools]
    err = pkv.new_error_word(DEV)
    args = (dev[0], dev[2], dev[1], dev[3], k.to(DEV), v.to(DEV))
    pkv.kv_append_f8(*args, torch.tensor([35], device=DEV), error_word=err)
    assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_VALUE"]
    assert all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8)) for a, b in zip(dev, pools))
    pkv.kv_append_f8(*args, torch.tensor([32], device=DEV), error_word=err)
    assert pkv.read_error(err) == 0 and float(dev[3][2, 0]) == f8_model.needed_scale(float(v.abs().max()))


def test_host_refusals():
    c, s = torch.zeros((2, 1, 16, 64), dtype=torch.float8_e4m3fn), torch.zeros((2, 1))
    r, at = torch.zeros((1, 1, 64), dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_append_f8(c, c, s, s, r, r, at)
    with pytest.raises(TypeError, match="float8"):
        pkv.kv_append_f8(c.view(torch.uint8), c, s, s, r, r, at)
