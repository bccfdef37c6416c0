"""Capped scores of the prefill attention where the cap is far above them: masked keys of any size, rows
past a sequence and other rows' scores leave a row's logits alone (to the cap's last bits, 2^-22 of it in base 2,
for caps up to 177: with 150 3.6e-5 of a weight, which the bound's 2^-16 and roundings of the logit allow); and the cap's polynomials by
themselves, read from the kernel's source."""
import os
import re

import numpy as np
import pytest
import torch

import test_gpu_prefill_attention as prefill
from paged_kv_cache_mapped_gb300._build import CSRC

LARGE_CAPS = [150.0, 300.0, 1e5, 1e6, 1e8, 1e30]


def _poison(c, b, keys, x):
    """K of these masked keys becomes x (the model keeps the values that they had)."""
    for t in keys:
        c["pools"][0][int(c["bt"][b, t // 16]), :, t % 16] = x


@pytest.mark.gpu
@pytest.mark.parametrize("x", [float("inf"), -3e38, 1e20])
@pytest.mark.parametrize("softcap", LARGE_CAPS)
@pytest.mark.parametrize("d", [64, 128])
def test_masked_keys_of_any_size_leave_the_cap_alone(d, softcap, x):
    """Keys before every window and past every length, in tiles that the rows' own keys share, in short rows
    (weights in two terms) and in long ones."""
    c = prefill._case([200, 1700, 450], [1, 60, 100], 4, 2, d, 40, fill=x)
    _poison(c, 0, range(160, 170), x)    # the token at 199 sees 30 keys
    _poison(c, 1, range(1600, 1611), x)  # the first of 60 sees 1611 on
    r = dict(softcap=softcap, window=30)
    prefill._run(c, **r)
    c = prefill._case([200, 1700, 450], [1, 60, 100], 4, 2, d, 41, fill=x)
    prefill._run(c, softcap=softcap, alibi_slopes=prefill._slopes(4))


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", LARGE_CAPS)
@pytest.mark.parametrize("new", [[40, 90], [2, 3]], ids=["chunks", "few tokens"])
def test_rows_of_large_scores_leave_the_others_alone(softcap, new):
    """One token's queries are 10^6 or 10^8 times the others', which share its warp."""
    for size in (1e6, 1e8):
        c = prefill._case([900, 300], new, 4, 2, 128, 42)
        c["q"][1] *= size
        c["q"][new[0] + 1] *= size
        small = [(row, h) for row, h in prefill._rows(c, 2) if row not in (1, new[0] + 1)]
        for r in (dict(softcap=softcap), dict(softcap=softcap, alibi_slopes=prefill._slopes(4), prefix_lens=[70, 0])):
            prefill._check(c, prefill._call(c, **r), rows=small, **r)


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", LARGE_CAPS)
def test_large_caps_with_a_negative_scale(softcap):
    c = prefill._case([700, 130], [90, 130], 4, 2, 64, 43)
    c["scale"] = -0.09
    prefill._run(c, softcap=softcap)


def _constants():
    with open(os.path.join(CSRC, "prefill_attention.cu")) as f:
        text = f.read()
    near, far = (float(x) for x in re.search(r"kCapNear = ([0-9.]+)f, kCapFar = ([0-9.]+)f", text).groups())
    polys = [[float(x.strip().rstrip("f")) for x in re.search(name + r"\[\d\] = \{([^}]*)\}", text).group(1).split(",")]
             for name in ("kCap2", "kCap5")]
    return (near, polys[0]), (far, polys[1])


@pytest.mark.parametrize("which,in_reals,in_fp32", [(0, 1.41e-7, 2.05e-7), (1, 1.0e-7, 2.05e-7)], ids=["near", "far"])
def test_polynomials_of_the_cap(which, in_reals, in_fp32):
    """tanh(u) / u over the whole range with the stored coefficients, in 64 bits and by Horner's rule in fp32.
    The polynomials of least error are off by 1.1e-7 and 5.8e-8; the constant term, just below 1, is stored to
    half a step of 2^-24 and the others to finer ones times u^2 and more, over P of at least 0.987 and 0.83: 3.1e-8
    and 4.2e-8 more.  In fp32 the last sum rounds by 2^-24 (6.1e-8, 7.2e-8 relative), the earlier ones by that
    times at most a third of u^2."""
    reach, coef = _constants()[which]
    c = np.array(coef, dtype=np.float32)
    u = np.linspace(reach / 200001, reach, 200001).astype(np.float32)
    want = np.tanh(u.astype(np.float64)) / u
    p = np.zeros(u.shape)
    for k in c[::-1].astype(np.float64):
        p = p * u.astype(np.float64) ** 2 + k
    assert np.abs(p / want - 1).max() <= in_reals
    w = u * u
    p = np.full_like(w, c[-1])
    for k in c[-2::-1]:  # a fused multiply-add rounds once
        p = (p.astype(np.float64) * w.astype(np.float64) + np.float64(k)).astype(np.float32)
    assert np.abs(p / want - 1).max() <= in_fp32
