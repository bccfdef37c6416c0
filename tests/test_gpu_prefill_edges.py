"""The prefill attention where there is nothing to do, and where its result is worked out twice."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
import rules_model
import test_gpu_prefill_attention as prefill
from paged_kv_cache_mapped_gb300 import header_constants
from test_gpu_guard_bands import Guarded, _check

C = header_constants()
DEV = torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("B,hkv", [(1, 1), (3, 8), (600, 2), (4096, 1)])
@pytest.mark.parametrize("what", ["idle", "idle and empty", "refused"])
def test_steps_without_an_entry(what, B, hkv):
    """No sequence has a row to compute: the output stays as it was, and a call with rows on the same workspace
    is as ever (the plan of the empty one has no items and no splits)."""
    c = prefill._case([40, 17, 16] * (B // 3) + [33] * (B % 3), [0] * B, 2 * hkv, hkv, 64, 60, pad=50)
    c["bt"][:, :] = c["bt"][:, :].clamp(min=0)
    want_err = 0
    if what == "idle and empty":
        c["lens"] = [0] * B
    if what == "refused":  # more rows than keys, for the last, and the others behind its start
        c["starts"] = np.array([0] * B + [50], dtype=np.int32)
        c["lens"][-1] = 20
        want_err = C["PKV_DEV_BAD_CONTEXT_LEN"]
    err = pkv.new_error_word(DEV)
    out = Guarded((50, 2 * hkv, 64), torch.bfloat16)
    ws = Guarded((pkv.prefill_workspace_bytes(50, B, 2 * hkv, hkv, 64, c["pools"][0].shape[0], c["bt"].shape[1]),), torch.uint8)
    for r in ({}, dict(softcap=5.0, window=9)):
        out.t.fill_(3.0)
        prefill._call(c, out=out.t, workspace=ws.t, error_word=err, **r)
        assert pkv.read_error(err, clear=True) == want_err
        assert bool((out.t == 3.0).all())
        _check(("out", out), ("workspace", ws))
    rows = dict(c, starts=np.array([0] + [min(9, c["lens"][0] or 9)] * B, dtype=np.int32), lens=[40] + [17] * (B - 1))
    want = prefill._call(rows)[:9]
    out.t.fill_(3.0)
    prefill._call(rows, out=out.t, workspace=ws.t, error_word=err)
    assert pkv.read_error(err) == 0
    # bit for bit: a length past the sequence's own reads the pools' NaN fill
    assert torch.equal(out.t[:9].view(torch.int16), want.view(torch.int16)) and bool((out.t[9:] == 3.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new", [([3000, 2500], [2, 1]), ([900, 700], [400, 130]), ([300, 90], [20, 90])],
                         ids=["in shares", "chunks", "short"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_computed_again_are_the_ones_kept(d, lens, new):
    """NaN and infinities in V rows before the windows, in blocks that the windows share: every row that has such
    a block is computed again, and its second result stands, the same in every one of 40 calls."""
    c = prefill._case(lens, new, 8, 2, d, 61)
    for b, (L, n) in enumerate(zip(lens, new)):
        for row in range(n):
            t = L - n + row - 40  # the first key that the row does not see
            if t >= 0 and row % 97 == 0:
                blk = int(c["bt"][b, t // 16])
                c["pools"][1][blk, :, t % 16, ::3] = (float("nan"), float("inf"), -float("inf"))[row % 3]
    clean = []
    for r in range(int(c["starts"][-1])):
        b = int(np.searchsorted(c["starts"], r, side="right") - 1)
        n, row = new[b], r - int(c["starts"][b])
        # sees [i - 39, i]: no key i' - 40 of a poisoned row i' of its sequence
        if not any(0 <= lens[b] - n + k - 40 and row - 39 <= k - 40 <= row for k in range(0, n, 97)):
            clean += [(r, 0), (r, 5)]
    assert len(clean) >= 4
    err = pkv.new_error_word(DEV)
    first = prefill._call(c, window=40, error_word=err)
    prefill._check(c, first, window=40, rows=clean[:200])
    for _ in range(40):
        assert torch.equal(prefill._call(c, window=40, error_word=err).view(torch.int16), first.view(torch.int16))
    assert pkv.read_error(err) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("rule", ["causal", "prefix and window", "documents"])
@pytest.mark.parametrize("lens,new", [([3000, 2500], [2, 1]), ([1900, 700], [400, 130])], ids=["in shares", "chunks"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_value_that_is_no_number_stays_with_its_columns(d, lens, new, rule):
    """NaN in some columns of a few V rows: NaN in those columns of the rows that see one, the other columns and
    the other rows as without them."""
    c = prefill._case(lens, new, 8, 2, d, 62)
    r = prefill._fill_rules(c, {"causal": {}, "prefix and window": dict(window=300, prefix_lens=200),
                                "documents": dict(doc_starts=90, prefix_lens=40)}[rule])
    at = {0: [3, lens[0] - new[0] // 2, lens[0] - 250], 1: [lens[1] - 90, 190, lens[1] - 1]}
    for b in at:
        for t in at[b]:
            c["pools"][1][int(c["bt"][b, t // 16]), :, t % 16, 3:9] = float("nan")
    err = pkv.new_error_word(DEV)
    got = prefill._call(c, error_word=err, **r)
    assert pkv.read_error(err) == 0
    nan = torch.isnan(got.float()).cpu().numpy()
    assert not nan[:, :, :3].any() and not nan[:, :, 9:].any()
    for row in range(int(c["starts"][-1])):
        b = int(np.searchsorted(c["starts"], row, side="right") - 1)
        i = lens[b] - new[b] + row - int(c["starts"][b])
        lo = max(0, i - r["window"] + 1 if r.get("window") else 0, int(r["doc_starts"][row]) if "doc_starts" in r else 0)
        sees = any(lo <= t <= i or t < (r["prefix_lens"][b] if "prefix_lens" in r else 0) for t in at[b])
        assert nan[row, :, 3:9].all() if sees else not nan[row].any(), (row, i)
    got = got.double().cpu().numpy()
    for row, h in prefill._rows(c, 3):
        b = int(np.searchsorted(c["starts"], row, side="right") - 1)
        L, i = lens[b], lens[b] - new[b] + row - int(c["starts"][b])
        ref, mass, size = rules_model.row(c["q"][row, h].double().numpy(), c["k"][b, :L, h // 4], c["v"][b, :L, h // 4], i, c["scale"],
                                          r.get("window", 0), 0.0, 0.0, int(r["doc_starts"][row]) if "doc_starts" in r else 0,
                                          int(r["prefix_lens"][b]) if "prefix_lens" in r else 0)
        far = np.abs(got[row, h] - ref) - rules_model.bound(ref, mass, size, d, prefill._weight_eps(L))
        assert float(far[~nan[row, h]].max()) <= 0, (row, h)


@pytest.mark.gpu
@pytest.mark.parametrize("t,most_ms", [(0, 5.0), (4032, 5.0), (4046, 20.0)])
def test_cost_of_a_value_that_is_no_number(t, most_ms):
    """A prompt of 4096 tokens (0.1 ms) with a NaN in the first V row, which all rows see, or in the first of the last
    64-token tile, which all its rows see: the result is NaN there by right and not worked out twice but for the rows of
    at most 512 keys (computing every such row again took some 70 ms).  In the middle of that tile the rows before it
    are computed again.  The limits are two to four times what the calls take."""
    c = prefill._case([4096], [4096], 8, 2, 128, 63)
    ins = [c["q"].to(DEV), *c["pools"], c["bt"], torch.tensor([4096], dtype=torch.int32, device=DEV), torch.from_numpy(c["starts"]).to(DEV)]
    c["pools"][1][int(c["bt"][0, t // 16]), :, t % 16] = float("nan")
    pkv.paged_prefill_attention(*ins, c["scale"])
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    got = pkv.paged_prefill_attention(*ins, c["scale"])
    b.record()
    torch.cuda.synchronize()
    assert torch.isnan(got[t:]).all() and not torch.isnan(got[:t]).any()
    assert a.elapsed_time(b) < most_ms


@pytest.mark.gpu
@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("lens,new", [([3000, 2500], [2, 1]), ([1900, 700], [400, 130])], ids=["in shares", "chunks"])
@pytest.mark.parametrize("d", [64, 128])
def test_large_finite_values(d, lens, new, window):
    """V of some 2^120, of either sign: a weight of up to 2^8 times that is past fp32, the output is not.  (Relative
    to the largest, 3000 weights 2^x of normal scores make sums of some 2^120 sqrt(3000 E 4^(x - 4)), below 2^124.)"""
    c = prefill._case(lens, new, 8, 2, d, 64)
    big = 2.0 ** 120
    c["pools"][1].mul_(big)
    c["v"] = c["v"] * big
    err = pkv.new_error_word(DEV)
    got = prefill._call(c, window=window, error_word=err)
    assert pkv.read_error(err) == 0
    assert bool(torch.isfinite(got.float()).all())
    prefill._check(c, got, window=window)
