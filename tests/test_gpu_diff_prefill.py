"""Differential attention of many query tokens against the 64-bit model: ragged batches, every group size, both head sizes,
factors of heads and of rows, with and without the norm, score rules, rows that see nothing, what is not finite in masked
and in seen places, long contexts whose result names the blocks, padding, streams and graphs, refusals; and the run
of tables, append, prefill, decode with scores and eviction."""
import ctypes

import numpy as np
import pytest
import torch

import diff_model
import paged_kv_cache_mapped_gb300 as pkv
import rules_model
import test_gpu_prefill_attention as prefill
import test_gpu_prefill_long_rows as long_rows
from helpers import rand_bf16
from paged_kv_cache_mapped_gb300 import _lib, header_constants
from test_gpu_guard_bands import Guarded
from test_gpu_guard_bands import _check as guards

C = header_constants()
DEV = torch.device("cuda:0")
EPS = 1e-5


def _case(lens, new, hq, hkv, d, seed, per_row=False, norm=True, **kw):
    c = prefill._case(lens, new, hq, hkv, d, seed, **kw)
    g = torch.Generator().manual_seed(seed + 1000)
    T = c["q"].shape[0]
    c.update(scale=(d // 2) ** -0.5, lam=torch.rand((T, hq) if per_row else (hq,), generator=g) * 1.2 - 0.2,
             w=1 + 0.3 * torch.randn((d,), generator=g) if norm else None)
    return c


def _call(c, window=0, **r):
    kw = {n: r[n] for n in ("out", "workspace", "error_word", "stream") if n in r}
    for n, t in (("alibi_slopes", torch.float32), ("doc_starts", torch.int32), ("prefix_lens", torch.int32)):
        if r.get(n) is not None:
            kw[n] = torch.as_tensor(np.asarray(r[n]), dtype=t, device=DEV)
    return pkv.paged_diff_prefill_attention(
        c["q"].to(DEV), *c["pools"], c["bt"], torch.tensor(c["lens"], dtype=torch.int32, device=DEV),
        torch.from_numpy(c["starts"]).to(DEV), c["lam"].to(DEV), c["scale"], window, softcap=r.get("softcap", 0.0),
        norm_weight=None if c["w"] is None else c["w"].to(DEV), norm_eps=EPS, **kw)


def _check(c, got, window=0, rows=None, **r):
    got = got.float().cpu().double().numpy()
    g = c["hq"] // c["hkv"]
    w = None if c["w"] is None else c["w"].double().numpy()
    for row, h in rows or prefill._rows(c, 1):
        b = int(np.searchsorted(c["starts"], row, side="right") - 1)
        L = c["lens"][b]
        i = L - c["new"][b] + row - int(c["starts"][b])
        lam = float(c["lam"][row, h] if c["lam"].dim() == 2 else c["lam"][h])
        ref, tol = diff_model.row(
            c["q"][row, h].double().numpy(), c["k"][b, :L, h // g], c["v"][b, :L, h // g], i, c["scale"], lam, w, EPS,
            prefill._weight_eps(L), window=window, softcap=r.get("softcap", 0.0),
            slope=0.0 if r.get("alibi_slopes") is None else float(np.float32(r["alibi_slopes"][h])),
            doc_start=0 if r.get("doc_starts") is None else int(r["doc_starts"][row]),
            prefix=0 if r.get("prefix_lens") is None else int(r["prefix_lens"][b]))
        far = np.abs(got[row, h] - ref) - tol
        assert np.all(far <= 0), (row, h, b, i, float(far.max()), float(np.abs(got[row, h] - ref).max()))


def _run(c, **r):
    err = pkv.new_error_word(DEV)
    got = _call(c, error_word=err, **r)
    assert pkv.read_error(err) == 0
    _check(c, got, **r)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("rule", prefill.RULES)
@pytest.mark.parametrize("batch", prefill.BATCHES)
@pytest.mark.parametrize("hq,hkv,d,norm", [(4, 4, 64, False), (12, 2, 128, True), (8, 2, 128, False)])
def test_matches_the_model(batch, rule, hq, hkv, d, norm):
    c = _case(*prefill.BATCHES[batch], hq, hkv, d, hq * d, norm=norm, per_row=hq == 12)
    _run(c, **prefill._fill_rules(c, prefill.RULES[rule]))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", range(1, 9))
def test_every_group_size(group, d):
    c = _case([150, 31], [70, 31], 2 * group, 2, d, group)
    _run(c, softcap=4.0, alibi_slopes=prefill._slopes(2 * group))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
def test_lengths_at_tile_edges(n):
    c = _case([n, n + 100, n + 1], [n, n, 1], 4, 1, 128, n, norm=n % 2 == 0)
    _run(c)
    _run(c, window=17)


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_long_contexts(d, norm):
    """Few rows over long contexts (split over the keys) beside a long prompt."""
    c = _case([20000, 3000, 5000], [2, 1500, 1], 8, 2, d, 3, norm=norm)
    rows = [(0, 0), (1, 7), (2, 3), (700, 1), (1499, 5), (1501, 0), (1502, 6)]
    for r in ({}, dict(softcap=10.0, window=2500, prefix_lens=[3000, 100, 17], alibi_slopes=prefill._slopes(8))):
        err = pkv.new_error_word(DEV)
        got = _call(c, error_word=err, **r)
        assert pkv.read_error(err) == 0
        _check(c, got, rows=rows, **r)


@pytest.mark.gpu
def test_many_sequences():
    rng = np.random.default_rng(4)
    lens = rng.integers(1, 90, 333)
    new = [int(min(L, n)) for L, n in zip(lens, rng.choice([0, 1, 1, 1, 20, 60], 333))]
    c = _case([int(x) for x in lens], new, 6, 3, 64, 5, per_row=True)
    _run(c, prefix_lens=[int(x) for x in rng.integers(0, 30, 333)], window=25)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("norm", [False, True])
def test_rows_that_see_nothing_are_zero(d, norm):
    c = _case([100, 64], [100, 3], 4, 2, d, 6, norm=norm)
    c["lam"][1] = float("inf")   # no key, whatever the factor
    pos = np.concatenate([np.arange(100), np.arange(61, 64)])
    docs = np.where(np.arange(103) % 3 == 0, pos + 1 + np.arange(103) % 7, np.maximum(pos - 5, 0))
    got = _call(c, doc_starts=docs)
    assert not got[torch.arange(0, 103, 3)].any()
    c["lam"][1] = 0.3
    _run(c, doc_starts=docs)
    assert not _run(c, doc_starts=np.full(103, 1 << 30)).any()
    _run(c, doc_starts=np.full(103, 1 << 30), prefix_lens=[5, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new", [([3000, 2500], [2, 1]), ([900, 700], [400, 130]), ([300, 90], [20, 90])],
                         ids=["in shares", "chunks", "short"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_computed_again_are_the_ones_kept(d, lens, new):
    """NaN and infinities in V and K rows before the windows, in blocks that the windows share: rows that do not see
    one are as without them, the same in every one of 20 calls."""
    c = _case(lens, new, 8, 2, d, 61, norm=d == 64)
    for b, (L, n) in enumerate(zip(lens, new)):
        for row in range(n):
            t = L - n + row - 40  # the first key that the row does not see
            if t >= 0 and row % 97 == 0:
                blk, bad = int(c["bt"][b, t // 16]), (float("nan"), float("inf"), -float("inf"))[row % 3]
                c["pools"][1][blk, :, t % 16, ::3] = bad
                c["pools"][0][blk, :, t % 16, 5] = bad
    clean = []
    for r in range(int(c["starts"][-1])):
        b = int(np.searchsorted(c["starts"], r, side="right") - 1)
        n, row = new[b], r - int(c["starts"][b])
        if not any(0 <= lens[b] - n + k - 40 and row - 39 <= k - 40 <= row for k in range(0, n, 97)):
            clean += [(r, 0), (r, 5)]
    assert len(clean) >= 4
    err = pkv.new_error_word(DEV)
    first = _call(c, window=40, error_word=err)
    _check(c, first, window=40, rows=clean[:200])
    for _ in range(20):
        assert torch.equal(_call(c, window=40, error_word=err).view(torch.int16), first.view(torch.int16))
    assert pkv.read_error(err) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("lens,new", [([3000, 2500], [2, 1]), ([1900, 700], [400, 130])], ids=["in shares", "chunks"])
@pytest.mark.parametrize("d", [64, 128])
def test_a_value_that_is_no_number_stays_with_its_rows(d, lens, new, norm):
    """NaN in some columns of a few V rows: the rows that see one have NaN in those columns (a norm spreads it over the
    row), the others are as without them."""
    c = _case(lens, new, 8, 2, d, 62, norm=norm)
    r = dict(window=300, prefix_lens=[200, 100])
    at = {0: [3, lens[0] - new[0] // 2, lens[0] - 250], 1: [lens[1] - 90, 190, lens[1] - 1]}
    for b in at:
        for t in at[b]:
            c["pools"][1][int(c["bt"][b, t // 16]), :, t % 16, 3:9] = float("nan")
    err = pkv.new_error_word(DEV)
    got = _call(c, error_word=err, **r)
    assert pkv.read_error(err) == 0
    nan = torch.isnan(got.float()).cpu().numpy()
    clean = []
    for row in range(int(c["starts"][-1])):
        b = int(np.searchsorted(c["starts"], row, side="right") - 1)
        i = lens[b] - new[b] + row - int(c["starts"][b])
        if any(i - 299 <= t <= i or t < r["prefix_lens"][b] for t in at[b]):
            assert nan[row, :, 3:9].all() and (norm or not (nan[row, :, :3].any() or nan[row, :, 9:].any())), (row, i)
        else:
            assert not nan[row].any(), (row, i)
            clean.append((row, row % 8))
    if clean:
        _check(c, got, rows=clean[::7], **r)


@pytest.mark.gpu
def test_the_halves_do_not_mix():
    """An infinity in one half of a seen K row gives that map a weight of 0 (its logit is -infinity) and leaves the other map alone."""
    for d in (64, 128):
        c = _case([300], [60], 4, 2, d, 8, fill=0.0)
        blk = int(c["bt"][0, 1])
        for half in (0, 1):
            at = d // 2 * half + 5
            c["q"][:, :, at] = 1.0
            old = c["pools"][0][blk, :, 3].clone()
            outs = []
            for x in (-3e38, float("-inf")):
                c["pools"][0][blk, :, 3, at] = x
                outs.append(_call(c))
            c["pools"][0][blk, :, 3] = old
            assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])


@pytest.mark.gpu
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("lens,new", [([3000, 2500], [2, 1]), ([1900, 700], [400, 130])], ids=["in shares", "chunks"])
def test_large_finite_values(lens, new, norm):
    """V of some 2^120: weights of up to 2^8 times that, and squares, are past fp32, the output is not."""
    c = _case(lens, new, 8, 2, 128, 64, norm=norm)
    c["pools"][1].mul_(2.0 ** 120)
    c["v"] = c["v"] * 2.0 ** 120
    got = _run(c, window=300)
    assert bool(torch.isfinite(got.float()).all())


@pytest.mark.gpu
def test_padding_rows_and_guards():
    c = _case([60, 130], [60, 70], 4, 2, 128, 8, pad=37, per_row=True)
    c["q"][130:] = float("nan")
    c["lam"][130:] = float("nan")
    out = Guarded((167, 4, 128), torch.bfloat16)
    ws = Guarded((pkv.diff_prefill_workspace_bytes(167, 2, 4, 2, 128, c["pools"][0].shape[0], c["bt"].shape[1]),), torch.uint8)
    out.t.fill_(7.0)
    got = _call(c, out=out.t, workspace=ws.t)
    assert got is out.t and bool((out.t[130:] == 7.0).all())
    guards(("out", out), ("workspace", ws))
    _check(c, out.t)


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [0.0, 200.0])
@pytest.mark.parametrize("shape", long_rows.SHAPES)
def test_every_block_counts_once_in_its_place(shape, softcap):
    """The first map points at two blocks of up to 8192, the second at two others: the result names all four.  (K's
    halves are the test's own directions of half the size, whose 32 or 64 signs keep other blocks apart at twice the
    scale or more.)"""
    lens, new, hq, hkv, d, seed = long_rows.SHAPES[shape]
    c = long_rows._case(lens, new, hq, hkv, d, seed)
    cache = [t.to(DEV) for t in (*c["pools"], c["bt"])]
    half = d // 2
    # a block's own keys stand half / 4 * scale = 24 + above the mean; of 32 signs several blocks may share
    # many, so the reference is the model over all keys, not the blocks' mean
    scale = 2 * long_rows.SCALE[d]
    lam = torch.linspace(0.3, 0.9, hq)
    qs = []
    for _ in range(2):
        q, at = long_rows._aim(c)
        qs.append(q)
    q = torch.cat([qs[0][..., :half], qs[1][..., half:]], -1)
    err = pkv.new_error_word(DEV)
    got = pkv.paged_diff_prefill_attention(q.to(DEV), *cache, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                           torch.from_numpy(c["starts"]).to(DEV), lam.to(DEV), scale, softcap=softcap, error_word=err)
    assert pkv.read_error(err) == 0
    got = got.float().cpu().double().numpy()
    some = list(at)
    if len(some) > 80:
        some = [some[int(x)] for x in c["rng"].integers(0, len(some), 80)]
    for row, h in some:
        b = at[row, h][0]
        L, g = lens[b], hq // hkv
        i = L - new[b] + row - int(c["starts"][b])
        ref, tol = diff_model.row(q[row, h].double().numpy(), c["k"][b, :i + 1, h // g].double().numpy(),
                                  c["v"][b, :i + 1, h // g].double().numpy(), i, scale, float(lam[h]), None, EPS,
                                  prefill._weight_eps(L), softcap=softcap)
        assert np.all(np.abs(got[row, h] - ref) <= tol), (row, h, at[row, h], float(np.abs(got[row, h] - ref).max()))


@pytest.mark.parametrize("d", [64, 128])
def test_planted_mistakes_are_past_the_bound(d):
    """A 128-key tile lost to one of the maps, or read from the place of another, at the tiles that the map points at."""
    c = long_rows._case([9000], [4], 4, 2, d, 9)
    half, scale, g = d // 2, 2 * long_rows.SCALE[d], 2
    aims = [long_rows._aim(c) for _ in range(2)]
    for (row, h), _ in aims[0][1].items():
        n = 9000 - 4 + row + 1
        k, v = c["k"][0, :n, h // g].double().numpy(), c["v"][0, :n, h // g].double().numpy()
        maps = []
        for m in range(2):
            at = slice(m * half, (m + 1) * half)
            maps.append((aims[m][0][row, h, at].double().numpy(), k[:, at]))
        lam = 0.6
        q = np.concatenate([maps[0][0], maps[1][0]])
        ref, tol = diff_model.row(q, k, v, n - 1, scale, lam, None, EPS, 2.0 ** -8)
        for m in range(2):
            _, i, j = aims[m][1][row, h]
            if i // 8 == j // 8:
                continue
            seen = np.arange(n)
            inside = seen // 128 == i // 8
            other = (i // 8 + 5) % (n // 128)
            for keys in (seen[~inside], np.where(inside, other * 128 + seen % 128, seen)):
                good = rules_model.row(*[x for x in (maps[m][0], maps[m][1], v)], n - 1, scale)[0]
                wrong = rules_model.row(maps[m][0], maps[m][1][keys], v[keys], len(keys) - 1, scale)[0]
                off = np.abs((wrong - good) * (1.0 if m == 0 else lam))
                assert np.mean(off > 2 * tol) > 0.3, (row, h, m, i, j)


@pytest.mark.gpu
def test_one_token_equals_the_decode_to_rounding():
    lens = [700, 1, 64, 4000]
    c = _case(lens, [1] * 4, 8, 2, 128, 9, norm=False)
    r = dict(softcap=9.0, prefix_lens=[10, 0, 3, 99], alibi_slopes=prefill._slopes(8))
    got = _call(c, window=300, **r).float()
    t = {n: torch.tensor(v, dtype=torch.float32 if n[0] == "a" else torch.int32, device=DEV) for n, v in r.items() if n != "softcap"}
    want = pkv.paged_diff_decode_attention(c["q"].to(DEV), *c["pools"], c["bt"], torch.tensor(lens, dtype=torch.int32, device=DEV),
                                           c["lam"].to(DEV), c["scale"], 300, softcap=9.0, **t).float()
    # each within half a bf16 step of the exact result, the long rows' weights off by up to 2^-8 each in both maps
    # (factors below 1): 2.1 * 2^-8 of twice the sum of p |v|, which is below 1.5 for normal values
    assert torch.allclose(got, want, rtol=2.0 ** -6, atol=2 * 2.1 * 2.0 ** -8 * 1.5)


@pytest.mark.gpu
def test_other_streams_graph_and_steps_without_an_entry():
    cs = [_case([500, 90], [33, 90], 8, 2, 128, 11 + i) for i in range(2)]
    want = [_call(c, softcap=3.0) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    outs = []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            outs.append(_call(c, softcap=3.0))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    c = cs[0]
    i32 = dict(dtype=torch.int32, device=DEV)
    q, lam, w, lens, starts = (c["q"].to(DEV), c["lam"].to(DEV), c["w"].to(DEV), torch.tensor(c["lens"], **i32),
                               torch.from_numpy(c["starts"]).to(DEV))
    ws = torch.empty(pkv.diff_prefill_workspace_bytes(123, 2, 8, 2, 128, c["pools"][0].shape[0], c["bt"].shape[1]), dtype=torch.uint8,
                     device=DEV)
    out = torch.empty_like(want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_diff_prefill_attention(q, *c["pools"], c["bt"], lens, starts, lam, c["scale"], norm_weight=w, norm_eps=EPS, softcap=3.0,
                                         out=out, workspace=ws)
    for new in (None, [0, 0], None, [1, 90]):
        out.fill_(5.0)
        starts.copy_(torch.from_numpy(c["starts"]) if new is None else torch.tensor([0, *np.cumsum(new)]))
        graph.replay()
        torch.cuda.synchronize()
        if new is None:
            assert torch.equal(out, want[0])
        elif sum(new) == 0:
            assert bool((out == 5.0).all())
        else:
            _check(dict(c, new=new, starts=np.array([0, 1, 91], dtype=np.int32)), out, softcap=3.0)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_cost_of_a_factor_that_is_no_number(bad):
    """A prompt of 4096 tokens, the factor of one head NaN or infinite: that head's rows are no numbers by right
    and are not worked out twice, and the others are as ever."""
    c = _case([4096], [4096], 8, 2, 128, 35, per_row=False)
    ins = [c["q"].to(DEV), *c["pools"], c["bt"], torch.tensor([4096], dtype=torch.int32, device=DEV), torch.from_numpy(c["starts"]).to(DEV)]
    lam = c["lam"].to(DEV)
    want = pkv.paged_diff_prefill_attention(*ins, lam, c["scale"])
    lam[3] = bad
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    got = pkv.paged_diff_prefill_attention(*ins, lam, c["scale"])
    b.record()
    torch.cuda.synchronize()
    assert not torch.isfinite(got[:, 3]).any()
    others = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(got[:, others], want[:, others])
    assert a.elapsed_time(b) < 10.0


@pytest.mark.gpu
def test_device_errors():
    c = _case([100, 60, 40], [50, 60, 1], 4, 2, 128, 13)
    good = _call(c)
    err = pkv.new_error_word(DEV)
    keep = c["starts"].copy()
    c["starts"] = np.asarray([0, 50, 45, 46], dtype=np.int32)
    out = torch.full_like(good, 5.0)
    _call(c, error_word=err, out=out)
    assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_QUERY_RANGE"] and torch.equal(out[:45], good[:45])
    c["starts"] = keep
    c["lens"] = [49, 60, 40]
    out = torch.full_like(good, 5.0)
    _call(c, error_word=err, out=out)
    assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_CONTEXT_LEN"]
    assert bool((out[:50] == 5.0).all()) and torch.equal(out[50:], good[50:])
    c["lens"] = [100, 60, 40]
    c["bt"][1, 2] = c["pools"][0].shape[0] + 7
    got = _call(c, error_word=err)
    assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_BLOCK_ID"]
    assert torch.equal(got[:50], good[:50]) and torch.equal(got[110:], good[110:]) and torch.equal(got[50:82], good[50:82])


@pytest.mark.gpu
def test_a_run_of_the_operators():
    """An engine over a differential layer: prompts through the tables, the append and the prefill; then single tokens with the decode that
    adds the keys' weights, and eviction past a trigger.  Every output is the model's over the tokens that are left."""
    B, mb, nb, T, hq, hkv, d = 3, 12, 30, 96, 4, 2, 64
    n_sink, k_top, n_recent, trigger = 3, 12, 10, 40
    budget, scale = n_sink + k_top + n_recent, (d // 2) ** -0.5
    g = torch.Generator().manual_seed(21)
    i32 = dict(dtype=torch.int32, device=DEV)
    bt, lens, gone, count = torch.full((B, mb), -1, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32), torch.tensor([nb], **i32)
    free = torch.randperm(nb, generator=g).to(**i32)
    kc, vc = (torch.full((nb, hkv, 16, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    scores, slot_pos = torch.zeros((B, hkv, mb * 16), device=DEV), torch.full((B, hkv, mb * 16), -1, **i32)
    lam, w = torch.rand(hq, generator=g), 1 + 0.2 * torch.randn(d, generator=g)
    lam_d, w_d, wn = lam.to(DEV), w.to(DEV), w.double().numpy()
    err = pkv.new_error_word(DEV)
    held = [[{} for _ in range(hkv)] for _ in range(B)]   # position -> [K row, V row, score]
    cuts = 0
    for step in range(50):
        new = [37, 20, 5] if step == 0 else [0, 0, 30] if step == 9 else [1, 1 if step % 4 else 0, 1]
        first = (lens + gone).tolist()
        q, k, v = (rand_bf16((T, n, d), g) for n in (hq, hkv, hkv))
        lens, starts, slots, _, count = pkv.kv_step_tables(bt, lens, torch.tensor(new, **i32), free, count, T, error_word=err)
        pkv.kv_append(kc, vc, k.to(DEV), v.to(DEV), slots, error_word=err)
        at = np.concatenate([[0], np.cumsum(new)])
        for b in range(B):
            for h in range(hkv):
                for i in range(new[b]):
                    held[b][h][first[b] + i] = [k[at[b] + i, h].double().numpy(), v[at[b] + i, h].double().numpy(), 0.0]
        single = max(new) == 1
        if single:   # rows of q by sequence
            rows = torch.tensor([int(at[b]) if new[b] else 0 for b in range(B)])
            qb = q[rows]
            out = pkv.paged_diff_decode_attention_scores(qb.to(DEV), kc, vc, bt, lens, lam_d, scores, scale, norm_weight=w_d,
                                                         error_word=err).float().cpu().double().numpy()
        else:
            out = pkv.paged_diff_prefill_attention(q.to(DEV), kc, vc, bt, lens, starts, lam_d, scale, norm_weight=w_d,
                                                   error_word=err).float().cpu().double().numpy()
        for b in range(B):
            for h in range(hq):
                order = list(held[b][h // 2])
                keys, vals = (np.stack([held[b][h // 2][t][z] for t in order]) for z in (0, 1))
                if single:
                    ref, tol = diff_model.row(qb[b, h].double().numpy(), keys, vals, len(order) - 1, scale, float(lam[h]), wn, 1e-5, 2.0 ** -15)
                    assert np.all(np.abs(out[b, h] - ref) <= tol), (step, b, h)
                elif gone[b] == 0:   # (after an eviction the slots are in no order, and a chunk's rows see what is before them in slots)
                    for i in range(new[b]):
                        n = len(order) - new[b] + i + 1
                        ref, tol = diff_model.row(q[at[b] + i, h].double().numpy(), keys[:n], vals[:n], n - 1, scale, float(lam[h]), wn, 1e-5,
                                                  2.0 ** -16)
                        assert np.all(np.abs(out[at[b] + i, h] - ref) <= tol), (step, b, h, i)
            if single:
                for n in range(hkv):
                    order = list(held[b][n])
                    keys = np.stack([held[b][n][t][0] for t in order])
                    add, _ = diff_model.score([qb[b, h].double().numpy() for h in (2 * n, 2 * n + 1)], keys, len(order) - 1, scale,
                                              [float(lam[2 * n]), float(lam[2 * n + 1])], [{}, {}])
                    for t, x in zip(order, add):
                        held[b][n][t][2] += x
        lens_was = lens.tolist()
        lens, gone, count = pkv.kv_evict(kc, vc, bt, lens, scores, slot_pos, gone, n_sink, k_top, n_recent, trigger=trigger,
                                         free_blocks=free, free_count=count, error_word=err)
        L, lost, sc, ps = lens.tolist(), gone.tolist(), scores.cpu().numpy(), slot_pos.cpu().numpy()
        for b in range(B):
            seen = L[b] + lost[b]
            assert seen == first[b] + new[b]
            if lens_was[b] <= trigger:
                continue
            cuts += 1
            for n in range(hkv):
                kept = ps[b, n, :budget].tolist()
                assert L[b] == budget and len(set(kept)) == budget
                assert set(range(n_sink)) <= set(kept) and set(range(seen - n_recent, seen)) <= set(kept)
                for i, t in enumerate(kept):
                    assert abs(sc[b, n, i] - held[b][n][t][2]) <= 1e-5 * (1 + held[b][n][t][2])
                rest = [r[2] for t, r in held[b][n].items() if t not in kept]
                assert max(rest) <= min(held[b][n][t][2] for t in kept if n_sink <= t < seen - n_recent) + 1e-5
                held[b][n] = {t: held[b][n][t] for t in kept}
        owned = [int(x) for b in range(B) for x in bt[b, :(L[b] + 15) // 16].tolist()] + free[:int(count)].tolist()
        assert sorted(owned) == list(range(nb))
    assert pkv.read_error(err) == 0 and cuts >= 5


def test_host_validation_codes():
    from paged_kv_cache_mapped_gb300 import _build
    _build.build()
    lib, P = _lib.load(), ctypes.c_void_p

    def call(T=64, ws=1 << 40, cap=0.0, q=0x10000, starts=0x10000, lam=0x10000, rows=0, eps=1e-5, w=0x10000, **kw):
        dims = dict(B=4, hq=32, hkv=8, d=128, bs=16, nb=1000, mb=64)
        dims.update(kw)
        d = _lib.PkvDims(*dims.values())
        r, p = _lib.PkvScoreRules(cap, 0, None, None, None), _lib.PkvDiffParams(lam, rows, eps, w)
        return lib.pkv_paged_diff_prefill_attention(P(0x10000), P(q), P(0x10000), P(0x10000), P(0x10000), P(0x10000), P(starts), T, 0.1,
                                                    ctypes.byref(p), ctypes.byref(r), P(0x20000), ws, ctypes.byref(d), None, None)

    assert call(B=0) == C["PKV_OK"] and call(T=0) == C["PKV_OK"]
    assert call(T=-1) == C["PKV_ERR_DIMS"] and call(B=4097) == C["PKV_ERR_DIMS"] and call(T=1 << 27) == C["PKV_ERR_DIMS"]
    assert call(d=80) == C["PKV_ERR_HEAD_DIM"] and call(hq=72) == C["PKV_ERR_GQA"] and call(bs=8) == C["PKV_ERR_BLOCK_SIZE"]
    assert call(cap=float("nan")) == C["PKV_ERR_ARGUMENT"] and call(ws=16) == C["PKV_ERR_WORKSPACE"]
    assert call(q=0x10002) == C["PKV_ERR_ALIGNMENT"] and call(starts=None) == call(lam=None) == C["PKV_ERR_NULL_POINTER"]
    assert call(rows=3) == call(eps=0.0) == call(eps=float("nan")) == C["PKV_ERR_ARGUMENT"] and call(w=0x10002) == C["PKV_ERR_ALIGNMENT"]
    d = _lib.PkvDims(4, 32, 8, 128, 16, 1000, 64)
    n = lib.pkv_diff_prefill_workspace_bytes(ctypes.byref(d), 64)
    assert n >= lib.pkv_prefill_workspace_bytes(ctypes.byref(d), 64) > 0 and call(ws=n - 1) == C["PKV_ERR_WORKSPACE"]
    for at, x in (("head_dim", 96), ("num_q_heads", 72), ("batch", 4097)):
        bad = _lib.PkvDims(4, 32, 8, 128, 16, 1000, 64)
        setattr(bad, at, x)
        assert lib.pkv_diff_prefill_workspace_bytes(ctypes.byref(bad), 64) == 0
    ok = (64, 4, 32, 8, 128, 1000, 64)
    for i in range(len(ok)):
        for x in (2**32 + ok[i], 2**31, -1):
            with pytest.raises(ValueError):
                pkv.diff_prefill_workspace_bytes(*ok[:i], x, *ok[i + 1:])
