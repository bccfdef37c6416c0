"""Attention of many query tokens per sequence over the paged cache against the 64-bit model: ragged
batches from one token to chunks that span many tiles, every group size, both head sizes, score rules
alone and together, rows that see nothing, NaN and infinities in what is masked, padding rows, a run
with the step tables and the append, streams and graphs, refusals."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
import rules_model
from helpers import paged_from_contiguous, rand_bf16
from paged_kv_cache_mapped_gb300 import _lib, header_constants

C = header_constants()
DEV = torch.device("cuda:0")


def _case(lens, new, hq, hkv, d, seed, fill=float("nan"), pad=0):
    g = torch.Generator().manual_seed(seed)
    B, lmax = len(lens), max(max(lens), 1)
    k, v = rand_bf16((B, lmax, hkv, d), g), rand_bf16((B, lmax, hkv, d), g)
    nb = sum((L + 15) // 16 for L in lens) + 3
    kc, vc, bt = paged_from_contiguous(k, v, lens, nb, g, fill=fill)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = rand_bf16((int(starts[-1]) + pad, hq, d), g)
    return dict(q=q, k=k.double().numpy(), v=v.double().numpy(), pools=[kc.to(DEV), vc.to(DEV)], bt=bt.to(DEV), lens=list(lens),
                new=list(new), starts=starts, scale=d ** -0.5, hq=hq, hkv=hkv, d=d)


def _call(c, window=0, **r):
    kw = {n: r[n] for n in ("out", "workspace", "error_word", "stream") if n in r}
    for n, t in (("alibi_slopes", torch.float32), ("doc_starts", torch.int32), ("prefix_lens", torch.int32)):
        if r.get(n) is not None:
            kw[n] = torch.as_tensor(np.asarray(r[n]), dtype=t, device=DEV)
    return pkv.paged_prefill_attention(c["q"].to(DEV), *c["pools"], c["bt"], torch.tensor(c["lens"], dtype=torch.int32, device=DEV),
                                       torch.from_numpy(c["starts"]).to(DEV), c["scale"], window, softcap=r.get("softcap", 0.0), **kw)


def _rows(c, seed, most=60):
    """Rows to look at: the first and last of every sequence, some at tile edges, some at random."""
    rng = np.random.default_rng(seed)
    rows = set()
    for b, n in enumerate(c["new"]):
        q0 = int(c["starts"][b])
        rows |= {q0 + j for j in (0, 1, n // 2, n - 2, n - 1) if 0 <= j < n}
        rows |= {q0 + int(j) for j in rng.integers(0, n, min(n, 6))} if n else set()
    return [(r, int(h)) for r in sorted(rows) for h in ({0, c["hq"] - 1} | set(rng.integers(0, c["hq"], 2).tolist()))]


def _weight_eps(L):
    """Half a step of the weights in the product with V: two bf16 terms (2^-8 * 2^-8) over at most four
    128-key tiles, which a sequence of up to 512 keys cannot exceed; one bf16 term (2^-8) beyond."""
    return 2.0 ** -16 if L <= 512 else 2.0 ** -8


def _check(c, got, window=0, rows=None, **r):
    got = got.float().cpu().double().numpy()
    g = c["hq"] // c["hkv"]
    for row, h in rows or _rows(c, 1):
        b = int(np.searchsorted(c["starts"], row, side="right") - 1)
        L = c["lens"][b]
        i = L - c["new"][b] + row - int(c["starts"][b])
        ref, mass, size = rules_model.row(
            c["q"][row, h].double().numpy(), c["k"][b, :L, h // g], c["v"][b, :L, h // g], i, c["scale"], window,
            r.get("softcap", 0.0), 0.0 if r.get("alibi_slopes") is None else float(np.float32(r["alibi_slopes"][h])),
            0 if r.get("doc_starts") is None else int(r["doc_starts"][row]),
            0 if r.get("prefix_lens") is None else int(r["prefix_lens"][b]))
        far = np.abs(got[row, h] - ref) - rules_model.bound(ref, mass, size, c["d"], _weight_eps(L))
        assert np.all(far <= 0), (row, h, b, i, float(far.max()), float(np.abs(got[row, h] - ref).max()))


def _slopes(hq):
    return [2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]


def _run(c, **r):
    err = pkv.new_error_word(DEV)
    got = _call(c, error_word=err, **r)
    assert pkv.read_error(err) == 0
    _check(c, got, **r)
    return got


BATCHES = {
    "one token": ([1], [1]),
    "tokens of long and short contexts": ([700, 1, 33], [1, 1, 1]),
    "whole prompts": ([300, 17, 128, 1], [300, 17, 128, 1]),
    "chunks": ([400, 260, 129], [100, 131, 128]),
    "an idle sequence": ([40, 50, 0, 60], [3, 0, 0, 60]),
}
RULES = {
    "causal": {},
    "cap": dict(softcap=5.0),
    "alibi": dict(alibi_slopes=True),
    "window": dict(window=37),
    "window 1": dict(window=1),
    "prefix": dict(prefix_lens=70),
    "prefix and window": dict(window=20, prefix_lens=45),
    "documents": dict(doc_starts=23),
    "all": dict(window=64, softcap=30.0, alibi_slopes=True, doc_starts=90, prefix_lens=18),
}


def _fill_rules(c, r):
    r = dict(r)
    if r.get("alibi_slopes"):
        r["alibi_slopes"] = _slopes(c["hq"])
    if "prefix_lens" in r:
        r["prefix_lens"] = [r["prefix_lens"] * (b % 3) // 2 for b in range(len(c["lens"]))]
    if "doc_starts" in r:
        pos = np.concatenate([np.arange(L - n, L) for L, n in zip(c["lens"], c["new"])])
        r["doc_starts"] = pos // r["doc_starts"] * r["doc_starts"]
    return r


@pytest.mark.gpu
@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (12, 2, 128), (8, 2, 128)])
def test_matches_the_model(batch, rule, hq, hkv, d):
    c = _case(*BATCHES[batch], hq, hkv, d, hq * d)
    _run(c, **_fill_rules(c, RULES[rule]))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", range(1, 9))
def test_every_group_size(group, d):
    c = _case([150, 31], [70, 31], 2 * group, 2, d, group)
    r = dict(softcap=4.0, alibi_slopes=_slopes(2 * group))
    _run(c, **r)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257])
def test_lengths_at_tile_edges(n):
    c = _case([n, n + 100, n + 1], [n, n, 1], 4, 1, 128, n)
    _run(c)
    _run(c, window=17)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_long_contexts(d):
    """Few rows over long contexts (split over the keys) beside a long prompt."""
    c = _case([20000, 3000, 5000], [2, 1500, 1], 8, 2, d, 3)
    rows = [(0, 0), (1, 7), (2, 3), (700, 1), (1499, 5), (1501, 0), (1502, 6)]
    for r in ({}, dict(softcap=10.0, window=2500, prefix_lens=[3000, 100, 17], alibi_slopes=_slopes(8))):
        err = pkv.new_error_word(DEV)
        got = _call(c, error_word=err, **r)
        assert pkv.read_error(err) == 0
        _check(c, got, rows=rows, **r)


@pytest.mark.gpu
def test_many_sequences():
    """More sequences than any tile holds, lengths all different, most of one token."""
    rng = np.random.default_rng(4)
    lens = rng.integers(1, 90, 333)
    new = [int(min(L, n)) for L, n in zip(lens, rng.choice([0, 1, 1, 1, 20, 60], 333))]
    c = _case([int(x) for x in lens], new, 6, 3, 64, 5)
    _run(c, prefix_lens=[int(x) for x in rng.integers(0, 30, 333)], window=25)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_see_nothing_are_zero(d):
    c = _case([100, 64], [100, 3], 4, 2, d, 6)
    pos = np.concatenate([np.arange(100), np.arange(61, 64)])
    docs = np.where(np.arange(103) % 3 == 0, pos + 1 + np.arange(103) % 7, np.maximum(pos - 5, 0))
    got = _run(c, doc_starts=docs)
    assert not got[torch.arange(0, 103, 3)].any()
    got = _run(c, doc_starts=np.full(103, 1 << 30))
    assert not got.any()
    _run(c, doc_starts=np.full(103, 1 << 30), prefix_lens=[5, 0])
    _run(c, doc_starts=np.full(103, -5))


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_masked_infinities_stay_out(d):
    """NaN and infinities in keys that some rows see and others do not: rows that do not see them are as
    without them, in whatever tile they share."""
    c = _case([200, 90], [150, 90], 4, 2, d, 7)
    r = _fill_rules(c, dict(window=30, doc_starts=41, prefix_lens=12))
    bt = c["bt"].cpu()
    at = [(0, 60, float("nan")), (0, 111, float("inf")), (0, 199, -float("inf")), (1, 33, float("nan")), (1, 89, float("nan"))]
    for b, t, x in at:
        blk = int(bt[b, t // 16])
        c["pools"][1][blk, :, t % 16, 3:9] = x
        c["pools"][0][blk, :, t % 16, 5] = x
    got = _call(c, **r)
    clean = []
    for row in range(240):
        b = int(row >= 150)
        i = 50 + row if b == 0 else row - 150
        lo = max(0, i - 29, int(r["doc_starts"][row]))
        if any(bb == b and (lo <= t <= i or t < r["prefix_lens"][b]) for bb, t, _ in at):
            continue
        clean += [(row, h) for h in range(4)]
    assert len(clean) > 400
    _check(c, got, rows=clean, **r)  # against the keys as they were before


@pytest.mark.gpu
def test_padding_rows_and_guard():
    """Rows past the last sequence stay as they were, q's there may hold anything."""
    c = _case([60, 130], [60, 70], 4, 2, 128, 8, pad=37)
    c["q"][130:] = float("nan")
    out = torch.full((167, 4, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    got = _call(c, out=out)
    assert got is out and bool((out[130:] == 7.0).all())
    _check(c, out)


@pytest.mark.gpu
def test_prefill_of_one_token_equals_the_decode_to_rounding():
    lens = [700, 1, 64, 4000]
    c = _case(lens, [1] * 4, 8, 2, 128, 9)
    r = dict(softcap=9.0, prefix_lens=[10, 0, 3, 99], alibi_slopes=_slopes(8))
    got = _call(c, window=300, **r).float()
    t = {n: torch.tensor(v, dtype=torch.float32 if n[0] == "a" else torch.int32, device=DEV) for n, v in r.items() if n != "softcap"}
    want = pkv.paged_decode_attention_rules(c["q"].to(DEV), *c["pools"], c["bt"], torch.tensor(lens, dtype=torch.int32, device=DEV),
                                            c["scale"], 300, softcap=9.0, **t).float()
    # each is within half a bf16 step (2^-8 of the value) of the exact result, and the long rows' weights are off by
    # up to 2^-8 each: 2.1 * 2^-8 of the sum of p |v|, which is below 1.5 for normal values
    assert torch.allclose(got, want, rtol=2.0 ** -6, atol=2.1 * 2.0 ** -8 * 1.5)


@pytest.mark.gpu
def test_a_run_of_the_operators():
    """Tables, append, attention over three engine steps (prompts; a chunk with decodes; a release and an
    admission), all shapes fixed and captured once: the model sees the same keys and outputs agree."""
    B, mb, nb, T, hq, hkv, d = 4, 12, 30, 96, 4, 2, 64
    g = torch.Generator().manual_seed(10)
    i32 = dict(dtype=torch.int32, device=DEV)
    bt, lens, new, count = torch.full((B, mb), -1, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32), torch.tensor([nb], **i32)
    free = torch.randperm(nb, generator=g).to(**i32)
    kc, vc = (torch.full((nb, hkv, 16, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    starts, slots = torch.empty(B + 1, **i32), torch.empty(T, dtype=torch.int64, device=DEV)
    pos, out = torch.empty(T, **i32), torch.empty((T, hq, d), dtype=torch.bfloat16, device=DEV)
    q, k, v = (torch.empty((T, n, d), dtype=torch.bfloat16, device=DEV) for n in (hq, hkv, hkv))
    ws = torch.empty(pkv.prefill_workspace_bytes(T, B, hq, hkv, d, nb, mb), dtype=torch.uint8, device=DEV)
    err = pkv.new_error_word(DEV)

    def step():
        pkv.kv_step_tables(bt, lens, new, free, count, T, context_lens_out=lens, free_count_out=count, query_starts=starts,
                           slot_mapping=slots, positions=pos, error_word=err)
        pkv.kv_append(kc, vc, k, v, slots, error_word=err)
        pkv.paged_prefill_attention(q, kc, vc, bt, lens, starts, d ** -0.5, 50, softcap=20.0, out=out, workspace=ws, error_word=err)

    q.zero_(), k.zero_(), v.zero_()
    step()  # nothing new: one-time set-up
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    keys = [[] for _ in range(B)]
    for want in ([40, 0, 17, 1], [1, 60, 1, 1], [1, 1, -1, 33], [1, 1, 20, 1]):
        rows = [rand_bf16((T, n, d), g) for n in (hq, hkv, hkv)]
        for t, x in zip((q, k, v), rows):
            t.copy_(x)
        new.copy_(torch.tensor(want, **i32))
        graph.replay()
        assert pkv.read_error(err) == 0
        at = 0
        got = out.float().cpu().double().numpy()
        for b, n in enumerate(want):
            if n < 0:
                keys[b] = []
            for j in range(max(n, 0)):
                keys[b].append((rows[1][at + j].double().numpy(), rows[2][at + j].double().numpy()))
            kk, vv = ((np.stack([x[z] for x in keys[b]]) if keys[b] else None) for z in (0, 1))
            for j in range(max(n, 0)):
                for h in range(hq):
                    ref, mass, size = rules_model.row(rows[0][at + j, h].double().numpy(), kk[:, h // 2], vv[:, h // 2],
                                                      len(keys[b]) - n + j, d ** -0.5, 50, 20.0)
                    far = np.abs(got[at + j, h] - ref) - rules_model.bound(ref, mass, size, d, _weight_eps(len(keys[b])))
                    assert np.all(far <= 0), (b, j, h)
            at += max(n, 0)


@pytest.mark.gpu
def test_another_stream_and_two_workspaces():
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


@pytest.mark.gpu
def test_device_errors():
    c = _case([100, 60, 40], [50, 60, 1], 4, 2, 128, 13)
    good = _call(c)
    err = pkv.new_error_word(DEV)
    keep = c["starts"].copy()
    for bad, code, ok in (([0, 50, 45, 46], "PKV_DEV_BAD_QUERY_RANGE", slice(0, 45)),
                          ([-1, 50, 110, 111], "PKV_DEV_BAD_QUERY_RANGE", slice(50, 111)),
                          ([0, 50, 110, 112], "PKV_DEV_BAD_QUERY_RANGE", slice(0, 110))):
        c["starts"] = np.asarray(bad, dtype=np.int32)
        out = torch.full_like(good, 5.0)
        _call(c, error_word=err, out=out)
        assert pkv.read_error(err, clear=True) == C[code], bad
        assert torch.equal(out[ok], good[ok]), bad
    c["starts"] = keep
    for lens in ([49, 60, 40], [100, -1, 40], [100, 60, 16 * c["bt"].shape[1] + 1]):
        c["lens"] = lens
        out = torch.full_like(good, 5.0)
        _call(c, error_word=err, out=out)
        assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_CONTEXT_LEN"], lens
        same = [torch.equal(out[a:z], good[a:z]) for a, z in ((0, 50), (50, 110), (110, 111))]
        kept = [bool((out[a:z] == 5.0).all()) for a, z in ((0, 50), (50, 110), (110, 111))]
        bad = [x not in (100, 60, 40) for x in lens]
        assert kept == bad and same == [not x for x in bad], lens
    c["lens"] = [100, 60, 40]
    c["bt"][1, 2] = c["pools"][0].shape[0] + 7
    got = _call(c, error_word=err)
    assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_BLOCK_ID"]
    assert torch.equal(got[:50], good[:50]) and torch.equal(got[110:], good[110:]) and torch.equal(got[50:82], good[50:82])


def test_host_validation_codes():
    from paged_kv_cache_mapped_gb300 import _build
    _build.build()
    lib, P = _lib.load(), ctypes.c_void_p

    def call(T=64, ws=1 << 40, cap=0.0, q=0x10000, starts=0x10000, **kw):
        dims = dict(B=4, hq=32, hkv=8, d=128, bs=16, nb=1000, mb=64)
        dims.update(kw)
        d = _lib.PkvDims(*dims.values())
        r = _lib.PkvScoreRules(cap, 0, None, None, None)
        return lib.pkv_paged_prefill_attention(P(0x10000), P(q), P(0x10000), P(0x10000), P(0x10000), P(0x10000), P(starts), T, 0.1,
                                               ctypes.byref(r), P(0x20000), ws, ctypes.byref(d), None, None)

    assert call(B=0) == C["PKV_OK"] and call(T=0) == C["PKV_OK"]
    assert call(T=-1) == C["PKV_ERR_DIMS"] and call(B=4097) == C["PKV_ERR_DIMS"] and call(T=1 << 27) == C["PKV_ERR_DIMS"]
    assert call(d=80) == C["PKV_ERR_HEAD_DIM"] and call(hq=72) == C["PKV_ERR_GQA"] and call(bs=8) == C["PKV_ERR_BLOCK_SIZE"]
    assert call(cap=float("nan")) == C["PKV_ERR_ARGUMENT"] and call(ws=16) == C["PKV_ERR_WORKSPACE"]
    assert call(q=0x10002) == C["PKV_ERR_ALIGNMENT"] and call(starts=None) == C["PKV_ERR_NULL_POINTER"]
    d = _lib.PkvDims(4, 32, 8, 96, 16, 1000, 64)
    assert lib.pkv_prefill_workspace_bytes(ctypes.byref(d), 64) == 0
