"""Differential attention of one token against the 64-bit model: lengths from 0 up, every group size, both head
sizes, factors of heads and of rows, with and without the norm, score rules, rows that see nothing, NaN and
infinities in what is masked, the weights added into the scores; the inputs-ready flag, streams, graphs, guard bands,
refusals."""
import ctypes

import numpy as np
import pytest
import torch

import diff_model
import paged_kv_cache_mapped_gb300 as pkv
from helpers import paged_from_contiguous, rand_bf16
from paged_kv_cache_mapped_gb300 import _lib, header_constants

C = header_constants()
DEV = torch.device("cuda:0")
EPS = 1e-5


def _case(lens, hq, hkv, d, seed, fill=float("nan"), per_row=False, norm=True):
    g = torch.Generator().manual_seed(seed)
    B, lmax = len(lens), max(max(lens), 1)
    q = rand_bf16((B, hq, d), g)
    k, v = rand_bf16((B, lmax, hkv, d), g), rand_bf16((B, lmax, hkv, d), g)
    nb = sum((L + 15) // 16 for L in lens) + 3
    kc, vc, bt = paged_from_contiguous(k, v, lens, nb, g, fill=fill)
    lam = torch.rand((B, hq) if per_row else (hq,), generator=g) * 1.2 - 0.2
    w = 1 + 0.3 * torch.randn((d,), generator=g) if norm else None
    return dict(q=q, k=k.double().numpy(), v=v.double().numpy(), pools=[kc.to(DEV), vc.to(DEV)], bt=bt.to(DEV), lens=list(lens),
                scale=(d // 2) ** -0.5, hq=hq, hkv=hkv, d=d, lam=lam, w=w)


def _kw(c, r):
    kw = {n: r[n] for n in ("out", "workspace", "error_word", "inputs_ready", "stream", "scores_out", "softcap") if n in r}
    for n, t in (("alibi_slopes", torch.float32), ("doc_starts", torch.int32), ("prefix_lens", torch.int32)):
        if r.get(n) is not None:
            kw[n] = torch.as_tensor(r[n], dtype=t, device=DEV)
    return dict(kw, norm_weight=None if c["w"] is None else c["w"].to(DEV), norm_eps=EPS)


def _call(c, window=0, scores=None, **r):
    args = (c["q"].to(DEV), *c["pools"], c["bt"], torch.tensor(c["lens"], dtype=torch.int32, device=DEV), c["lam"].to(DEV))
    if scores is None:
        return pkv.paged_diff_decode_attention(*args, c["scale"], window, **_kw(c, r))
    return pkv.paged_diff_decode_attention_scores(*args, scores, c["scale"], window, **_kw(c, r))


def _rules(c, b, h, window, r):
    at = lambda n: 0 if r.get(n) is None else int(r[n][b])  # noqa: E731
    return dict(window=window, softcap=r.get("softcap", 0.0),
                slope=0.0 if r.get("alibi_slopes") is None else float(np.float32(r["alibi_slopes"][h])),
                doc_start=at("doc_starts"), prefix=at("prefix_lens"))


def _lam(c, b, h):
    return float(c["lam"][b, h] if c["lam"].dim() == 2 else c["lam"][h])


def _check(c, got, window=0, rows=None, **r):
    g = c["hq"] // c["hkv"]
    got = got.float().cpu().double().numpy()
    w = None if c["w"] is None else c["w"].double().numpy()
    for b, L in enumerate(c["lens"]):
        for h in range(c["hq"]):
            if rows is not None and (b, h) not in rows:
                continue
            ref, tol = diff_model.row(c["q"][b, h].double().numpy(), c["k"][b, :L, h // g], c["v"][b, :L, h // g], L - 1, c["scale"],
                                      _lam(c, b, h), w, EPS, 2.0 ** -15, **_rules(c, b, h, window, r))
            far = np.abs(got[b, h] - ref) - tol
            assert np.all(far <= 0), (b, h, float(far.max()), float(np.abs(got[b, h] - ref).max()))


def _check_scores(c, before, got, window=0, **r):
    g = c["hq"] // c["hkv"]
    before, got = before.double().numpy(), got.double().cpu().numpy()
    S = before.shape[2]
    for b, L in enumerate(c["lens"]):
        for n in range(c["hkv"]):
            hs = range(n * g, n * g + g)
            add, tol = diff_model.score([c["q"][b, h].double().numpy() for h in hs], c["k"][b, :L, n], L - 1, c["scale"],
                                        [_lam(c, b, h) for h in hs], [_rules(c, b, h, window, r) for h in hs])
            m = min(L, S)
            want = before[b, n, :m] + add[:m]
            far = np.abs(got[b, n, :m] - want) - tol[:m] - np.abs(want) * 2.0 ** -24
            assert np.all(far <= 0), (b, n, float(far.max()))


def _slopes(hq):
    return [2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]


LENS = [1, 16, 17, 100, 255, 0, 700]
RULES = {
    "none": {},
    "cap": dict(softcap=5.0),
    "alibi": dict(alibi_slopes=True),
    "window": dict(window=40),
    "window 1": dict(window=1),
    "prefix and window": dict(window=20, prefix_lens=[0, 3, 16, 33, 300, 5, 64]),
    "documents": dict(doc_starts=[0, 15, 16, 40, 255, 0, 689]),
    "nothing to see": dict(doc_starts=[1, 16, 2000, 100, 254, 0, -4]),
    "only the prefix": dict(doc_starts=[9, 99, 999, 9999, 255, 1, 700], prefix_lens=[1, 4, 17, 2, 0, 4, 333]),
    "all": dict(window=64, softcap=30.0, alibi_slopes=True, doc_starts=[0, 3, 9, 70, 100, 0, 650],
                prefix_lens=[1, 2, 3, 20, 40, 0, 100]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", RULES)
@pytest.mark.parametrize("hq,hkv,d,norm", [(8, 8, 64, True), (12, 2, 128, False), (8, 1, 64, False), (32, 8, 128, True)])
def test_rules_match_the_model(name, hq, hkv, d, norm):
    r = dict(RULES[name])
    if r.get("alibi_slopes"):
        r["alibi_slopes"] = _slopes(hq)
    c = _case(LENS, hq, hkv, d, hq + d, norm=norm, per_row=norm)
    err = pkv.new_error_word(DEV)
    got = _call(c, error_word=err, **r)
    _check(c, got, **r)
    # with the scores: the same output, and each key's weight added
    before = torch.rand((len(LENS), hkv, 720))
    scores, beside = before.to(DEV), torch.full(before.shape, 5.0, device=DEV)
    again = _call(c, scores=scores, scores_out=beside, error_word=err, **r)
    assert torch.equal(again, got) and torch.equal(scores.cpu(), before)
    _check_scores(c, before, beside, **r)
    for b, L in enumerate(LENS):
        assert (beside[b, :, L:] == 5.0).all()
    again = _call(c, scores=scores, error_word=err, **r)
    assert torch.equal(again, got)
    for b, L in enumerate(LENS):
        assert torch.equal(scores[b, :, :L], beside[b, :, :L]) and torch.equal(scores[b, :, L:].cpu(), before[b, :, L:])
    assert pkv.read_error(err) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("group", range(1, 9))
def test_every_group_size(group):
    c = _case([33, 5], 3 * group, 3, 128, group)
    r = dict(softcap=4.0, alibi_slopes=_slopes(3 * group))
    _check(c, _call(c, **r), **r)
    before = torch.rand((2, 3, 40))
    after = before.to(DEV)
    _call(c, scores=after, **r)
    _check_scores(c, before, after, **r)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[9000], [4000, 1, 7000], [2500] * 9])
def test_long_sequences_split_over_the_gpu(lens, d):
    c = _case(lens, 8, 2, d, 3)
    err = pkv.new_error_word(DEV)
    rows = {(0, 0), (0, 7), (len(lens) - 1, 3)}
    _check(c, _call(c, error_word=err), rows=rows)
    before = torch.rand((len(lens), 2, (max(lens) + 15) // 16 * 16))
    after = before.to(DEV)
    _call(c, scores=after, error_word=err)
    assert pkv.read_error(err) == 0
    c["lens"], c["q"], c["lam"] = c["lens"][:1], c["q"][:1], c["lam"][:1] if c["lam"].dim() == 2 else c["lam"]
    _check_scores(c, before[:1], after[:1])


@pytest.mark.gpu
def test_more_sequences_than_the_merge_scans():
    lens = np.random.default_rng(5).integers(0, 60, 600).tolist()
    c = _case(lens, 4, 2, 64, 5, per_row=True)
    got = _call(c)
    _check(c, got, rows={(b, h) for b in range(0, 600, 37) for h in range(4)} | {(599, 3)})


@pytest.mark.gpu
def test_one_key_alone_gives_one_minus_lambda():
    """One key: both maps are 1, y = (1 - lambda) V."""
    c = _case([1, 1], 8, 4, 64, 6, norm=False)
    got = _call(c).float().cpu()
    v = torch.from_numpy(c["v"][:, 0]).repeat_interleave(2, 1)
    want = (1 - c["lam"].double())[None, :, None] * v
    assert ((got - want).abs() <= want.abs() * 2**-8 + v.abs() * 2**-15).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), 3e38])
def test_masked_places_may_hold_anything(bad):
    """K and V outside of window, prefix and length: the output is as with other values there, bit for bit."""
    c = _case([300, 77], 4, 2, 64, 7, fill=0.0)
    r = dict(window=50, prefix_lens=[20, 0])
    want, s0 = _call(c, **r), torch.zeros((2, 2, 320), device=DEV)
    _call(c, scores=s0, **r)
    for b, (L, p) in enumerate(((300, 20), (77, 0))):
        for t in [*range(p, L - 50), *range(L, (L + 15) // 16 * 16)]:
            blk = int(c["bt"][b, t // 16])
            for pool in c["pools"]:
                pool[blk, :, t % 16] = bad
    assert torch.equal(_call(c, **r), want)
    s1 = torch.zeros_like(s0)
    _call(c, scores=s1, **r)
    assert torch.equal(s0, s1)


@pytest.mark.gpu
def test_the_halves_do_not_mix():
    """An infinity in one half of a seen K row gives that map a weight of 0 (its logit is -infinity) and leaves the other map alone."""
    c = _case([40], 4, 2, 128, 8, fill=0.0)
    blk = int(c["bt"][0, 1])
    for half in (0, 1):
        at = 64 * half + 5
        c["q"][0, :, at] = 1.0
        old = c["pools"][0][blk, :, 3].clone()
        outs = []
        for x in (-3e38, float("-inf")):
            c["pools"][0][blk, :, 3, at] = x
            outs.append(_call(c))
        c["pools"][0][blk, :, 3] = old
        assert torch.isfinite(outs[0]).all() and torch.equal(outs[0], outs[1])


@pytest.mark.gpu
def test_large_values_and_equal_maps():
    """Large scores and values; and equal halves under a factor of 1: the difference is 0 up to the weights' rounding."""
    c = _case([500, 60], 8, 2, 128, 9)
    c["q"] = (c["q"].float() * 30).bfloat16()
    _check(c, _call(c))
    c = _case([300], 4, 2, 64, 10, norm=False)
    c["q"][..., 32:] = c["q"][..., :32]
    c["pools"][0][..., 32:] = c["pools"][0][..., :32]
    c["k"][..., 32:] = c["k"][..., :32]
    c["lam"] = torch.ones(4)
    _check(c, _call(c))


@pytest.mark.gpu
def test_a_length_past_the_scores_and_bad_inputs():
    c = _case([100, 40], 4, 2, 64, 11, fill=0.0)
    err = pkv.new_error_word(DEV)
    before = torch.rand((2, 2, 70))
    after = before.to(DEV)
    got = _call(c, scores=after, error_word=err)
    assert pkv.read_error(err) == C["PKV_DEV_BAD_CONTEXT_LEN"]
    _check(c, got)
    _check_scores(c, before, after)
    good = c["lens"]
    for b, L in ((0, -1), (1, 7 * 16 + 1)):
        c["lens"] = list(good)
        c["lens"][b] = L
        err = pkv.new_error_word(DEV)
        got = _call(c, error_word=err)
        assert pkv.read_error(err) == C["PKV_DEV_BAD_CONTEXT_LEN"]
        assert not got[b].any()
    c["lens"] = good
    for x in (-1, c["pools"][0].shape[0]):
        bt = c["bt"].clone()
        c["bt"] = bt.clone()
        c["bt"][0, 2] = x
        err = pkv.new_error_word(DEV)
        got = _call(c, error_word=err)
        assert pkv.read_error(err) == C["PKV_DEV_BAD_BLOCK_ID"] and torch.isfinite(got).all()
        c["bt"] = bt
        _check(c, got, rows={(1, h) for h in range(4)})


@pytest.mark.gpu
@pytest.mark.parametrize("hq", [4, 12], ids=["pairs", "wide"])
@pytest.mark.parametrize("stride", [320, 321])
def test_keys_of_a_bad_block_get_no_weight(hq, stride):
    """After a call on the same workspace whose keys there had weights: those scores stay, bit for bit."""
    c = _case([300, 77], hq, 2, 64, 12, fill=0.0)
    err = pkv.new_error_word(DEV)
    ws = torch.zeros((pkv.diff_decode_workspace_bytes(2, hq, 2, 64, c["pools"][0].shape[0], c["bt"].shape[1], score_stride=stride),),
                     dtype=torch.uint8, device=DEV)
    before = torch.rand((2, 2, stride), device=DEV)
    _call(c, scores=before.clone(), workspace=ws, error_word=err)
    assert pkv.read_error(err) == 0
    for x in (-1, c["pools"][0].shape[0]):
        c["bt"][0, 3] = x
        after = before.clone()
        _call(c, scores=after, workspace=ws, error_word=err)
        assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_BLOCK_ID"]
        assert torch.equal(after[0, :, 48:64], before[0, :, 48:64])
        assert (after[0, :, :48] > before[0, :, :48]).all() and (after[0, :, 64:300] > before[0, :, 64:300]).all()


@pytest.mark.gpu
def test_inputs_ready_streams_graphs_and_one_workspace():
    cases = [_case([300, 2, 1000], 8, 2, 128, s) for s in (12, 13)]
    want = [_call(c) for c in cases]
    n = pkv.diff_decode_workspace_bytes(3, 8, 2, 128, cases[0]["pools"][0].shape[0], 63, score_stride=1008)
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    for c, w in zip(cases * 2, want * 2):   # one workspace, calls one after another
        assert torch.equal(_call(c, workspace=ws, inputs_ready=True), w)
        scores = torch.zeros((3, 2, 1008), device=DEV)
        assert torch.equal(_call(c, workspace=ws, scores=scores, inputs_ready=True), w)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = _call(cases[0], stream=side)
    side.synchronize()
    assert torch.equal(got, want[0])
    out = torch.empty_like(want[0])
    lens = torch.tensor(cases[0]["lens"], dtype=torch.int32, device=DEV)
    q, lam, w = cases[0]["q"].to(DEV), cases[0]["lam"].to(DEV), cases[0]["w"].to(DEV)
    scores = torch.zeros((3, 2, 1008), device=DEV)
    c = cases[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_diff_decode_attention_scores(q, *c["pools"], c["bt"], lens, lam, scores, c["scale"], norm_weight=w, norm_eps=EPS,
                                               out=out, workspace=ws)
    scores.zero_()
    for i in range(1, 4):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0])
    once = torch.zeros_like(scores)
    _call(c, scores=once)
    for b, L in enumerate(c["lens"]):
        assert torch.allclose(scores[b, :, :L], 3 * once[b, :, :L], rtol=2**-22, atol=0)
    lens[0] = 5
    q.copy_(torch.randn(q.shape, device=DEV))
    graph.replay()
    torch.cuda.synchronize()
    c = dict(c, lens=[5, 2, 1000], q=q.cpu())
    _check(c, out)


@pytest.mark.gpu
def test_guard_bands():
    c = _case([90, 33], 4, 2, 64, 14)
    pad = 256

    def inside(shape, dtype, fill):
        n = int(np.prod(shape))
        big = torch.full((n + 2 * pad,), fill, dtype=dtype, device=DEV)
        return big, big[pad:pad + n].view(shape)

    n = pkv.diff_decode_workspace_bytes(2, 4, 2, 64, c["pools"][0].shape[0], c["bt"].shape[1], score_stride=96)
    ws, out, sc = inside((n,), torch.uint8, 0), inside((2, 4, 64), torch.bfloat16, 3), inside((2, 2, 96), torch.float32, 3)
    ws[0][:pad] = ws[0][pad + n:] = 3
    _call(c, scores=sc[1], out=out[1], workspace=ws[1])
    torch.cuda.synchronize()
    for big, t in (ws, out, sc):
        assert (big[:pad] == 3).all() and (big[pad + t.numel():] == 3).all()
    _check(c, out[1])


# ------------------------------------------------------------------------------------- refusals (no GPU)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_mapped_gb300 import _build
    _build.build()
    return _lib.load()


def test_header_is_exported(lib):
    names = _lib.header_functions(_lib.DIFF_HEADER)
    assert "pkv_paged_diff_decode_attention" in names and "pkv_paged_diff_decode_attention_scores" in names
    for n in names:
        assert hasattr(lib, n), n


def test_host_validation_codes(lib):
    P = ctypes.c_void_p

    def dims(B=4, hq=32, hkv=8, d=128, bs=16, nb=1000, mb=64):
        return ctypes.byref(_lib.PkvDims(B, hq, hkv, d, bs, nb, mb))

    def params(lam=0x10000, rows=0, eps=1e-5, w=0x10000):
        return ctypes.byref(_lib.PkvDiffParams(lam, rows, eps, w))

    def decode(p=None, r=None, d=None, ws=16, flags=0, out=0x10000):
        return lib.pkv_paged_diff_decode_attention(P(out), P(0x10000), P(0x10000), P(0x10000), P(0x10000), P(0x10000), 0.1,
                                                   params() if p is None else p, r, P(0x20000), ws, dims() if d is None else d, flags,
                                                   None, None)

    def scores(sc=0x10000, so=0x10000, stride=64, ws=16, d=None):
        return lib.pkv_paged_diff_decode_attention_scores(P(0x10000), P(sc), P(so), stride, P(0x10000), P(0x10000), P(0x10000),
                                                          P(0x10000), P(0x10000), 0.1, params(), None, P(0x20000), ws,
                                                          dims() if d is None else d, 0, None, None)

    assert decode(params(lam=None)) == C["PKV_ERR_NULL_POINTER"] and decode(params(rows=2)) == C["PKV_ERR_ARGUMENT"]
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert decode(params(eps=eps)) == C["PKV_ERR_ARGUMENT"], eps
        assert decode(params(eps=eps, w=None)) == C["PKV_ERR_WORKSPACE"]
    assert decode(params(lam=0x10002)) == decode(params(w=0x10001)) == decode(out=0x10008) == C["PKV_ERR_ALIGNMENT"]
    assert decode() == C["PKV_ERR_WORKSPACE"] and decode(flags=2) == C["PKV_ERR_ARGUMENT"]
    assert decode(d=dims(hq=32, hkv=2)) == C["PKV_ERR_GQA"] and decode(d=dims(d=96)) == C["PKV_ERR_HEAD_DIM"]
    assert decode(d=dims(bs=8)) == C["PKV_ERR_BLOCK_SIZE"] and decode(d=dims(B=0)) == C["PKV_OK"]
    assert decode(r=ctypes.byref(_lib.PkvScoreRules(-1.0, 0, None, None, None))) == C["PKV_ERR_ARGUMENT"]
    assert scores(sc=None) == scores(so=None) == C["PKV_ERR_NULL_POINTER"] and scores(stride=0) == C["PKV_ERR_DIMS"]
    assert scores(so=0x10002) == C["PKV_ERR_ALIGNMENT"] and scores() == C["PKV_ERR_WORKSPACE"]
    n, m = lib.pkv_diff_decode_workspace_bytes(dims(), 0), lib.pkv_diff_decode_workspace_bytes(dims(), 1000)
    assert n >= 2 * lib.pkv_decode_workspace_bytes(dims()) - 4096 and m >= n + 2 * 4 * 32 * 4 * 1001 and m % 256 == 0
    for bad in (dims(d=96), dims(hq=30), dims(bs=8), dims(B=-1)):
        assert lib.pkv_diff_decode_workspace_bytes(bad, 0) == 0
    assert lib.pkv_diff_decode_workspace_bytes(dims(), -1) == 0
    # room for the partials, none for the logits
    assert scores(ws=n, stride=1 << 20) == C["PKV_ERR_WORKSPACE"]


def test_binding_refusals():
    q, kc = torch.zeros(2, 8, 64).bfloat16(), torch.zeros(4, 8, 16, 64).bfloat16()
    bt, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_diff_decode_attention(q, kc, kc, bt, lens, torch.ones(8), 0.125)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_diff_decode_attention_scores(q, kc, kc, bt, lens, torch.ones(8), torch.zeros(2, 8, 32), 0.125)
    with pytest.raises(TypeError):
        pkv.paged_diff_decode_attention_scores(q, kc, kc, bt, lens, torch.ones(8), None, 0.125)
    ok = (4, 32, 8, 128, 1000, 64)
    assert pkv.diff_decode_workspace_bytes(*ok) > 0
    for at in range(len(ok)):
        for x in (2**32 + ok[at], 2**31, -1):
            with pytest.raises(ValueError):
                pkv.diff_decode_workspace_bytes(*ok[:at], x, *ok[at + 1:])
    for x in (-1, 2**31, 2**32 + 4):
        with pytest.raises(ValueError):
            pkv.diff_decode_workspace_bytes(*ok, score_stride=x)


@pytest.mark.gpu
def test_binding_refuses_wrong_shapes_and_types():
    c = _case([20, 33], 8, 2, 64, 15)
    q, lens, lam, w = c["q"].to(DEV), torch.tensor(c["lens"], dtype=torch.int32, device=DEV), c["lam"].to(DEV), c["w"].to(DEV)
    starts = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    sc = torch.zeros(2, 2, 48, device=DEV)

    def decode(q=q, bt=c["bt"], lens=lens, lam=lam, **kw):
        kw = dict(dict(norm_weight=w), **kw)
        return pkv.paged_diff_decode_attention(q, *c["pools"], bt, lens, lam, 0.2, **kw)

    def prefill(lam=lam, **kw):
        return pkv.paged_diff_prefill_attention(q, *c["pools"], c["bt"], lens, starts, lam, 0.2, **dict(dict(norm_weight=w), **kw))

    def scores(sc=sc, **kw):
        return pkv.paged_diff_decode_attention_scores(q, *c["pools"], c["bt"], lens, lam, sc, 0.2, **kw)

    for call in (decode, prefill):
        for bad in (lam[:7], lam[None], torch.zeros(3, 8, device=DEV), torch.zeros(2, 7, device=DEV), torch.zeros(2, 2, 8, device=DEV)):
            with pytest.raises(ValueError):
                call(lam=bad)
        for bad in (lam.double(), 0.5, None):
            with pytest.raises(TypeError):
                call(lam=bad)
        for eps in (0.0, -1.0, float("nan"), float("inf"), 1e-50, 1e300):
            with pytest.raises(ValueError, match="norm_eps"):
                call(norm_eps=eps)
        for kw in (dict(norm_weight=w[:32]), dict(out=torch.empty_like(q[:1])), dict(out=q.permute(1, 0, 2)), dict(softcap=-1.0),
                   dict(alibi_slopes=lam[:3].clone()), dict(workspace=torch.zeros(16, dtype=torch.uint8))):
            with pytest.raises(ValueError):
                call(**kw)
        with pytest.raises(pkv.PkvError):
            call(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
    for kw in (dict(q=q[:, :, :32].contiguous()), dict(bt=c["bt"][:1]), dict(lens=lens[:1])):
        with pytest.raises(ValueError):
            decode(**kw)
    for kw in (dict(sc=sc[:1]), dict(sc=sc[:, :1].contiguous()), dict(sc=sc[0]), dict(scores_out=sc[:, :, :40].contiguous()), dict(sc=sc.cpu())):
        with pytest.raises(ValueError):
            scores(**kw)
    with pytest.raises(pkv.PkvError):   # rows of no slots
        scores(sc=sc[:, :, :0].contiguous())
