"""Decode attention with score rules over bf16 and FP8 pools against the 64-bit model: caps, distance
bias, windows, documents and prefixes, alone and together, over every group size, both head sizes and
lengths from 0 up; rows that see nothing; NaN and infinities in what is masked; equality with the plain
decode where no rule applies; the inputs-ready flag, other streams, graphs; refusals."""
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


def _case(lens, hq, hkv, d, seed, f8, fill=None, vscale=0):
    g = torch.Generator().manual_seed(seed)
    B, lmax = len(lens), max(max(lens), 1)
    q = rand_bf16((B, hq, d), g)
    nb = sum((L + 15) // 16 for L in lens) + 3
    if not f8:
        k, v = rand_bf16((B, lmax, hkv, d), g), rand_bf16((B, lmax, hkv, d), g)
        kc, vc, bt = paged_from_contiguous(k, v, lens, nb, g, fill=fill)
        pools = [kc, vc]
        k, v = k.double().numpy(), v.double().numpy()
    else:
        # random codes; blocks' scales a few binades apart.  Rows past a sequence hold `fill` (a NaN code)
        pools, vals = [], []
        zero, one = torch.zeros((B, lmax, hkv, d)).bfloat16(), torch.ones((B, lmax, hkv, d)).bfloat16()
        live, _, bt = paged_from_contiguous(one, zero, lens, nb, g, fill=0.0)
        for spread in (3, 3 + vscale):
            codes = (torch.randn((nb, hkv, 16, d), generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
            e = torch.randint(-8, -8 + spread, (nb, hkv), generator=g).float()
            scales = torch.exp2(e) * (1 + torch.rand((nb, hkv), generator=g) * (seed % 2))
            x = codes.double().numpy() * scales.double().numpy()[:, :, None, None]
            if fill is not None:
                b8 = codes.view(torch.uint8)
                b8[live == 0] = 0x7F
            pools += [codes, scales]
            w = np.zeros((B, lmax, hkv, d))
            for b, L in enumerate(lens):
                for t in range(L):
                    w[b, t] = x[int(bt[b, t // 16]), :, t % 16]
            vals.append(w)
        k, v = vals
    return dict(q=q, k=k, v=v, pools=[p.to(DEV) for p in pools], bt=bt.to(DEV), lens=list(lens), f8=f8,
                scale=d ** -0.5, hq=hq, hkv=hkv, d=d)


def _call(c, window=0, out=None, ws=None, err=None, inputs_ready=False, stream=None, **rules):
    dev_rules = {n: None if rules.get(n) is None else torch.as_tensor(rules[n], dtype=t, device=DEV)
                 for n, t in (("alibi_slopes", torch.float32), ("doc_starts", torch.int32), ("prefix_lens", torch.int32))}
    kw = dict(softcap=rules.get("softcap", 0.0), out=out, workspace=ws, error_word=err, inputs_ready=inputs_ready, stream=stream,
              **dev_rules)
    q, lens = c["q"].to(DEV), torch.tensor(c["lens"], dtype=torch.int32, device=DEV)
    if c["f8"]:
        kc, ks, vc, vs = c["pools"]
        return pkv.paged_decode_attention_f8(q, kc, vc, ks, vs, c["bt"], lens, c["scale"], window, **kw)
    return pkv.paged_decode_attention_rules(q, *c["pools"], c["bt"], lens, c["scale"], window, **kw)


def _check(c, got, window=0, rows=None, **r):
    g = c["hq"] // c["hkv"]
    got = got.float().cpu().double().numpy()
    eps = 2.0 ** -11 if c["f8"] else 2.0 ** -15  # weights: one fp16 term, or a bf16 pair
    for b, L in enumerate(c["lens"]):
        for h in range(c["hq"]):
            if rows is not None and (b, h) not in rows:
                continue
            at = lambda n: 0 if r.get(n) is None else r[n][b]  # noqa: E731
            ref, mass, size = rules_model.row(
                c["q"][b, h].double().numpy(), c["k"][b, :L, h // g], c["v"][b, :L, h // g], L - 1, c["scale"], window,
                r.get("softcap", 0.0), 0.0 if r.get("alibi_slopes") is None else float(np.float32(r["alibi_slopes"][h])),
                at("doc_starts"), at("prefix_lens"))
            far = np.abs(got[b, h] - ref) - rules_model.bound(ref, mass, size, c["d"], eps)
            assert np.all(far <= 0), (b, h, float(far.max()))


def _slopes(hq):
    return [2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]


LENS = [1, 16, 17, 100, 255, 0, 700]
RULES = {
    "cap": dict(softcap=5.0),
    "alibi": dict(alibi_slopes=True),
    "window": dict(window=40),
    "window 1": dict(window=1),
    "prefix and window": dict(window=20, prefix_lens=[0, 3, 16, 33, 300, 5, 64]),
    "prefix at the window": dict(window=100, prefix_lens=[1, 1, 1, 1, 155, 1, 599]),
    "prefix into the window's block": dict(window=90, prefix_lens=[1, 1, 1, 10, 161, 1, 605]),
    "documents": dict(doc_starts=[0, 15, 16, 40, 255, 0, 689]),
    "nothing to see": dict(doc_starts=[1, 16, 2000, 100, 254, 0, -4]),
    "only the prefix": dict(doc_starts=[9, 99, 999, 9999, 255, 1, 700], prefix_lens=[1, 4, 17, 2, 0, 4, 333]),
    "all": dict(window=64, softcap=30.0, alibi_slopes=True, doc_starts=[0, 3, 9, 70, 100, 0, 650],
                prefix_lens=[1, 2, 3, 20, 40, 0, 100]),
    "negative": dict(prefix_lens=[-1, -5, -99, -1, -1, -1, -1], window=-3),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", RULES)
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 8, 64), (12, 2, 128), (8, 1, 64), (32, 8, 128)])
def test_rules_match_the_model(name, f8, hq, hkv, d):
    r = dict(RULES[name])
    if r.get("alibi_slopes"):
        r["alibi_slopes"] = _slopes(hq)
    c = _case(LENS, hq, hkv, d, hq + d, f8, fill=float("nan"))
    err = pkv.new_error_word(DEV)
    got = _call(c, err=err, **r)
    assert pkv.read_error(err) == 0
    _check(c, got, **r)


@pytest.mark.gpu
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("group", range(1, 9))
def test_every_group_size(f8, group):
    c = _case([33, 5], 3 * group, 3, 128, group, f8)
    r = dict(softcap=4.0, alibi_slopes=_slopes(3 * group))
    _check(c, _call(c, **r), **r)


@pytest.mark.gpu
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
def test_long_ragged_batch(f8, d):
    """Rows split over many workers and merged, with prefixes far from their windows."""
    lens = [9000, 1, 4000, 12345, 64, 3001]
    c = _case(lens, 8, 2, d, 5, f8)
    r = dict(window=2500, softcap=20.0, alibi_slopes=_slopes(8), prefix_lens=[1000, 0, 17, 333, 64, 3000])
    err = pkv.new_error_word(DEV)
    got = _call(c, err=err, **r)
    assert pkv.read_error(err) == 0
    _check(c, got, rows={(b, h) for b in range(6) for h in (b, 7 - b)}, **r)


@pytest.mark.gpu
def test_block_scales_far_apart():
    """FP8 blocks whose V scales differ by up to 2^40: small blocks matter only where large ones are not seen."""
    c = _case([300, 40, 17], 8, 2, 128, 8, True, vscale=40)
    _check(c, _call(c))
    _check(c, _call(c, window=20), window=20)


@pytest.mark.gpu
def test_large_caps_leave_the_scores():
    """A cap far above the scores changes nothing beyond their own rounding."""
    c = _case([100, 700], 4, 2, 64, 9, False)
    for cap in (1e4, 1e8, 1e30):
        _check(c, _call(c, softcap=cap), softcap=cap)
    _check(c, _call(c, softcap=1e-30), softcap=1e-30)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_no_rule_equals_the_plain_decode(d):
    c = _case([1, 40, 1000, 4097, 0], 8, 2, d, 11, False)
    lens = torch.tensor(c["lens"], dtype=torch.int32, device=DEV)
    for window in (0, 50):
        want = pkv.paged_decode_attention(c["q"].to(DEV), *c["pools"], c["bt"], lens, c["scale"], window)
        assert torch.equal(_call(c, window=window), want)


@pytest.mark.gpu
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
def test_masked_infinities_stay_out(f8):
    """Keys outside the window, before the document or past the length hold NaN and infinities."""
    c = _case([100, 37], 4, 2, 64, 13, f8)
    want = _call(c, window=10, prefix_lens=[3, 3])
    bt = c["bt"].cpu()
    for b, L in enumerate(c["lens"]):
        for t in range(((L + 15) // 16) * 16):
            if 3 <= t < L - 10 or t >= L:
                blk = int(bt[b, t // 16])
                for p in (c["pools"] if not f8 else (c["pools"][0], c["pools"][2])):
                    if f8:
                        p.view(torch.uint8)[blk, :, t % 16] = 0xFF if t % 2 else 0x7F
                    else:
                        p[blk, :, t % 16] = (float("nan"), float("inf"), -float("inf"))[t % 3]
    assert torch.equal(_call(c, window=10, prefix_lens=[3, 3]), want)


@pytest.mark.gpu
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
def test_flag_stream_graph_and_one_workspace(f8):
    """Three layers back to back on one workspace: eager, declared ready, on another stream and in a
    replayed graph, bit for bit the same; rows of the output past the batch stay."""
    cs = [_case([500, 77, 3000], 8, 2, 128, 20 + i, f8) for i in range(3)]
    r = dict(window=600, softcap=15.0, prefix_lens=[32, 8, 100])
    want = [_call(c, **r) for c in cs]
    nb = max(c["pools"][0].shape[0] for c in cs)
    ws = torch.zeros(pkv.decode_workspace_bytes(3, 8, 2, 128, nb, cs[0]["bt"].shape[1]), dtype=torch.uint8, device=DEV)
    prefix = torch.tensor(r["prefix_lens"], dtype=torch.int32, device=DEV)
    lens = torch.tensor(cs[0]["lens"], dtype=torch.int32, device=DEV)
    qs = [c["q"].to(DEV) for c in cs]
    outs = [torch.empty_like(q) for q in qs]

    def layers(ready):
        for c, q, o in zip(cs, qs, outs):
            kw = dict(softcap=15.0, prefix_lens=prefix, out=o, workspace=ws, inputs_ready=ready)
            if f8:
                kc, ks, vc, vs = c["pools"]
                pkv.paged_decode_attention_f8(q, kc, vc, ks, vs, c["bt"], lens, c["scale"], 600, **kw)
            else:
                pkv.paged_decode_attention_rules(q, *c["pools"], c["bt"], lens, c["scale"], 600, **kw)

    def same():
        torch.cuda.synchronize()
        ok = all(torch.equal(o, w) for o, w in zip(outs, want))
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        return ok

    for ready in (False, True):
        layers(ready)
        assert same()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        layers(True)
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layers(True)
    for _ in range(2):
        g.replay()
        assert same()


@pytest.mark.gpu
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
def test_device_errors(f8):
    r = dict(window=9, prefix_lens=[20, 20])
    c = _case([50, 60], 4, 2, 128, 30, f8)
    good = _call(c, **r)
    err = pkv.new_error_word(DEV)
    c["bt"][1, 0] = c["pools"][0].shape[0]
    got = _call(c, err=err, **r)
    assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_BLOCK_ID"] and torch.equal(got[0], good[0])
    c["bt"][1, 0] = 0
    c["lens"] = [50, 5000]
    got = _call(c, err=err, **r)
    assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_CONTEXT_LEN"] and torch.equal(got[0], good[0])
    assert not got[1].any()


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_mapped_gb300 import _build
    _build.build()
    return _lib.load()


def test_step_header_is_exported(lib):
    names = _lib.header_functions(_lib.STEP_HEADER)
    assert "pkv_kv_step_tables" in names and "pkv_paged_decode_attention_f8" in names
    for n in names:
        assert hasattr(lib, n), n


def test_host_validation_codes(lib):
    P = ctypes.c_void_p

    def dims(B=4, hq=32, hkv=8, d=128, bs=16, nb=1000, mb=64):
        return ctypes.byref(_lib.PkvDims(B, hq, hkv, d, bs, nb, mb))

    def rules(cap=0.0, slopes=None, docs=None, prefix=None):
        return ctypes.byref(_lib.PkvScoreRules(cap, 0, slopes, docs, prefix))

    def decode(r=None, d=None, ws=16, flags=0, out=0x10000):
        return lib.pkv_paged_decode_attention_rules(P(out), P(0x10000), P(0x10000), P(0x10000), P(0x10000), P(0x10000),
                                                    0.1, rules() if r is None else r, P(0x20000), ws,
                                                    dims() if d is None else d, flags, None, None)

    def f8(ks=0x30000, r=None, d=None):
        return lib.pkv_paged_decode_attention_f8(P(0x10000), P(0x10000), P(0x10000), P(0x10000), P(ks), P(0x30000),
                                                 P(0x10000), P(0x10000), 0.1, r, P(0x20000), 16,
                                                 dims() if d is None else d, 0, None, None)

    for cap in (-1.0, float("nan"), float("inf"), 1e-31, 1e31):
        assert decode(rules(cap)) == C["PKV_ERR_ARGUMENT"], cap
        assert f8(r=rules(cap)) == C["PKV_ERR_ARGUMENT"], cap
    assert decode(rules(slopes=0x30002)) == C["PKV_ERR_ALIGNMENT"]
    assert decode(rules(docs=0x30001)) == C["PKV_ERR_ALIGNMENT"]
    assert decode() == C["PKV_ERR_WORKSPACE"] and f8() == C["PKV_ERR_WORKSPACE"]
    assert f8(r=rules(3.0)) == C["PKV_ERR_WORKSPACE"]
    assert decode(flags=2) == C["PKV_ERR_ARGUMENT"] and decode(out=0x10008) == C["PKV_ERR_ALIGNMENT"]
    assert decode(d=dims(hq=32, hkv=2)) == C["PKV_ERR_GQA"] and f8(d=dims(d=96)) == C["PKV_ERR_HEAD_DIM"]
    assert f8(ks=None) == C["PKV_ERR_NULL_POINTER"] and f8(ks=0x30002) == C["PKV_ERR_ALIGNMENT"]
    assert decode(d=dims(B=0)) == C["PKV_OK"] and f8(d=dims(B=0)) == C["PKV_OK"]
    assert lib.pkv_paged_decode_attention_rules(P(16), P(16), P(16), P(16), P(16), P(16), 0.1, None, P(16), 16, dims(), 0,
                                                None, None) == C["PKV_ERR_NULL_POINTER"]

    def append(n=4, ks=0x30000, k=0x10000):
        return lib.pkv_kv_append_f8(P(0x10000), P(0x10000), P(ks), P(0x30000), P(k), P(0x10000), P(0x10000), n, dims(), None, None)

    assert append(0) == C["PKV_OK"] and append(-1) == C["PKV_ERR_DIMS"] and append(1 << 40) == C["PKV_ERR_DIMS"]
    assert append(ks=None) == C["PKV_ERR_NULL_POINTER"] and append(ks=0x30002) == C["PKV_ERR_ALIGNMENT"]
    assert append(k=0x10008) == C["PKV_ERR_ALIGNMENT"]

    def tables(T=8, d=None, bt=0x10000, slots=0x10000):
        return lib.pkv_kv_step_tables(P(bt), P(0x10000), P(0x10000), P(slots), P(0x10000), P(0x10000), P(0x10000), P(0x10000),
                                      P(0x10000), P(0x10000), T, dims() if d is None else d, None, None)

    assert tables(-1) == C["PKV_ERR_ARGUMENT"] and tables(C["PKV_MAX_STEP_TOKENS"] + 1) == C["PKV_ERR_ARGUMENT"]
    assert tables(d=dims(B=4097)) == C["PKV_ERR_DIMS"] and tables(d=dims(bs=8)) == C["PKV_ERR_BLOCK_SIZE"]
    assert tables(d=dims(mb=1 << 28)) == C["PKV_ERR_DIMS"]
    assert tables(bt=None) == C["PKV_ERR_NULL_POINTER"] and tables(slots=None) == C["PKV_ERR_NULL_POINTER"]


def test_binding_refuses_cpu_tensors_and_bad_rules():
    q, kc = torch.zeros(2, 8, 64).bfloat16(), torch.zeros(4, 8, 16, 64).bfloat16()
    bt, lens = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.paged_decode_attention_rules(q, kc, kc, bt, lens, 0.125)
    from paged_kv_cache_mapped_gb300 import step
    for cap in (-1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError, match="softcap"):
            step._rules(cap, 0, None, None, None, 8, 2, 2, None)
