"""The serving-step operators at their edges: guard bands around everything that they write, packed
ranges that are not ascending, the shares that the prefill's plan cuts when there are more items than
the GPU runs at once, scales and caps at the ends of their range, calls on a stream of their own, two
captured graphs, and refusals of workspaces and addresses."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
import test_gpu_decode_rules as decode
import test_gpu_prefill_attention as prefill
from helpers import paged_from_contiguous, rand_bf16
from paged_kv_cache_mapped_gb300 import _lib, header_constants
from test_gpu_guard_bands import Guarded, _check

C = header_constants()
DEV = torch.device("cuda:0")


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.mark.gpu
@pytest.mark.parametrize("B,T", [(5, 90), (5, 2500), (2500, 2500)])
def test_step_tables_write_inside_their_arrays(B, T):
    mb, nb = 64, 2 * B + 200
    new = np.zeros(B, dtype=np.int32)
    new[:5] = [33, -1, 1, min(T - 55, 900), 20]
    lens = np.zeros(B, dtype=np.int32)
    lens[:3] = [15, 40, 16]
    bt = Guarded((B, mb), torch.int32, init=-1)
    bt.t[0, 0], bt.t[2, 0] = 0, 1
    bt.t[1, :3] = _i32([2, 3, 4])
    free = Guarded((nb,), torch.int32, init=-1)
    free.t[:nb - 5] = torch.arange(5, nb, device=DEV, dtype=torch.int32)
    lo, st, sl, po, co = (Guarded(s, t) for s, t in (((B,), torch.int32), ((B + 1,), torch.int32), ((T,), torch.int64),
                                                     ((T,), torch.int32), ((1,), torch.int32)))
    err = pkv.new_error_word(DEV)
    for count in (nb - 5, nb + 1):  # the second is refused
        pkv.kv_step_tables(bt.t, _i32(lens), _i32(new), free.t, _i32([count]), T, context_lens_out=lo.t, free_count_out=co.t,
                           query_starts=st.t, slot_mapping=sl.t, positions=po.t, error_word=err)
        assert pkv.read_error(err, clear=True) == (0 if count < nb else C["PKV_DEV_NO_BLOCKS"])
    _check(("tables", bt), ("free", free), ("lengths", lo), ("starts", st), ("slots", sl), ("positions", po), ("count", co))


@pytest.mark.gpu
@pytest.mark.parametrize("d,hq,hkv", [(128, 16, 2), (64, 5, 5)])
def test_attention_and_fp8_calls_write_inside_their_arrays(d, hq, hkv):
    lens, new = [700, 3, 0, 1200, 257], [150, 3, 0, 1, 257]
    c = prefill._case(lens, new, hq, hkv, d, 21, pad=9)
    B, T, nb, mb = 5, c["q"].shape[0], c["pools"][0].shape[0], c["bt"].shape[1]
    rules = dict(softcap=4.0, prefix_lens=[3, 0, 9, 40, 300], alibi_slopes=prefill._slopes(hq), doc_starts=np.arange(T) % 7)
    err = pkv.new_error_word(DEV)
    pools = [Guarded(p.shape, torch.bfloat16, init=p) for p in c["pools"]]
    c["pools"] = [p.t for p in pools]
    out = Guarded((T, hq, d), torch.bfloat16)
    ws = Guarded((pkv.prefill_workspace_bytes(T, B, hq, hkv, d, nb, mb),), torch.uint8)
    for r in ({}, rules):
        prefill._call(c, window=90 if r else 0, out=out.t, workspace=ws.t, error_word=err, **r)
    dout = Guarded((B, hq, d), torch.bfloat16)
    dws = Guarded((pkv.decode_workspace_bytes(B, hq, hkv, d, nb, mb),), torch.uint8, init=0)
    pkv.paged_decode_attention_rules(c["q"][:B].to(DEV), *c["pools"], c["bt"], _i32(lens), 0.1, 90, softcap=4.0,
                                     prefix_lens=_i32([3, 0, 9, 40, 300]), out=dout.t, workspace=dws.t, error_word=err)
    codes = [Guarded((nb, hkv, 16, d), torch.float8_e4m3fn, init=torch.zeros((nb, hkv, 16, d)).to(torch.float8_e4m3fn)) for _ in range(2)]
    scales = [Guarded((nb, hkv), torch.float32, init=0) for _ in range(2)]
    slots = np.concatenate([[int(c["bt"][b, t // 16]) * 16 + t % 16 for t in range(L)] for b, L in enumerate(lens)]).astype(np.int64)
    g = torch.Generator().manual_seed(5)
    rows = [rand_bf16((len(slots), hkv, d), g).to(DEV) for _ in range(2)]
    pkv.kv_append_f8(codes[0].t, codes[1].t, scales[0].t, scales[1].t, *rows, torch.from_numpy(slots).to(DEV), error_word=err)
    pkv.paged_decode_attention_f8(c["q"][:B].to(DEV), codes[0].t, codes[1].t, scales[0].t, scales[1].t, c["bt"], _i32(lens), 0.1,
                                  out=dout.t, workspace=dws.t, error_word=err)
    assert pkv.read_error(err) == 0
    _check(("out", out), ("workspace", ws), ("decode out", dout), ("decode workspace", dws),
           *(("pool", p) for p in pools + codes + scales))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 300])
def test_starts_that_are_not_ascending(n):
    """Ranges that lie over one another: only those above every start before them are taken, the others'
    rows stay as they were, and nothing lands outside the workspace and the output."""
    B, hq, hkv, d = 96, 4, 2, 64
    c = prefill._case([n + 20] + [1] * (B - 1), [n] + [0] * (B - 1), hq, hkv, d, 22)
    c["lens"] = [n + 20] * B
    c["bt"] = c["bt"][:1].expand(B, -1).contiguous()
    good = prefill._call(dict(c, starts=np.array([0] + [n] * B, dtype=np.int32)))
    err = pkv.new_error_word(DEV)
    out = Guarded((n, hq, d), torch.bfloat16)
    ws = Guarded((pkv.prefill_workspace_bytes(n, B, hq, hkv, d, c["pools"][0].shape[0], c["bt"].shape[1]),), torch.uint8)
    # every other sequence has all rows, then every sequence a range below the first's end
    for starts in (np.arange(B + 1) % 2 * n, np.array([0, n] + [0, 1] * B)[:B + 1]):
        out.t.fill_(3.0)
        c["starts"] = starts.astype(np.int32)
        prefill._call(c, out=out.t, workspace=ws.t, error_word=err)
        assert pkv.read_error(err, clear=True) == C["PKV_DEV_BAD_QUERY_RANGE"]
        assert torch.equal(out.t, good)
        _check(("out", out), ("workspace", ws))
    c["starts"] = (n - np.arange(B + 1) % 2 * n).astype(np.int32)  # n, 0, n, ..: all below the first start
    out.t.fill_(3.0)
    prefill._call(c, out=out.t, workspace=ws.t, error_word=err)
    assert pkv.read_error(err) == C["PKV_DEV_BAD_QUERY_RANGE"] and bool((out.t == 3.0).all())
    _check(("out", out), ("workspace", ws))


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new", [([1500] * 20, 1), ([3000, 2900] + [90] * 18, 1), ([1500] * 20, 300), ([3000, 90] * 10, 90)],
                         ids=["tail of single tokens", "two long of many", "tail of chunks", "uneven chunks"])
def test_more_items_than_run_at_once(lens, new):
    """16 kv heads and 20 sequences: more items than CTAs, the last of equal ones and the longest of uneven
    ones in shares."""
    c = prefill._case(lens, [new] * 20, 16, 16, 64, 23)
    for r in ({}, dict(softcap=6.0, prefix_lens=[7] * 20)):
        err = pkv.new_error_word(DEV)
        got = prefill._call(c, error_word=err, **r)
        assert pkv.read_error(err) == 0
        T = 20 * new
        prefill._check(c, got, rows=[(r_, h) for r_ in {0, 1, new, T // 2, T - new - 1, T - 2, T - 1} for h in (0, 7, 15)], **r)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.0, -0.09, 1e-20])
@pytest.mark.parametrize("r", [{}, dict(softcap=2.0), dict(alibi_slopes=True)], ids=["plain", "cap", "slopes"])
def test_scales_of_either_sign(scale, r):
    c = prefill._case([900, 130], [140, 130], 4, 2, 64, 24)
    c["scale"] = scale
    prefill._run(c, **({"alibi_slopes": prefill._slopes(4)} if "alibi_slopes" in r else r))


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [1e-30, 1e-3, 1e30])
def test_caps_at_the_ends_of_their_range(softcap):
    c = prefill._case([900, 130], [140, 130], 4, 2, 64, 25)
    prefill._run(c, softcap=softcap)
    c["pools"][0].nan_to_num_(nan=0.0).mul_(0)  # every score 0: the mean of V
    c["k"] = c["k"] * 0
    prefill._run(c, softcap=softcap)


@pytest.mark.gpu
def test_a_window_past_any_length_hides_nothing():
    c = prefill._case([300, 40], [30, 1], 4, 2, 64, 26)
    want = prefill._call(c)
    lens = _i32(c["lens"])
    q = c["q"][:2].to(DEV)
    base = pkv.paged_decode_attention_rules(q, *c["pools"], c["bt"], lens, c["scale"])
    for window in (2**31 - 1, 2**31, 2**40):
        assert torch.equal(prefill._call(c, window=window), want)
        assert torch.equal(pkv.paged_decode_attention_rules(q, *c["pools"], c["bt"], lens, c["scale"], window), base)


@pytest.mark.gpu
def test_a_stream_given_to_the_call():
    """Outputs and workspaces that a call makes itself belong to the stream that it is given: memory handed
    out on the current stream meanwhile is not theirs."""
    c = prefill._case([2000, 90], [70, 90], 8, 2, 128, 27)
    q, starts, lens = c["q"].to(DEV), torch.from_numpy(c["starts"]).to(DEV), _i32(c["lens"])
    s = torch.cuda.Stream()
    want = pkv.paged_prefill_attention(q, *c["pools"], c["bt"], lens, starts, c["scale"])
    want_d = pkv.paged_decode_attention_rules(q[:2], *c["pools"], c["bt"], lens, c["scale"], 50)
    torch.cuda.synchronize()
    n = pkv.prefill_workspace_bytes(160, 2, 8, 2, 128, c["pools"][0].shape[0], c["bt"].shape[1])
    m = pkv.decode_workspace_bytes(2, 8, 2, 128, c["pools"][0].shape[0], c["bt"].shape[1])
    for _ in range(20):
        got = pkv.paged_prefill_attention(q, *c["pools"], c["bt"], lens, starts, c["scale"], stream=s)
        noise = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
        got_d = pkv.paged_decode_attention_rules(q[:2], *c["pools"], c["bt"], lens, c["scale"], 50, stream=s)
        noise_d = torch.full((m,), 255, dtype=torch.uint8, device=DEV)
        s.synchronize()
        assert torch.equal(got, want) and torch.equal(got_d, want_d)
        del noise, noise_d


@pytest.mark.gpu
def test_two_graphs_with_workspaces_of_their_own():
    cs = [prefill._case([3000, 700], [3, 200], 8, 2, 128, 28 + i) for i in range(2)]
    ins, graphs, outs = [], [], []
    for c in cs:
        x = [c["q"].to(DEV), *c["pools"], c["bt"], _i32(c["lens"]), torch.from_numpy(c["starts"]).to(DEV)]
        ws = torch.empty(pkv.prefill_workspace_bytes(203, 2, 8, 2, 128, x[1].shape[0], x[3].shape[1]), dtype=torch.uint8, device=DEV)
        out = torch.empty_like(x[0])
        want = pkv.paged_prefill_attention(*x, c["scale"], softcap=5.0)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.paged_prefill_attention(*x, c["scale"], softcap=5.0, out=out, workspace=ws)
        ins.append((x, ws, want)), graphs.append(g), outs.append(out)
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, (_, _, w) in zip(outs, ins))


@pytest.mark.gpu
def test_workspaces_and_outputs_that_do_not_fit():
    c = prefill._case([100, 64], [10, 3], 4, 2, 64, 29)
    n = pkv.prefill_workspace_bytes(13, 2, 4, 2, 64, c["pools"][0].shape[0], c["bt"].shape[1])
    prefill._call(c, workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    with pytest.raises(pkv.PkvError):
        prefill._call(c, workspace=torch.empty(n - 1, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="out"):
        prefill._call(c, out=torch.empty((12, 4, 64), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(TypeError, match="out"):
        prefill._call(c, out=torch.empty((13, 4, 64), dtype=torch.float32, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        prefill._call(c, out=torch.empty((13, 4, 128), dtype=torch.bfloat16, device=DEV)[..., ::2])


def test_addresses_are_aligned_to_their_elements():
    from paged_kv_cache_mapped_gb300 import _build
    _build.build()
    lib, P = _lib.load(), ctypes.c_void_p
    d = _lib.PkvDims(2, 8, 2, 128, 16, 100, 8)

    def tables(bt=0x1000, slots=0x1000, count=0x1000):
        return lib.pkv_kv_step_tables(P(bt), P(0x1000), P(0x1000), P(slots), P(0x1000), P(0x1000), P(0x1000), P(count), P(0x1000),
                                      P(0x1000), 4, ctypes.byref(d), None, None)

    assert tables(bt=0x1002) == tables(slots=0x1004) == tables(count=0x1001) == C["PKV_ERR_ALIGNMENT"]

    def append(slots=0x1000, scales=0x1000):
        return lib.pkv_kv_append_f8(P(0x1000), P(0x1000), P(scales), P(0x1000), P(0x1000), P(0x1000), P(slots), 4, ctypes.byref(d),
                                    None, None)

    assert append(slots=0x1004) == append(scales=0x1002) == C["PKV_ERR_ALIGNMENT"]

    def attend(lens=0x1000):
        return lib.pkv_paged_prefill_attention(P(0x1000), P(0x1000), P(0x1000), P(0x1000), P(0x1000), P(lens), P(0x1000), 4, 0.1,
                                               None, P(0x1000), 1 << 40, ctypes.byref(d), None, None)

    assert attend(lens=0x1002) == C["PKV_ERR_ALIGNMENT"]


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[400, 130], [3, 1]], ids=["chunks", "few tokens"])
@pytest.mark.parametrize("d", [64, 128])
def test_caps_around_the_scores(d, new):
    """Scores (normal, up to about 4) far below, near and above the cap, alone and with a distance bias and a
    prefix: the cap's short and long polynomials and its general form."""
    c = prefill._case([1700, 900], new, 4, 2, d, 30)
    for softcap in (60.0, 14.0, 5.0, 1.0, 0.1):
        prefill._run(c, softcap=softcap)
        prefill._run(c, softcap=softcap, alibi_slopes=prefill._slopes(4), prefix_lens=[200, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("slope", [-1.5, 0.25, 3.0])
@pytest.mark.parametrize("d", [64, 128])
def test_fp8_blocks_of_large_values_under_small_weights(d, slope):
    """V scales up to 2^40 apart with a distance bias that leaves the large blocks of some rows next to no
    weight: the small blocks that carry those rows keep their digits."""
    c = decode._case([300, 40, 17, 1700], 8, 2, d, 8, True, vscale=40)
    decode._check(c, decode._call(c, alibi_slopes=[slope] * 8), alibi_slopes=[slope] * 8)
    decode._check(c, decode._call(c, softcap=3.0, alibi_slopes=[slope] * 8), softcap=3.0, alibi_slopes=[slope] * 8)


@pytest.mark.gpu
def test_blocks_past_32_bits():
    """Pools of more than 2^32 bytes: sequences at the far end give what the same rows give in a small pool, and
    the append writes its codes and scales there."""
    hq, hkv, d, B = 8, 8, 128, 2
    lens, new = [300, 77], [40, 1]
    c = prefill._case(lens, new, hq, hkv, d, 31, fill=0.0)
    small, bt = c["pools"], c["bt"]
    n = small[0].shape[0]
    q, starts, ld = c["q"].to(DEV), torch.from_numpy(c["starts"]).to(DEV), _i32(lens)
    r = dict(softcap=5.0, prefix_lens=_i32([9, 0]))
    want = pkv.paged_prefill_attention(q, *small, bt, ld, starts, c["scale"], 200, **r)
    want_d = pkv.paged_decode_attention_rules(q[:B], *small, bt, ld, c["scale"], 200, **r)
    nb = (1 << 32) // (hkv * 16 * d) + 2 * n
    far = torch.where(bt >= 0, bt + nb - n, bt)
    big = []
    for p in small:
        t = torch.empty((nb, hkv, 16, d), dtype=torch.bfloat16, device=DEV)
        t[nb - n:] = p
        big.append(t)
    err = pkv.new_error_word(DEV)
    assert torch.equal(pkv.paged_prefill_attention(q, *big, far, ld, starts, c["scale"], 200, error_word=err, **r), want)
    assert torch.equal(pkv.paged_decode_attention_rules(q[:B], *big, far, ld, c["scale"], 200, error_word=err, **r), want_d)
    rows = [big[0][nb - n:].transpose(1, 2).reshape(n * 16, hkv, d).clone(), big[1][nb - n:].transpose(1, 2).reshape(n * 16, hkv, d).clone()]
    del big
    got = []
    for first, total in ((0, n), (nb - n, nb)):
        codes = [torch.zeros((total, hkv, 16, d), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2)]
        scales = [torch.zeros((total, hkv), device=DEV) for _ in range(2)]
        pkv.kv_append_f8(*codes, *scales, *rows, torch.arange(n * 16, device=DEV) + first * 16, error_word=err)
        out = pkv.paged_decode_attention_f8(q[:B], *codes, *scales, far if first else bt, ld, c["scale"], 200, error_word=err, **r)
        got.append([x[first:].view(torch.uint8).clone() for x in codes] + [x[first:].clone() for x in scales] + [out])
        del codes, scales
    assert pkv.read_error(err) == 0
    assert all(torch.equal(x, y) for x, y in zip(*got))


@pytest.mark.gpu
def test_a_prompt_of_131072_tokens():
    """The plan's lists far past its shared memory, and rows at both ends of a long prompt."""
    n = 131072
    c = prefill._case([n], [n], 4, 1, 64, 32)
    err = pkv.new_error_word(DEV)
    got = prefill._call(c, error_word=err, window=5000, prefix_lens=[100])
    assert pkv.read_error(err) == 0
    prefill._check(c, got, rows=[(x, x % 4) for x in (0, 1, 127, 4999, 5000, 65535, 100001, n - 2, n - 1)], window=5000, prefix_lens=[100])
