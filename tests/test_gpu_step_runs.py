"""Engine steps over the FP8 cache, captured once and replayed, against host models of every part; and the
largest batches and head counts that the calls take."""
import numpy as np
import pytest
import torch

import f8_model
import paged_kv_cache_mapped_gb300 as pkv
import rules_model
import test_gpu_decode_rules as decode
import test_gpu_prefill_attention as prefill
from helpers import rand_bf16

DEV = torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (8, 1, 128)])
def test_a_run_over_the_fp8_cache(hq, hkv, d):
    """Tables, append and decode, captured in one graph: prompts, single tokens whose rows grow from step to step (so
    that blocks change their scale), a release and an admission into the blocks that it freed."""
    B, mb, nb, T = 4, 8, 16, 48
    g = torch.Generator().manual_seed(70)
    i32 = dict(dtype=torch.int32, device=DEV)
    bt, lens, new, count = torch.full((B, mb), -1, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32), torch.tensor([nb], **i32)
    free = torch.randperm(nb, generator=g).to(**i32)
    codes = [torch.zeros((nb, hkv, 16, d), device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros((nb, hkv), device=DEV) for _ in range(2)]
    starts, slots, pos = torch.empty(B + 1, **i32), torch.empty(T, dtype=torch.int64, device=DEV), torch.empty(T, **i32)
    k, v = (torch.zeros((T, hkv, d), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, out = torch.zeros((B, hq, d), dtype=torch.bfloat16, device=DEV), torch.empty((B, hq, d), dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(pkv.decode_workspace_bytes(B, hq, hkv, d, nb, mb), dtype=torch.uint8, device=DEV)
    err = pkv.new_error_word(DEV)

    def step():
        pkv.kv_step_tables(bt, lens, new, free, count, T, context_lens_out=lens, free_count_out=count, query_starts=starts,
                           slot_mapping=slots, positions=pos, error_word=err)
        pkv.kv_append_f8(*codes, *scales, k, v, slots, error_word=err)
        pkv.paged_decode_attention_f8(q, *codes, *scales, bt, lens, d ** -0.5, 40, softcap=9.0, out=out, workspace=ws, error_word=err)

    step()  # nothing new: one-time set-up
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    state = [(np.zeros((nb, hkv, 16, d)), np.zeros((nb, hkv))) for _ in range(2)]
    held = np.zeros(B, dtype=int)
    for n, want in enumerate([[17, 0, 16, 1], [1, 30, 1, 1], [1, 1, 1, 1], [1, 1, -1, 1], [1, 1, 33, 1], [1] * 4, [0] * 4, [-1, 1, 1, 5]]):
        rows = [(rand_bf16((T, hkv, d), g).float() * 2.0 ** n).bfloat16() for _ in range(2)]
        x = rand_bf16((B, hq, d), g)
        k.copy_(rows[0]), v.copy_(rows[1]), q.copy_(x), new.copy_(torch.tensor(want, **i32))
        out.fill_(7.0)
        graph.replay()
        assert pkv.read_error(err) == 0
        held = np.where(np.array(want) < 0, 0, held + np.array(want))
        assert lens.tolist() == held.tolist()
        at = slots.tolist()
        assert sum(s >= 0 for s in at) == sum(max(w, 0) for w in want)
        for i in range(2):
            state[i] = f8_model.append(*state[i], rows[i].double().numpy(), at)
            assert np.array_equal(scales[i].cpu().double().numpy(), state[i][1])
            assert np.array_equal(codes[i].float().cpu().double().numpy(), state[i][0])
        kk, vv = (c * s[:, :, None, None] for c, s in state)
        got, tab = out.double().cpu().numpy(), bt.cpu().numpy()
        for b, L in enumerate(held):
            blocks = tab[b, :(L + 15) // 16]
            for h in range(hq):
                if L == 0:
                    assert not got[b, h].any()
                    continue
                ks, vs = (y[blocks, h // (hq // hkv)].reshape(-1, d)[:L] for y in (kk, vv))
                ref, mass, size = rules_model.row(x[b, h].double().numpy(), ks, vs, L - 1, d ** -0.5, 40, 9.0)
                far = np.abs(got[b, h] - ref) - rules_model.bound(ref, mass, size, d, 2.0 ** -11)
                assert float(far.max()) <= 0, (n, b, h)


@pytest.mark.gpu
@pytest.mark.parametrize("f8", [False, True], ids=["bf16", "fp8"])
@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_decode_batch(f8, d):
    B = 4096
    lens = np.random.default_rng(1).integers(0, 70, B)
    c = decode._case([int(x) for x in lens], 4, 1, d, 71, f8)
    r = dict(window=30, softcap=6.0, alibi_slopes=decode._slopes(4), prefix_lens=[int(x) % 9 for x in range(B)],
             doc_starts=[int(x) // 2 for x in lens])
    err = pkv.new_error_word(DEV)
    got = decode._call(c, err=err, **r)
    assert pkv.read_error(err) == 0
    decode._check(c, got, rows={(b, b % 4) for b in (0, 1, 255, 256, 257, 1000, 2047, 2048, 4000, 4094, 4095)}, **r)
    assert not got[torch.from_numpy(lens == 0)].any()


@pytest.mark.gpu
def test_the_largest_prefill_batch():
    B = 4096
    lens = [int(x) for x in np.random.default_rng(2).integers(1, 60, B)]
    new = [min(L, 1 + b % 3) for b, L in enumerate(lens)]
    c = prefill._case(lens, new, 4, 1, 64, 72)
    err = pkv.new_error_word(DEV)
    got = prefill._call(c, error_word=err, softcap=6.0)
    assert pkv.read_error(err) == 0
    T = int(c["starts"][-1])
    prefill._check(c, got, rows=[(r, r % 4) for r in (0, 1, 2, 500, 1023, 1024, T // 2, T - 2, T - 1)], softcap=6.0)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new", [([40], [3]), ([40, 900], [3, 1]), ([3000], [200])], ids=["short", "few tokens", "chunk"])
def test_more_kv_heads_than_ctas(lens, new):
    """400 kv heads: one entry has more items than the GPU runs at once."""
    c = prefill._case(lens, new, 400, 400, 64, 73)
    for r in ({}, dict(softcap=6.0, window=50)):
        err = pkv.new_error_word(DEV)
        got = prefill._call(c, error_word=err, **r)
        assert pkv.read_error(err) == 0
        prefill._check(c, got, rows=[(row, h) for row in {0, 1, sum(new) - 1} for h in (0, 151, 152, 303, 304, 399)], **r)
