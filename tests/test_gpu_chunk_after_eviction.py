"""A chunk that comes after an eviction: its rows see the kept tokens, which lie in the slots below it in no order, and the
chunk's own before them; the step tables' positions are slots, to which `dropped` adds up to the tokens' positions."""
import numpy as np
import pytest
import torch

import diff_model
import paged_kv_cache_mapped_gb300 as pkv
import rules_model
from helpers import rand_bf16

DEV = torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("hq,d", [(4, 64), (12, 128)])
@pytest.mark.parametrize("prompts,chunks,rules", [
    ([90, 70, 33], [25, 60, 7], (3, 20, 15)),
    ([700, 650, 120], [1, 130, 64], (4, 400, 100)),
], ids=["short", "past 512 keys"])
def test_a_chunk_sees_the_kept_tokens_and_its_own(hq, d, prompts, chunks, rules):
    B, hkv, budget = len(prompts), 2, sum(rules)
    mb = (max(p + c for p, c in zip(prompts, chunks)) + 15) // 16
    nb = sum((p + c + 15) // 16 for p, c in zip(prompts, chunks)) + 3
    g = torch.Generator().manual_seed(hq)
    i32 = dict(dtype=torch.int32, device=DEV)
    bt, lens, gone, count = torch.full((B, mb), -1, **i32), torch.zeros(B, **i32), torch.zeros(B, **i32), torch.tensor([nb], **i32)
    free = torch.randperm(nb, generator=g).to(**i32)
    kc, vc = (torch.full((nb, hkv, 16, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    err = pkv.new_error_word(DEV)
    rows = [[], []]   # of all tokens, by position: [B][position, hkv, d] of K and of V

    def step(new, lens, count):
        T = sum(new)
        q, k, v = (rand_bf16((T, n, d), g) for n in (hq, hkv, hkv))
        lens, starts, slots, positions, count = pkv.kv_step_tables(bt, lens, torch.tensor(new, **i32), free, count, T, error_word=err)
        pkv.kv_append(kc, vc, k.to(DEV), v.to(DEV), slots, error_word=err)
        for t, x in zip(rows, (k, v)):
            t.append([y.double().numpy() for y in torch.split(x, new)])
        return q, lens, starts, positions, count

    _, lens, _, _, count = step(prompts, lens, count)
    scores = torch.rand((B, hkv, mb * 16), generator=g).to(DEV)
    pos = torch.full((B, hkv, mb * 16), -1, **i32)
    lens, gone, count = pkv.kv_evict(kc, vc, bt, lens, scores, pos, gone, *rules, free_blocks=free, free_count=count, error_word=err)
    kept, lost = lens.tolist(), gone.tolist()
    assert kept == [min(p, budget) for p in prompts] and lost == [p - L for p, L in zip(prompts, kept)]
    slot_pos = pos.cpu().numpy()
    q, lens, starts, positions, count = step(chunks, lens, count)
    at = np.concatenate([[0], np.cumsum(chunks)])
    for b in range(B):
        p = positions[at[b]:at[b + 1]].cpu().numpy()
        assert np.array_equal(p, kept[b] + np.arange(chunks[b]))
        assert np.array_equal(p + lost[b], prompts[b] + np.arange(chunks[b]))
    lam, w = torch.rand(hq, generator=g), 1 + 0.2 * torch.randn(d, generator=g)
    scale, plain_scale = (d // 2) ** -0.5, d ** -0.5
    out = pkv.paged_diff_prefill_attention(q.to(DEV), kc, vc, bt, lens, starts, lam.to(DEV), scale, norm_weight=w.to(DEV), error_word=err)
    plain = pkv.paged_prefill_attention(q.to(DEV), kc, vc, bt, lens, starts, plain_scale, error_word=err)
    assert pkv.read_error(err) == 0
    out, plain = (t.float().cpu().double().numpy() for t in (out, plain))
    for b, n in enumerate(chunks):
        weight_eps = 2.0 ** -16 if kept[b] + n <= 512 else 2.0 ** -8
        for h in range(hq):
            kv = h // (hq // hkv)
            order = slot_pos[b, kv, :kept[b]] if lost[b] else np.arange(kept[b])
            assert len(set(order.tolist())) == kept[b] and order.max(initial=-1) < prompts[b]
            keys, vals = (np.concatenate([t[0][b][order, kv], t[1][b][:, kv]]) for t in rows)
            for i in sorted({0, 1, n // 2, n - 1} & set(range(n))):
                m, row = kept[b] + i + 1, q[at[b] + i, h].double().numpy()
                ref, tol = diff_model.row(row, keys[:m], vals[:m], m - 1, scale, float(lam[h]), w.double().numpy(), 1e-5, weight_eps)
                assert np.all(np.abs(out[at[b] + i, h] - ref) <= tol), (b, h, i)
                ref, mass, size = rules_model.row(row, keys[:m], vals[:m], m - 1, plain_scale)
                assert np.all(np.abs(plain[at[b] + i, h] - ref) <= rules_model.bound(ref, mass, size, d, weight_eps)), (b, h, i)
