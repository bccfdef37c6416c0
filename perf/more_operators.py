"""Timed cases of differential attention over the paged cache (for one token, with the keys' accumulated
weights, and for many tokens) and of eviction from the cache by accumulated attention weight.

A differential layer's K rows hold two keys side by side, its q rows two queries; a head's output is the
difference of the two softmax maps' weighted V, the second map times a learned factor, often followed by a
root-mean-square norm of the head.  The pools are those of every other layer, so the appends, tables and
compactions serve it as they are.  A long-running request's cache is kept small by eviction: past a limit the
tokens with the least accumulated weight go, the kept rows move into the first slots and the blocks behind
them go back on the free stack.

`own = False` computes the plain form (elementary torch operations in fp32); `own = True` calls the library.
Cases are dicts; `op` names the operator, `B` sequences, `hq`/`hkv`/`d` heads and head size (of both halves).
"""
import math
import zlib

import numpy as np
import torch

own = False

BS = 16  # tokens per cache block
EPS = 1e-5


def _case(name, op, **kw):
    c = {"name": name, "op": op, "B": 1, "hq": 1, "hkv": 1, "d": 128, "lo": 1, "hi": 1}
    if op == "evict":
        c.update({"sink": 4, "top": 1, "recent": 1, "trigger": 0, "steady": False, "q8": False})
    else:
        c.update({"nlo": 1, "nhi": 1, "window": 0, "cap": 0.0, "alibi": False, "docs": False, "prefix": 0, "rowlam": False,
                  "norm": True})
    c.update(kw)
    return c


def listed():
    return [
        # two short requests of a small model: launch latency
        _case("diff decode 2 x 200", "decode", B=2, hq=8, hkv=8, d=64, lo=100, hi=256),
        # one decode layer of a 32/8-head model, ~4000 tokens a request
        _case("diff decode 32 x 4000", "decode", B=32, hq=32, hkv=8, lo=3500, hi=4500),
        # four very long contexts, factors of each token and head, no norm
        _case("diff decode 4 x 131072", "decode", B=4, hq=32, hkv=8, lo=131072, hi=131072, rowlam=True, norm=False),
        # windows that keep a shared prompt in sight, capped scores, 6 heads a kv head
        _case("diff decode rules 64 x 2048", "decode", B=64, hq=12, hkv=2, lo=16, hi=4096, window=1000, cap=50.0, prefix=100),
        # a decode step that also adds each key's weight into the layer's scores
        _case("diff decode scores 16 x 4000", "scores", B=16, hq=32, hkv=8, lo=3500, hi=4500),
        # a mixed step: most requests decode one token, some bring chunks; packed documents after a prefix
        _case("diff prefill mixed 24", "prefill", B=24, hq=12, hkv=2, lo=16, hi=4096, nlo=1, nhi=1024, docs=True, prefix=64),
        # a 4096-token chunk that ends a 16384-token prompt
        _case("diff prefill chunk of 16384", "prefill", B=1, hq=32, hkv=8, lo=16384, hi=16384, nlo=4096, nhi=4096),
        # whole prompts of a model with 64-wide heads, distance bias, factors of each token
        _case("diff prefill 4 prompts d64", "prefill", B=4, hq=8, hkv=8, d=64, lo=2001, hi=3001, nlo=3001, nhi=3001, alibi=True,
              rowlam=True),
        # a few short requests: latency
        _case("evict 2 x 300", "evict", B=2, hkv=2, d=64, lo=290, hi=310, top=100, recent=64),
        # prompts of ~4000 tokens cut to 1540 after their prefill
        _case("evict 32 x 4000", "evict", B=32, hkv=8, lo=3500, hi=4500, top=512, recent=1024),
        # requests that decode on, cut back each time they are 256 past the budget; INT8 pools; some are not yet there
        _case("evict int8 64 x 1800 steady", "evict", B=64, hkv=8, lo=1700, hi=1850, top=512, recent=1024, trigger=1795, steady=True,
              q8=True),
        # long contexts cut to an eighth
        _case("evict 4 x 65536", "evict", B=4, hkv=8, lo=65500, hi=65536, top=4096, recent=4091),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "scores", "prefill", "prefill", "evict", "evict"])
    hkv, g = rng.choice([1, 2, 4, 5, 8]), rng.randint(1, 8)
    c = _case("", op, hq=hkv * g, hkv=hkv, d=rng.choice([64, 128]))
    del c["name"]
    if op == "evict":
        c.update(hq=1, B=_log(rng, 1, 128))
        hi = _log(rng, 40, max(64, min(65536, 260000 // c["B"])))
        c.update(lo=rng.randint(hi // 2, hi), hi=hi, sink=rng.choice([0, 1, 4, 7]))
        budget = _log(rng, 16, max(17, hi - 8))
        c["recent"] = rng.randint(0, max(0, budget - c["sink"] - 1))
        c["top"] = max(1, budget - c["sink"] - c["recent"])
        c["trigger"] = rng.choice([0, budget + rng.randint(0, max(0, hi - budget))])
        c["steady"], c["q8"] = rng.random() < 0.5, rng.random() < 0.4
        return c
    if rng.random() < 0.3:
        c["cap"] = rng.choice([20.0, 30.0, 50.0])
    c["alibi"] = rng.random() < 0.3
    c["prefix"] = rng.choice([0, 0, rng.randint(1, 300)])
    c["rowlam"], c["norm"] = rng.random() < 0.4, rng.random() < 0.6
    if op != "prefill":
        c.update(B=_log(rng, 1, 128))
        hi = _log(rng, 2, max(64, min(131072, (260000 if op == "decode" else 100000) // c["B"])))
        c.update(lo=rng.randint(1, hi), hi=hi, docs=rng.random() < 0.3)
        c["window"] = rng.choice([0, 0, _log(rng, 1, hi)])
        return c
    c.update(B=_log(rng, 1, 24))
    hi = _log(rng, 2, max(32, min(8192, 40000 // c["B"])))
    c.update(lo=rng.randint(1, hi), hi=hi)
    # a bound on B * queries * keys * heads keeps the plain form's score matrix below a few GB
    most = max(1, int(1.2e9 / (c["B"] * c["hq"] * hi)))
    c.update(nhi=_log(rng, 1, max(1, min(hi, most))))
    c.update(nlo=rng.choice([1, c["nhi"]]), docs=rng.random() < 0.4)
    c["window"] = rng.choice([0, 0, _log(rng, 1, hi)])
    return c


# ------------------------------------------------------------------------------------------- inputs


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rs(c, salt):
    """Sizes come from the case, so that its outputs keep their shapes; the seed makes the data."""
    return np.random.RandomState(zlib.crc32(repr(sorted((k, v) for k, v in c.items() if k != "name")).encode()) ^ salt)


def _lens(c):
    """Cached tokens and query tokens of each request, on the host."""
    r = _rs(c, 0)
    B, lo, hi = c["B"], c["lo"], c["hi"]
    total = np.exp(r.uniform(math.log(lo), math.log(hi + 1), B)).astype(np.int64) if lo < hi // 8 else r.randint(lo, hi + 1, B)
    total = np.clip(total, 1, hi)
    if c["op"] != "prefill":
        return total, np.ones_like(total)
    nlo, nhi = c["nlo"], c["nhi"]
    if nhi - nlo > 8:   # most requests decode, some bring a chunk
        new = np.where(r.rand(B) < 0.75, 1, r.randint(nlo, nhi + 1, B))
    else:
        new = r.randint(nlo, nhi + 1, B)
    return total, np.minimum(np.maximum(new, 1), total)


def _tables(total, mb, nb, g):
    """Block tables [B, mb] over a shuffled pool of nb blocks, the permutation and the blocks in use."""
    nblk = (total + BS - 1) // BS
    perm = torch.randperm(nb, generator=g, device="cuda").int()
    t = torch.from_numpy(nblk).cuda()
    start = torch.cumsum(t, 0) - t
    j = torch.arange(mb, device="cuda")
    idx = (start[:, None] + j[None]).clamp(max=nb - 1)
    return torch.where(j[None] < t[:, None], perm[idx], torch.full_like(perm[idx], -1)), perm, int(nblk.sum())


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _budget(c):
    return c["sink"] + c["top"] + c["recent"]


def _trigger(c):
    return max(c["trigger"], _budget(c))


def _dropped(c, total):
    """Tokens that each request has lost before (a request at or under its budget has lost none)."""
    gone = _rs(c, 3).randint(1, 2000, len(total))
    return np.where((total >= _budget(c)) & c["steady"], gone, 0)


def _prepare_evict(c, g):
    B, hkv, d = c["B"], c["hkv"], c["d"]
    total, _ = _lens(c)
    gone = _dropped(c, total)
    budget = _budget(c)
    nb, mb = int(((total + BS - 1) // BS).sum()) + 5, int(((total + BS - 1) // BS).max())
    bt, perm, used = _tables(total, mb, nb, g)
    s = {"op": "evict", "case": c, "block_tables": bt, "context_lens": _dev(total, torch.int32), "dropped": _dev(gone, torch.int32)}
    free = torch.full((nb,), -1, dtype=torch.int32, device="cuda")
    free[:nb - used] = perm[used:]
    s.update(free_blocks=free, free_count=torch.tensor([nb - used], dtype=torch.int32, device="cuda"))
    S = mb * BS
    # accumulated weights: heavy-tailed, and none at all for a tenth of the tokens
    e = torch.rand((B, hkv, S), generator=g, device="cuda").clamp(min=1e-6).log().neg()
    e *= torch.exp(torch.randn((B, hkv, S), generator=g, device="cuda"))
    s["scores"] = torch.where(torch.rand((B, hkv, S), generator=g, device="cuda") < 0.1, torch.zeros_like(e), e)
    pos = torch.full((B, hkv, S), -1, dtype=torch.int32, device="cuda")
    if c["steady"]:   # what an earlier eviction left in the first `budget` slots: positions in no order
        for b in range(B):
            if gone[b] == 0:
                continue
            seen = int(total[b] + gone[b])
            old = seen - int(total[b] - budget)   # positions below this are in the first slots, or gone
            r = torch.rand((hkv, old), generator=g, device="cuda")
            r[:, :c["sink"]] += 2
            r[:, max(0, seen - c["recent"]):] += 2
            at = r.topk(budget, dim=1).indices
            pos[b, :, :budget] = torch.gather(at, 1, torch.rand((hkv, budget), generator=g, device="cuda").argsort(1)).int()
    s["slot_pos"] = pos
    # the outputs stand beside the inputs, so that a call can be repeated
    s.update(scores_out=s["scores"].clone(), slot_pos_out=pos.clone())
    for n in ("k", "v"):
        if c["q8"]:
            s[n] = torch.randint(1, 256, (nb, hkv, BS, d), generator=g, device="cuda", dtype=torch.uint8)
            s[n + "_scales"] = torch.rand((nb, hkv, BS), generator=g, device="cuda") * 0.02
        else:
            s[n] = torch.randn((nb, hkv, BS, d), generator=g, device="cuda", dtype=torch.bfloat16)
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "evict":
        return _prepare_evict(c, g)
    op, B, hkv, hq, d = c["op"], c["B"], c["hkv"], c["hq"], c["d"]
    total, new = _lens(c)
    s = {"op": op, "scale": 1.0 / math.sqrt(d // 2), "case": c, "eps": EPS}
    nb, mb = int(((total + BS - 1) // BS).sum()) + 5, int(((total + BS - 1) // BS).max())
    s["block_tables"], _, _ = _tables(total, mb, nb, g)
    s["context_lens"] = _dev(total, torch.int32)
    s["window"], s["softcap"] = c["window"], c["cap"]
    T = int(new.sum())
    s["q"] = torch.randn((T, hq, d), generator=g, device="cuda").bfloat16()
    # the learned factor of the second map: one a head, or from a projection of each token
    s["lambdas"] = torch.sigmoid(torch.randn((T, hq), generator=g, device="cuda")) if c["rowlam"] else \
        0.2 + 0.6 * torch.rand((hq,), generator=g, device="cuda")
    s["norm_weight"] = 0.2 * (1 + 0.2 * torch.randn((d,), generator=g, device="cuda")) if c["norm"] else None
    s["alibi_slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq) if c["alibi"] else None
    r = _rs(c, 1)
    s["prefix_lens"] = _dev(r.randint(0, c["prefix"] + 1, B), torch.int32) if c["prefix"] else None
    s["doc_starts"] = None
    if c["docs"]:   # packed documents of a few hundred tokens: each token sees its own from the start
        pos = np.concatenate([np.arange(L - n, L) for L, n in zip(total, new)])
        width = r.randint(50, 700, B)
        s["doc_starts"] = _dev(pos // np.repeat(width, new) * np.repeat(width, new), torch.int32)
    if op == "prefill":
        s["query_starts"] = _dev(np.concatenate([[0], np.cumsum(new)]), torch.int32)
        s["max_queries"] = int(new.max())
    if op == "scores":
        s["scores"] = torch.rand((B, hkv, mb * BS), generator=g, device="cuda").log().neg()
        s["scores_out"] = s["scores"].clone()
    s["k_cache"] = torch.randn((nb, hkv, BS, d), generator=g, device="cuda", dtype=torch.bfloat16)
    s["v_cache"] = torch.randn((nb, hkv, BS, d), generator=g, device="cuda", dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------------------------------- plain forms


def _plain_evict(s):
    c = s["case"]
    bt, lens, gone, scores = s["block_tables"].long(), s["context_lens"].long(), s["dropped"].long(), s["scores"]
    B, hkv, S = scores.shape
    budget, trigger = _budget(c), _trigger(c)
    slot = torch.arange(S, device=bt.device)
    pos = torch.where(s["slot_pos"] >= 0, s["slot_pos"].long(), slot + gone[:, None, None])
    live = (slot < lens[:, None])[:, None].expand(B, hkv, S)
    kept_anyway = (pos < c["sink"]) | (pos >= (lens + gone)[:, None, None] - c["recent"])
    key = torch.where(kept_anyway, torch.full_like(scores, math.inf), scores)
    key = torch.where(live, key, torch.full_like(key, -math.inf))
    order = torch.sort(key, dim=2, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, slot.expand(B, hkv, S))
    cut = (lens > trigger)[:, None, None]
    keep = live & (rank < budget)
    hole = (cut & (slot < budget) & ~keep).nonzero(as_tuple=True)
    from_ = (cut & (slot >= budget) & keep).nonzero(as_tuple=True)
    dst = (bt[hole[0], hole[2] // BS], hole[1], hole[2] % BS)
    src = (bt[from_[0], from_[2] // BS], from_[1], from_[2] % BS)
    out = {}
    for n in ("k", "v", "k_scales", "v_scales"):
        if n in s:
            s[n][dst] = s[n][src]
            out[n] = s[n]
    new_scores, new_pos = s["scores_out"], s["slot_pos_out"]
    front, behind = cut & (slot < budget), cut & (slot >= budget) & live
    new_scores.copy_(torch.where(behind, torch.zeros_like(scores), scores))
    new_scores[hole] = scores[from_]
    new_pos.copy_(torch.where(front, pos, torch.where(behind, torch.full_like(pos, -1), s["slot_pos"].long())))
    new_pos[hole] = pos[from_].int()
    over = lens > trigger
    col = torch.arange(bt.shape[1], device=bt.device)
    back = over[:, None] & (col >= (budget + BS - 1) // BS) & (col < ((lens + BS - 1) // BS)[:, None])
    free, count, nb = s["free_blocks"], s["free_count"], s["free_blocks"].shape[0]
    flat = back.reshape(-1)
    at = torch.where(flat, count + torch.cumsum(flat, 0) - 1, torch.full_like(flat, nb, dtype=torch.int64))
    free.copy_(torch.cat([free, free.new_zeros(1)]).scatter(0, at, s["block_tables"].reshape(-1))[:nb])
    out.update(context_lens=torch.where(over, torch.full_like(lens, budget), lens).int(),
               dropped=torch.where(over, gone + lens - budget, gone).int(), scores=new_scores, slot_pos=new_pos,
               free_blocks=free, free_count=(count + flat.sum()).int())
    return out


def _paged(pool, bt, n):
    """[B, hkv, n, d] fp32 rows of a pool [NB, hkv, 16, d] through block tables."""
    x = pool[bt.clamp(min=0).long()].float()                    # [B, mb, hkv, 16, d]
    return x.permute(0, 2, 1, 3, 4).reshape(bt.shape[0], pool.shape[1], -1, pool.shape[3])[:, :, :n]


def _softmax_map(s, q, k, pos, see):
    """The weights of one map: q [B, hq, n, d/2], k [B, hkv, L, d/2] -> [B, hq, n, L]."""
    B, hq, n, d = q.shape
    L, hkv = k.shape[2], k.shape[1]
    x = torch.matmul(q.reshape(B, hkv, hq // hkv * n, d), k.transpose(2, 3)).reshape(B, hq, n, L).mul_(s["scale"])
    if s["softcap"] > 0:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    if s["alibi_slopes"] is not None:
        x -= s["alibi_slopes"][None, :, None, None] * (pos[:, None, :, None] - torch.arange(L, device=q.device)).abs()
    x.masked_fill_(~see[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(torch.isinf(top), torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    return x.div_(torch.where(total > 0, total, torch.ones_like(total)))


def _plain_attention(s, q, pos, docs, lam, live):
    """q [B, hq, n, d], lam [B, hq, n] in fp32; pos, docs, live [B, n].  The rows and the weights."""
    bt = s["block_tables"]
    k, v = _paged(s["k_cache"], bt, bt.shape[1] * BS), _paged(s["v_cache"], bt, bt.shape[1] * BS)
    B, hq, n, d = q.shape
    L, hkv = k.shape[2], k.shape[1]
    t = torch.arange(L, device=q.device)
    lo = torch.zeros_like(pos)
    if s["window"] > 0:
        lo = torch.maximum(lo, pos - s["window"] + 1)
    if docs is not None:
        lo = torch.maximum(lo, docs)
    see = (t >= lo[..., None]) & (t <= pos[..., None])
    if s["prefix_lens"] is not None:
        see |= t < s["prefix_lens"].long()[:, None, None]
    see &= (t < s["context_lens"].long()[:, None, None]) & live[..., None]
    w = _softmax_map(s, q[..., d // 2:], k[..., d // 2:], pos, see).mul_(-lam[..., None])
    w += _softmax_map(s, q[..., :d // 2], k[..., :d // 2], pos, see)
    y = torch.matmul(w.reshape(B, hkv, hq // hkv * n, L), v).reshape(B, hq, n, d)
    if s["norm_weight"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * s["norm_weight"]
    return y, w


def _plain_decode(s):
    lens = s["context_lens"].long()
    B, hq, d = s["q"].shape
    pos = (lens - 1)[:, None]
    docs = s["doc_starts"].long()[:, None] if s["doc_starts"] is not None else None
    lam = s["lambdas"].expand(B, hq)[:, :, None]
    y, w = _plain_attention(s, s["q"].float()[:, :, None], pos, docs, lam, torch.ones_like(pos, dtype=torch.bool))
    out = y[:, :, 0].bfloat16()
    if s["op"] != "scores":
        return out
    hkv = s["scores"].shape[1]
    s["scores_out"].copy_(s["scores"] + w[:, :, 0].abs().reshape(B, hkv, hq // hkv, -1).sum(2))
    return {"out": out, "scores": s["scores_out"]}


def _plain_prefill(s):
    bt, lens, starts = s["block_tables"], s["context_lens"].long(), s["query_starts"].long()
    n, (T, hq, _) = s["max_queries"], s["q"].shape
    count = starts[1:] - starts[:-1]
    r = torch.arange(n, device=bt.device)
    live = r < count[:, None]
    at = (starts[:-1, None] + r).clamp(max=T - 1)
    pos = (lens - count)[:, None] + r
    docs = s["doc_starts"].long()[at] if s["doc_starts"] is not None else None
    lam = s["lambdas"].expand(T, hq)[at].transpose(1, 2)
    y, _ = _plain_attention(s, s["q"][at].float().transpose(1, 2), pos, docs, lam, live)
    i = torch.arange(T, device=bt.device)
    b = torch.searchsorted(starts, i, right=True) - 1
    return y[b, :, i - starts[b]].bfloat16()


# ------------------------------------------------------------------------------------------ the calls


def _own_evict(pkv, s):
    c = s["case"]
    if "workspace" not in s:   # kept by the program from step to step
        n = pkv.evict_workspace_bytes(c["B"], c["hkv"], c["sink"], c["top"], c["recent"])
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    args = (s["block_tables"], s["context_lens"], s["scores"], s["slot_pos"], s["dropped"], c["sink"], c["top"], c["recent"])
    kw = dict(trigger=c["trigger"], free_blocks=s["free_blocks"], free_count=s["free_count"], scores_out=s["scores_out"],
              slot_pos_out=s["slot_pos_out"], workspace=s["workspace"])
    if c["q8"]:
        lens, gone, count = pkv.kv_evict_q8(s["k"], s["v"], s["k_scales"], s["v_scales"], *args, **kw)
    else:
        lens, gone, count = pkv.kv_evict(s["k"], s["v"], *args, **kw)
    out = {n: s[n] for n in ("k", "v", "k_scales", "v_scales") if n in s}
    out.update(context_lens=lens, dropped=gone, scores=s["scores_out"], slot_pos=s["slot_pos_out"], free_blocks=s["free_blocks"],
               free_count=count)
    return out


def _own(s):
    import paged_kv_cache_mapped_gb300 as pkv
    op = s["op"]
    if op == "evict":
        return _own_evict(pkv, s)
    bt = s["block_tables"]
    B, hq, d = (bt.shape[0],) + s["q"].shape[1:]
    if "workspace" not in s:   # kept by the program from step to step
        dims = (hq, s["k_cache"].shape[1], d, s["k_cache"].shape[0], bt.shape[1])
        if op == "prefill":
            n = pkv.diff_prefill_workspace_bytes(s["q"].shape[0], B, *dims)
        else:
            n = pkv.diff_decode_workspace_bytes(B, *dims, score_stride=s["scores"].shape[2] if op == "scores" else 0)
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=bt.device)
    kw = dict(norm_weight=s["norm_weight"], norm_eps=s["eps"], softcap=s["softcap"], alibi_slopes=s["alibi_slopes"],
              doc_starts=s["doc_starts"], prefix_lens=s["prefix_lens"], workspace=s["workspace"])
    if op == "prefill":
        return pkv.paged_diff_prefill_attention(s["q"], s["k_cache"], s["v_cache"], bt, s["context_lens"], s["query_starts"],
                                                s["lambdas"], s["scale"], s["window"], **kw)
    if op == "decode":
        return pkv.paged_diff_decode_attention(s["q"], s["k_cache"], s["v_cache"], bt, s["context_lens"], s["lambdas"], s["scale"],
                                               s["window"], **kw)
    out = pkv.paged_diff_decode_attention_scores(s["q"], s["k_cache"], s["v_cache"], bt, s["context_lens"], s["lambdas"], s["scores"],
                                                 s["scale"], s["window"], scores_out=s["scores_out"], **kw)
    return {"out": out, "scores": s["scores_out"]}


def run(state):
    if own:
        return _own(state)
    if state["op"] == "evict":
        return _plain_evict(state)
    return _plain_prefill(state) if state["op"] == "prefill" else _plain_decode(state)


# ------------------------------------------------------------------------------------- work and exact


def _visible(c, L, pos, docs, prefix):
    """Keys seen by each query (host arrays): the interval [lo, pos] and the prefix beside it."""
    lo = np.zeros_like(pos)
    if c["window"] > 0:
        lo = np.maximum(lo, pos - c["window"] + 1)
    if docs is not None:
        lo = np.maximum(lo, docs)
    p = np.minimum(prefix, L)
    inside = np.maximum(0, pos - lo + 1)
    both = np.maximum(0, np.minimum(pos + 1, p) - np.minimum(lo, p))
    return inside + p - np.where(inside > 0, both, 0), lo, p


def work(case):
    c = case
    total, new = _lens(c)
    B, hq, hkv, d = c["B"], c["hq"], c["hkv"], c["d"]
    if c["op"] == "evict":
        budget, trigger = _budget(c), _trigger(c)
        row = 2 * (d + 4 if c["q8"] else 2 * d)   # a K and a V row
        n = 16 * B + 8
        for L in total[total > trigger]:
            tail = int(L) - budget
            late = min(tail, c["recent"])
            rest = max(1, int(L) - c["sink"] - c["recent"])
            moved = late + (tail - late) * c["top"] / rest   # kept rows behind the budget, as scores in no order leave them
            n += int(hkv * (16 * int(L) + 2 * row * moved)) + 8 * (tail // BS)
        return {"bytes": n, "flops": 0}
    r = _rs(c, 1)
    prefix = r.randint(0, c["prefix"] + 1, B) if c["prefix"] else np.zeros(B, dtype=np.int64)
    width = r.randint(50, 700, B) if c["docs"] else None
    pairs = keys = 0
    for b in range(B):
        L, n = int(total[b]), int(new[b])
        pos = np.arange(L - n, L)
        docs = pos // width[b] * width[b] if width is not None else None
        see, lo, p = _visible(c, L, pos, docs, int(prefix[b]))
        pairs += int(see.sum())
        keys += int(min(L, p + max(0, L - max(int(lo.min()), p))))
    n = int(keys * hkv * d * 4 + 2 * int(new.sum()) * hq * d * 2 + keys / BS * 4)
    if c["op"] == "scores":
        n += 8 * keys * hkv
    # a pair's two products of half heads, and one of its weight with V
    return {"bytes": n, "flops": 4 * pairs * hq * d}


def exact(case, seed):
    c = case
    if c["op"] == "evict":
        return None
    s = prepare(case, seed)
    lens = s["context_lens"].tolist()
    starts = s["query_starts"].tolist() if c["op"] == "prefill" else list(range(c["B"] + 1))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    group, half = c["hq"] // c["hkv"], c["d"] // 2
    acc = s["scores"].double() if c["op"] == "scores" else None
    for b, L in enumerate(lens):
        q0, q1 = starts[b], starts[b + 1]
        i = torch.arange(L - (q1 - q0), L, device="cuda")
        t = torch.arange(L, device="cuda")
        lo = torch.zeros_like(i)
        if c["window"] > 0:
            lo = (i + 1 - c["window"]).clamp(min=0)
        if s["doc_starts"] is not None:
            lo = torch.maximum(lo, s["doc_starts"][q0:q1].long())
        mask = (t[None] <= i[:, None]) & (t[None] >= lo[:, None])
        if s["prefix_lens"] is not None:
            mask = mask | (t[None] < int(s["prefix_lens"][b]))
        rows = s["block_tables"][b, : (L + BS - 1) // BS].long()
        for h in range(c["hq"]):
            k, v = (s[a][rows, h // group].double().reshape(-1, c["d"])[:L] for a in ("k_cache", "v_cache"))
            weight = 0
            for m in range(2):
                x = (s["q"][q0:q1, h, m * half:(m + 1) * half].double() @ k[:, m * half:(m + 1) * half].T) / math.sqrt(half)
                if c["cap"] > 0:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if s["alibi_slopes"] is not None:
                    x = x - s["alibi_slopes"][h].double() * (i[:, None] - t[None]).abs()
                x = torch.where(mask, x, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                top = x.amax(1, keepdim=True)
                p = torch.exp(x - torch.where(top > -math.inf, top, torch.zeros_like(top)))
                z = p.sum(1, keepdim=True)
                p = p / torch.where(z > 0, z, torch.ones_like(z))
                if m == 0:
                    weight = p
                else:
                    lam = s["lambdas"][q0:q1, h].double()[:, None] if c["rowlam"] else s["lambdas"][h].double()
                    weight = weight - lam * p
            y = weight @ v
            if s["norm_weight"] is not None:
                y = y / torch.sqrt(y.square().mean(1, keepdim=True) + EPS) * s["norm_weight"].double()
            out[q0:q1, h] = y
            if acc is not None:
                acc[b, h // group, :L] += weight[0].abs()
    return out if acc is None else {"out": out, "scores": acc}
