"""Timed cases of the serving-step operators: step tables, the FP8 block-scaled cache, and attention
with score rules (capped scores, distance bias, documents, prefixes) for one token and for many.

A serving engine runs them in this order for every step: `kv_step_tables` gives each request the
cache blocks and slots of its new tokens, an append writes their K and V, and an attention call reads
the cache: `paged_prefill_attention` for chunks of prompts (and mixed batches), the decode calls for
single tokens.  Each case below is one call of one operator on the inputs that an engine has in hand.

`own = False` computes the plain form (elementary torch operations in fp32); `own = True` calls the
library.  Cases are dicts; `op` names the operator, `B` sequences, `hq`/`hkv`/`d` heads and head size.
"""
import math
import zlib

import numpy as np
import torch

own = False

BS = 16           # tokens per cache block
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -120, 119   # exponents of the block scales


def _case(name, op, **kw):
    c = {"name": name, "op": op, "B": 1, "hq": 1, "hkv": 1, "d": 128, "lo": 1, "hi": 1, "nlo": 1, "nhi": 1,
         "window": 0, "cap": 0.0, "alibi": False, "docs": False, "prefix": 0}
    c.update(kw)
    return c


def listed():
    return [
        # a decode step of 64 requests: every request gets one slot, every 16th a new block
        _case("tables 64 decoding", "tables", B=64, lo=16, hi=4096, nlo=1, nhi=1),
        # a large engine step: 4096 request slots, most decode, some admit prompts or finish
        _case("tables 4096 mixed", "tables", B=4096, lo=0, hi=4096, nlo=-1, nhi=2048),
        # the decode step's K/V rows of a 2-kv-head model into its FP8 cache
        _case("append fp8 64 decoding", "append", B=64, hkv=2, lo=16, hi=4096, nlo=1, nhi=1),
        # sixteen prompts' K/V rows written in one call
        _case("append fp8 16 prompts", "append", B=16, hkv=8, lo=0, hi=0, nlo=3500, nhi=4500),
        # one decode layer of a 32/8-head model over the FP8 cache, ~4000 tokens a request
        _case("decode fp8, 32 x 4000", "decode_f8", B=32, hq=32, hkv=8, lo=3500, hi=4500),
        # four very long contexts: the split over the keys is all the parallelism there is
        _case("decode fp8, 4 x 131072", "decode_f8", B=4, hq=32, hkv=8, lo=131072, hi=131072),
        # capped scores and a sliding window that keeps a shared prompt in sight, 6 heads a kv head
        _case("decode rules, 64 x 2048", "decode", B=64, hq=12, hkv=2, lo=16, hi=4096, window=1024, cap=50.0,
              prefix=100),
        # the same layer size as the FP8 case with a distance bias over the whole context
        _case("decode rules, 32 x 4000", "decode", B=32, hq=32, hkv=8, lo=3500, hi=4500, cap=30.0, alibi=True),
        # two short requests of a small model: launch latency
        _case("decode rules, 2 x 200", "decode", B=2, hq=8, hkv=8, d=64, lo=100, hi=256, alibi=True),
        # a 4096-token chunk that ends a 16384-token prompt, capped scores
        _case("prefill chunk of 16384", "prefill", B=1, hq=32, hkv=8, lo=16384, hi=16384, nlo=4096, nhi=4096, cap=50.0),
        # a mixed step: most requests decode one token, some bring chunks; packed documents after a prefix
        _case("prefill mixed 24", "prefill", B=24, hq=12, hkv=2, lo=16, hi=4096, nlo=1, nhi=1024, docs=True, prefix=64),
        # whole prompts of a model with 64-wide heads, distance bias and a sliding window
        _case("prefill 4 prompts d64", "prefill", B=4, hq=8, hkv=8, d=64, lo=2001, hi=3001, nlo=3001, nhi=3001,
              alibi=True, window=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "decode_f8", "decode", "prefill", "prefill"])
    hkv, g = rng.choice([1, 2, 4, 5, 8]), rng.randint(1, 8)
    c = _case("", op, hq=hkv * g, hkv=hkv, d=rng.choice([64, 128]))
    del c["name"]
    if op == "tables":
        c.update(B=_log(rng, 1, 4096), lo=0, hi=_log(rng, 20, 8192))
        c.update(nlo=rng.choice([-1, 0, 1]), nhi=_log(rng, 1, 2048))
        return c
    if op == "append":
        c.update(B=_log(rng, 1, 256))
        n = min(4500, max(1, 60000 // c["B"]))
        c.update(nhi=_log(rng, 1, n))
        c.update(nlo=rng.randint(1, c["nhi"]), lo=0, hi=rng.choice([0, _log(rng, 1, 2000)]))
        return c
    if rng.random() < 0.5:
        c["cap"] = rng.choice([20.0, 30.0, 50.0])
    c["alibi"] = rng.random() < 0.4
    c["prefix"] = rng.choice([0, 0, rng.randint(1, 300)])
    if op in ("decode", "decode_f8"):
        c.update(B=_log(rng, 1, 128))
        hi = _log(rng, 2, max(64, min(131072, 260000 // c["B"])))
        c.update(lo=rng.randint(1, hi), hi=hi, docs=rng.random() < 0.3)
        c["window"] = rng.choice([0, 0, _log(rng, 1, hi)])
        return c
    c.update(B=_log(rng, 1, 24))
    hi = _log(rng, 2, max(32, min(8192, 40000 // c["B"])))
    c.update(lo=rng.randint(1, hi), hi=hi)
    # a bound on B * queries * keys * heads keeps the plain form's score matrix below a few GB
    most = max(1, int(1.5e9 / (c["B"] * c["hq"] * hi)))
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
    """Context lengths (cached tokens) and new tokens of each request, on the host."""
    r = _rs(c, 0)
    B, lo, hi = c["B"], c["lo"], c["hi"]
    ctx = np.exp(r.uniform(math.log(lo + 1), math.log(hi + 1), B)).round().astype(np.int64) - 1 if lo < hi // 8 \
        else r.randint(lo, hi + 1, B)
    nlo, nhi = c["nlo"], c["nhi"]
    if nhi - nlo > 8:   # most requests decode, some bring a chunk, some (nlo < 0) finish
        kind = r.rand(B)
        new = np.where(kind < 0.75, 1, r.randint(max(nlo, 0), nhi + 1, B))
        if nlo < 0:
            new = np.where(kind > 0.95, -1, new)
    else:
        new = r.randint(nlo, nhi + 1, B)
    if c["op"] in ("append",) and c["hi"] == 0:
        new = r.randint(nlo, nhi + 1, B)
    if c["op"] == "tables":   # an engine caps the new tokens of one step
        most = 1 << 17
        over = np.cumsum(np.maximum(new, 0)) > most
        new = np.where(over & (new > 0), 0, new)
    return ctx, new


def _tables(total, mb, nb, g):
    """Block tables [B, mb] over a shuffled pool of nb blocks, and the permutation."""
    nblk = (total + BS - 1) // BS
    perm = torch.randperm(nb, generator=g, device="cuda").int()
    t = torch.from_numpy(nblk).cuda()
    start = torch.cumsum(t, 0) - t
    j = torch.arange(mb, device="cuda")
    idx = (start[:, None] + j[None]).clamp(max=nb - 1)
    return torch.where(j[None] < t[:, None], perm[idx], torch.full_like(perm[idx], -1)), perm, int(nblk.sum())


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).cuda()


def _e4m3(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def prepare(case, seed):
    c, g = case, _gen(seed)
    op, B, hkv, hq, d = c["op"], c["B"], c["hkv"], c["hq"], c["d"]
    ctx, new = _lens(c)
    s = {"op": op, "scale": 1.0 / math.sqrt(d), "case": c}
    if op == "tables":
        mb = (c["hi"] + max(c["nhi"], 1) + BS - 1) // BS
        held = int(((ctx + BS - 1) // BS).sum())
        more = int(((ctx + np.maximum(new, 0) + BS - 1) // BS).sum()) - held
        nb = held + more + 7
        bt, perm, used = _tables(ctx, mb, nb, g)
        free = torch.full((nb,), -1, dtype=torch.int32, device="cuda")
        free[:nb - used] = perm[used:]
        T = int(np.maximum(new, 0).sum())
        s.update(block_tables=bt, context_lens=_dev(ctx, torch.int32), new_tokens=_dev(new, torch.int32), free_blocks=free,
                 free_count=torch.tensor([nb - used], dtype=torch.int32, device="cuda"), max_tokens=max(1, (T + 63) // 64 * 64))
        return s
    if op == "append":
        total = ctx + new
        nb = int(((total + BS - 1) // BS).sum()) + 5
        mb = int(((total + BS - 1) // BS).max())
        bt, _, _ = _tables(total, mb, nb, g)
        seq = np.repeat(np.arange(B), new)
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(ctx, new)])
        seq, pos = _dev(seq, torch.int64), _dev(pos, torch.int64)
        s["slots"] = bt[seq, pos // BS].long() * BS + pos % BS
        T = int(seq.shape[0])
        for n in ("k", "v"):
            # rows of varying size, as channels of a real cache have: some blocks' scales grow
            amp = torch.exp2(torch.randn((T, hkv, 1), generator=g, device="cuda") * 1.5)
            s[n] = (torch.randn((T, hkv, d), generator=g, device="cuda") * amp).bfloat16()
            codes = torch.randn((nb, hkv, BS, d), generator=g, device="cuda") * 100
            s[n + "_codes"] = _e4m3(codes)
            s[n + "_scales"] = torch.exp2(torch.randint(-8, -5, (nb, hkv), generator=g, device="cuda").float())
        return s
    if op == "prefill":
        total = np.maximum(ctx, 1)
        new = np.minimum(np.maximum(new, 1), total)
    else:
        total = np.maximum(ctx, 1)
        new = np.ones_like(total)
    nb = int(((total + BS - 1) // BS).sum()) + 5
    mb = int(((total + BS - 1) // BS).max())
    s["block_tables"], _, _ = _tables(total, mb, nb, g)
    s["context_lens"] = _dev(total, torch.int32)
    s["window"], s["softcap"] = c["window"], c["cap"]
    T = int(new.sum())
    r = _rs(c, 1)
    s["q"] = torch.randn((T, hq, d), generator=g, device="cuda").bfloat16()
    s["alibi_slopes"] = torch.exp2(-8.0 * torch.arange(1, hq + 1, device="cuda") / hq) if c["alibi"] else None
    s["prefix_lens"] = _dev(r.randint(0, c["prefix"] + 1, B), torch.int32) if c["prefix"] else None
    s["doc_starts"] = None
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(total, new)])
    if c["docs"]:   # packed documents of a few hundred tokens: each token sees its own from the start
        width = r.randint(50, 700, B)
        s["doc_starts"] = _dev(pos // np.repeat(width, new) * np.repeat(width, new), torch.int32)
    if op == "prefill":
        s["query_starts"] = _dev(np.concatenate([[0], np.cumsum(new)]), torch.int32)
        s["max_queries"] = int(new.max())
    if op == "decode_f8":
        for n in ("k", "v"):
            s[n + "_codes"] = _e4m3(torch.randn((nb, hkv, BS, d), generator=g, device="cuda") * 90)
            # powers of two, as the append writes them, around values of unit size
            s[n + "_scales"] = torch.exp2(torch.randint(-8, -5, (nb, hkv), generator=g, device="cuda").float())
    else:
        s["k_cache"] = torch.randn((nb, hkv, BS, d), generator=g, device="cuda", dtype=torch.bfloat16)
        s["v_cache"] = torch.randn((nb, hkv, BS, d), generator=g, device="cuda", dtype=torch.bfloat16)
    return s


# ---------------------------------------------------------------------------------------- plain forms


def _plain_tables(s):
    bt, lens, new, free, count = s["block_tables"], s["context_lens"].long(), s["new_tokens"].long(), s["free_blocks"], s["free_count"]
    B, mb, nb, T = bt.shape[0], bt.shape[1], free.shape[0], s["max_tokens"]
    dev = bt.device
    held = (lens + BS - 1) // BS
    col = torch.arange(mb, device=dev)
    # released blocks go onto the free stack, sequences and blocks ascending
    gone = ((new < 0)[:, None] & (col < held[:, None])).reshape(-1)
    at = torch.where(gone, count + torch.cumsum(gone, 0) - 1, torch.full_like(gone, nb, dtype=torch.int64))
    stack = torch.cat([free, free.new_zeros(1)]).scatter(0, at, bt.reshape(-1))[:nb]
    top = count + gone.sum()
    # new blocks come off its top, in the order of the sequences
    grow = new.clamp(min=0)
    after = torch.where(new < 0, torch.zeros_like(lens), lens + grow)
    need = torch.where(new > 0, (lens + grow + BS - 1) // BS - held, torch.zeros_like(held))
    first = torch.cumsum(need, 0) - need
    taken = (col >= held[:, None]) & (col < (held + need)[:, None])
    idx = top - 1 - first[:, None] - (col - held[:, None])
    tables = torch.where(taken, stack[idx.clamp(0, nb - 1)], bt)
    starts = torch.cat([grow.new_zeros(1), torch.cumsum(grow, 0)])
    i = torch.arange(T, device=dev)
    b = (torch.searchsorted(starts, i, right=True) - 1).clamp(max=B - 1)
    pos = lens[b] + i - starts[b]
    live = i < starts[B]
    slots = tables[b, (pos // BS).clamp(max=mb - 1)].long() * BS + pos % BS
    return {"block_tables": tables, "context_lens": after.int(), "query_starts": starts.int(),
            "slot_mapping": torch.where(live, slots, torch.full_like(slots, -1)),
            "positions": torch.where(live, pos, torch.full_like(pos, -1)).int(),
            "free_blocks": stack, "free_count": (top - need.sum()).int()}


def _needed_scale(amax):
    """The smallest power of two s with amax / s <= 448, its exponent kept in the table's range."""
    f, e = torch.frexp(amax)   # amax = f 2^e, f in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(f <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(MIN_EXP, MAX_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _plain_append(s):
    slots = s["slots"]
    blocks, inv = torch.unique(slots // BS, return_inverse=True)
    n, off = blocks.shape[0], slots % BS
    written = torch.zeros((n, BS), dtype=torch.bool, device=slots.device)
    written[inv, off] = True
    out = {}
    for name in ("k", "v"):
        x, codes, scales = s[name].float(), s[name + "_codes"], s[name + "_scales"]
        amax = torch.zeros((n, x.shape[1]), device=x.device)
        amax.scatter_reduce_(0, inv[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        need = _needed_scale(amax)
        had = scales[blocks]
        now = torch.where(written[:, :1], need, torch.maximum(need, had))   # offset 0 starts a block anew
        keep = codes[blocks]
        moved = _e4m3(keep.float() * (had / now)[:, :, None, None])
        new = torch.where((~written[:, None, :, None]) & (~written[:, :1, None, None]), moved.float(), keep.float()).to(keep.dtype)
        new[inv, :, off] = _e4m3(x / now[inv][:, :, None])
        codes.view(torch.uint8)[blocks] = new.view(torch.uint8)   # plain byte copies
        scales[blocks] = now
        out[name + "_codes"], out[name + "_scales"] = codes, scales
    return out


def _paged(pool, bt, n):
    """[B, hkv, n, d] fp32 rows of a pool [NB, hkv, 16, d] through block tables."""
    x = pool[bt.clamp(min=0).long()].float()                    # [B, mb, hkv, 16, d]
    return x.permute(0, 2, 1, 3, 4).reshape(bt.shape[0], pool.shape[1], -1, pool.shape[3])[:, :, :n]


def _plain_attention(s, k, v, q, pos, docs, live):
    """q [B, hq, n, d], k and v [B, hkv, L, d] in fp32; pos, docs, live [B, n]."""
    B, hq, n, d = q.shape
    L, hkv = k.shape[2], k.shape[1]
    x = torch.matmul(q.reshape(B, hkv, hq // hkv * n, d), k.transpose(2, 3)).reshape(B, hq, n, L) * s["scale"]
    if s["softcap"] > 0:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    t = torch.arange(L, device=q.device)
    if s["alibi_slopes"] is not None:
        x -= s["alibi_slopes"][None, :, None, None] * (pos[:, None, :, None] - t).abs()
    lo = torch.zeros_like(pos)
    if s["window"] > 0:
        lo = torch.maximum(lo, pos - s["window"] + 1)
    if docs is not None:
        lo = torch.maximum(lo, docs)
    see = (t >= lo[..., None]) & (t <= pos[..., None])
    if s["prefix_lens"] is not None:
        see |= t < s["prefix_lens"].long()[:, None, None]
    see &= (t < s["context_lens"].long()[:, None, None]) & live[..., None]
    x = x.masked_fill(~see[:, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(B, hkv, hq // hkv * n, L), v).reshape(B, hq, n, d)
    return o / torch.where(total > 0, total, torch.ones_like(total))


def _plain_decode(s):
    bt, lens = s["block_tables"], s["context_lens"].long()
    n = bt.shape[1] * BS
    if s["op"] == "decode_f8":
        at = bt.clamp(min=0).long()
        k, v = (_paged(s[a + "_codes"], bt, n) * s[a + "_scales"][at].permute(0, 2, 1).repeat_interleave(BS, 2)[..., None]
                for a in ("k", "v"))
    else:
        k, v = _paged(s["k_cache"], bt, n), _paged(s["v_cache"], bt, n)
    pos = (lens - 1)[:, None]
    docs = s["doc_starts"].long()[:, None] if s["doc_starts"] is not None else None
    o = _plain_attention(s, k, v, s["q"].float()[:, :, None], pos, docs, torch.ones_like(pos, dtype=torch.bool))
    return o[:, :, 0].bfloat16()


def _plain_prefill(s):
    bt, lens, starts = s["block_tables"], s["context_lens"].long(), s["query_starts"].long()
    n, T = s["max_queries"], s["q"].shape[0]
    k, v = _paged(s["k_cache"], bt, bt.shape[1] * BS), _paged(s["v_cache"], bt, bt.shape[1] * BS)
    count = starts[1:] - starts[:-1]
    r = torch.arange(n, device=bt.device)
    live = r < count[:, None]
    at = (starts[:-1, None] + r).clamp(max=T - 1)
    pos = (lens - count)[:, None] + r
    docs = s["doc_starts"].long()[at] if s["doc_starts"] is not None else None
    o = _plain_attention(s, k, v, s["q"][at].float().transpose(1, 2), pos, docs, live)
    out = torch.empty_like(s["q"])
    i = torch.arange(T, device=bt.device)
    b = torch.searchsorted(starts, i, right=True) - 1
    out[:] = o[b, :, i - starts[b]].bfloat16()
    return out


# ------------------------------------------------------------------------------------------ the calls


def _own(s):
    import paged_kv_cache_mapped_gb300 as pkv
    op = s["op"]
    if op == "tables":
        lens, starts, slots, pos, count = pkv.kv_step_tables(s["block_tables"], s["context_lens"], s["new_tokens"], s["free_blocks"],
                                                             s["free_count"], s["max_tokens"])
        return {"block_tables": s["block_tables"], "context_lens": lens, "query_starts": starts, "slot_mapping": slots,
                "positions": pos, "free_blocks": s["free_blocks"], "free_count": count}
    if op == "append":
        pkv.kv_append_f8(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["k"], s["v"], s["slots"])
        return {n: s[n] for n in ("k_codes", "k_scales", "v_codes", "v_scales")}
    bt = s["block_tables"]
    B, hq, d = (bt.shape[0],) + s["q"].shape[1:]
    pool = s["k_codes"] if op == "decode_f8" else s["k_cache"]
    if "workspace" not in s:   # kept by the program from step to step
        dims = (hq, pool.shape[1], d, pool.shape[0], bt.shape[1])
        n = pkv.prefill_workspace_bytes(s["q"].shape[0], B, *dims) if op == "prefill" else pkv.decode_workspace_bytes(B, *dims)
        s["workspace"] = torch.zeros(n, dtype=torch.uint8, device=bt.device)
    rules = dict(softcap=s["softcap"], alibi_slopes=s["alibi_slopes"], doc_starts=s["doc_starts"], prefix_lens=s["prefix_lens"])
    if op == "prefill":
        return pkv.paged_prefill_attention(s["q"], s["k_cache"], s["v_cache"], bt, s["context_lens"], s["query_starts"], s["scale"],
                                           s["window"], workspace=s["workspace"], **rules)
    if op == "decode_f8":
        return pkv.paged_decode_attention_f8(s["q"], s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], bt, s["context_lens"],
                                             s["scale"], s["window"], workspace=s["workspace"], **rules)
    return pkv.paged_decode_attention_rules(s["q"], s["k_cache"], s["v_cache"], bt, s["context_lens"], s["scale"], s["window"],
                                            workspace=s["workspace"], **rules)


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "tables":
        return _plain_tables(state)
    if op == "append":
        return _plain_append(state)
    return _plain_prefill(state) if op == "prefill" else _plain_decode(state)


# ------------------------------------------------------------------------------------- work and exact


def _visible(c, L, n, pos, docs, prefix):
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
    ctx, new = _lens(c)
    B, hq, hkv, d = c["B"], c["hq"], c["hkv"], c["d"]
    if c["op"] == "tables":
        grow = np.maximum(new, 0)
        T = int(grow.sum())
        blocks = int((np.where(new > 0, (ctx + grow + 15) // 16 - (ctx + 15) // 16, 0)).sum())
        gone = int(np.where(new < 0, (ctx + 15) // 16, 0).sum())
        # lengths and counts in, lengths and starts out, each new token's slot and position, each moved block once in, once out
        return {"bytes": 16 * B + 12 * T + 8 * (blocks + gone) + 16, "flops": 0}
    if c["op"] == "append":
        T = int(new.sum())
        blocks = int(((ctx + new + 15) // 16 - ctx // 16).sum())
        return {"bytes": T * (2 * hkv * d * 3 + 8) + blocks * hkv * 2 * 8, "flops": 0}
    total = np.maximum(ctx, 1)
    new = np.minimum(np.maximum(new, 1), total) if c["op"] == "prefill" else np.ones_like(total)
    r = _rs(c, 1)
    prefix = r.randint(0, c["prefix"] + 1, B) if c["prefix"] else np.zeros(B, dtype=np.int64)
    width = r.randint(50, 700, B) if c["docs"] else None
    pairs = keys = 0
    for b in range(B):
        L, n = int(total[b]), int(new[b])
        pos = np.arange(L - n, L)
        docs = pos // width[b] * width[b] if width is not None else None
        see, lo, p = _visible(c, L, n, pos, docs, int(prefix[b]))
        pairs += int(see.sum())
        keys += int(min(L, p + max(0, L - max(int(lo.min()), p))))
    elem = 1 + 4 / (BS * d) if c["op"] == "decode_f8" else 2
    return {"bytes": int(keys * hkv * d * 2 * elem + 2 * int(new.sum()) * hq * d * 2 + keys / BS * 4), "flops": 4 * pairs * hq * d}


def _round_e4m3(x):
    """fp64 values rounded to the nearest e4m3 value (ties to even), beyond 448 to 448."""
    a = x.abs().clamp(max=E4M3_MAX)
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -20))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=E4M3_MAX)


def _exact_append(s):
    slots = s["slots"].cpu().numpy()
    out = {}
    order = torch.from_numpy(np.argsort(slots, kind="stable")).cuda()
    blk = s["slots"][order] // BS
    for name in ("k", "v"):
        x = s[name].double()[order]
        codes, scales = s[name + "_codes"].to(torch.float32).double(), s[name + "_scales"].double()
        nb, hkv = scales.shape
        biggest = torch.zeros((nb, BS, hkv), dtype=torch.float64, device=x.device)
        fresh = torch.zeros((nb, BS), dtype=torch.bool, device=x.device)
        biggest[blk, s["slots"][order] % BS] = x.abs().amax(-1)
        fresh[blk, s["slots"][order] % BS] = True
        m = biggest.amax(1)
        e = torch.ceil(torch.log2(m.clamp(min=1e-300) / E4M3_MAX)).clamp(MIN_EXP, MAX_EXP)
        e = torch.where(torch.exp2(e - 1) * E4M3_MAX >= m, e - 1, e).clamp(MIN_EXP, MAX_EXP)   # a logarithm's last bit
        e = torch.where(torch.exp2(e) * E4M3_MAX < m, e + 1, e).clamp(MIN_EXP, MAX_EXP)
        need = torch.exp2(e)
        anew, touched = fresh[:, :1], fresh.any(1)[:, None]
        now = torch.where(touched, torch.where(anew, need, torch.maximum(need, scales)), scales)
        moved = _round_e4m3(codes * (scales / now)[:, :, None, None])
        codes = torch.where((touched & ~anew)[:, :, None, None], moved, codes)
        codes[blk, :, s["slots"][order] % BS] = _round_e4m3(x / now[blk][:, :, None])
        out[name + "_codes"], out[name + "_scales"] = codes, now
    return out


def exact(case, seed):
    c = case
    if c["op"] == "tables":
        return None
    s = prepare(case, seed)
    if c["op"] == "append":
        return _exact_append(s)
    lens = s["context_lens"].tolist()
    starts = s["query_starts"].tolist() if c["op"] == "prefill" else list(range(c["B"] + 1))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    g, cap = c["hq"] // c["hkv"], c["cap"]
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
        for h in range(c["hkv"]):
            if c["op"] == "decode_f8":
                k, v = ((s[a + "_codes"][rows, h].float().double() * s[a + "_scales"][rows, h].double()[:, None, None]).reshape(-1, c["d"])[:L]
                        for a in ("k", "v"))
            else:
                k, v = (s[a][rows, h].double().reshape(-1, c["d"])[:L] for a in ("k_cache", "v_cache"))
            for hh in range(h * g, h * g + g):
                x = (s["q"][q0:q1, hh].double() @ k.T) / math.sqrt(c["d"])
                if cap > 0:
                    x = cap * torch.tanh(x / cap)
                if s["alibi_slopes"] is not None:
                    x = x - s["alibi_slopes"][hh].double() * (i[:, None] - t[None]).abs()
                x = torch.where(mask, x, torch.tensor(-math.inf, dtype=torch.float64, device="cuda"))
                m = x.amax(1, keepdim=True)
                p = torch.exp(x - torch.where(m > -math.inf, m, torch.zeros_like(m)))
                z = p.sum(1, keepdim=True)
                out[q0:q1, hh] = (p @ v) / torch.where(z > 0, z, torch.ones_like(z))
    return out
