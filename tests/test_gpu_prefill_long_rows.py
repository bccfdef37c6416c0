"""Prefill rows over long contexts whose result names the keys: every 16-key block has its own direction of K
and its own V, and a query points at two blocks in equal parts, so the output is the mean of those two blocks'
V.  A tile that is lost, taken twice or from another place moves the output by a third of the difference or
more, far past the bound, which a CPU test shows on planted mistakes."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
import rules_model
import test_gpu_prefill_attention as prefill
from helpers import paged_from_contiguous

DEV = torch.device("cuda:0")


def _context(L, hkv, d, g):
    """K, V [1, L, hkv, d]: signs times 1/4 and values in (-1, 1), the same within a block."""
    nblk = (L + 15) // 16
    sign = torch.randint(0, 2, (nblk, hkv, d), generator=g).float() * 2 - 1
    val = torch.rand((nblk, hkv, d), generator=g) * 2 - 1
    each = lambda x: x.repeat_interleave(16, 0)[:L][None].bfloat16()  # noqa: E731
    return each(sign * 0.25), each(val)


def _case(lens, new, hq, hkv, d, seed):
    g = torch.Generator().manual_seed(seed)
    B, lmax = len(lens), max(lens)
    k, v = torch.zeros((B, lmax, hkv, d)).bfloat16(), torch.zeros((B, lmax, hkv, d)).bfloat16()
    for b, L in enumerate(lens):
        k[b:b + 1, :L], v[b:b + 1, :L] = _context(L, hkv, d, g)
    kc, vc, bt = paged_from_contiguous(k, v, lens, sum((L + 15) // 16 for L in lens) + 3, g, fill=float("nan"))
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(k=k, v=v, pools=[kc, vc], bt=bt, lens=list(lens), new=list(new), starts=starts, hq=hq, hkv=hkv,
                d=d, rng=np.random.default_rng(seed))


SCALE = {64: 1.5, 128: 0.75}  # two blocks' keys stand d / 4 * SCALE = 24 above the mean of the others


def _aim(c):
    """q [T, hq, d] and, for each (row, head), the two blocks that it points at: ends, neighbours across every
    128-key border, and random ones, as far as the row sees whole blocks."""
    rng, T = c["rng"], int(c["starts"][-1])
    q = torch.zeros((T, c["hq"], c["d"]))
    at = {}
    for b, (L, n) in enumerate(zip(c["lens"], c["new"])):
        for r in range(n):
            seen = (L - n + r + 1) // 16  # whole blocks
            for h in range(c["hq"]):
                kind = rng.integers(0, 4)
                border = 8 * int(rng.integers(1, max(2, seen // 8))) if seen > 8 else 1
                i, j = [(0, seen - 1), (border - 1, min(border, seen - 1)), tuple(rng.integers(0, seen, 2)),
                        (seen - 1 - rng.integers(0, min(9, seen)), rng.integers(0, seen))][kind]
                row = int(c["starts"][b]) + r
                at[row, h] = (b, int(i), int(j))
                kk = c["k"][b, :, h // (c["hq"] // c["hkv"])].float()
                q[row, h] = 4 * (kk[16 * i] + (kk[16 * j] if i != j else 0))
    return q.bfloat16(), at


def _reference(c, q, row, h, b, keys=None, **r):
    """rules_model's row; `keys` (a list of key indices) plants a mistake: these keys in place of all."""
    g, L = c["hq"] // c["hkv"], c["lens"][b]
    i = L - c["new"][b] + row - int(c["starts"][b])
    k, v = c["k"][b, :i + 1, h // g].double().numpy(), c["v"][b, :i + 1, h // g].double().numpy()
    if keys is not None:
        k, v, i = k[keys], v[keys], len(keys) - 1
    ref, mass, size = rules_model.row(q[row, h].double().numpy(), k, v, i, SCALE[c["d"]], **r)
    return ref, rules_model.bound(ref, mass, size, c["d"], prefill._weight_eps(L))


SHAPES = {
    "single tokens": ([131072, 20000, 9000], [1, 1, 1], 8, 1, 128, 1),
    "few tokens": ([65536, 20000], [3, 5], 8, 2, 64, 2),
    "a chunk": ([20000, 700], [200, 3], 4, 2, 128, 3),
    "chunks": ([6000, 5000, 4097], [300, 129, 600], 4, 1, 64, 4),
}


@pytest.mark.gpu
@pytest.mark.parametrize("softcap", [0.0, 200.0, 60.0])
@pytest.mark.parametrize("shape", SHAPES)
def test_every_block_counts_once_in_its_place(shape, softcap):
    lens, new, hq, hkv, d, seed = SHAPES[shape]
    c = _case(lens, new, hq, hkv, d, seed)
    cache = [t.to(DEV) for t in (*c["pools"], c["bt"])]
    for _ in range(4 if sum(new) < 10 else 1):
        q, at = _aim(c)
        err = pkv.new_error_word(DEV)
        got = pkv.paged_prefill_attention(q.to(DEV), *cache, torch.tensor(lens, dtype=torch.int32, device=DEV),
                                          torch.from_numpy(c["starts"]).to(DEV), SCALE[d], softcap=softcap, error_word=err)
        assert pkv.read_error(err) == 0
        got = got.float().cpu().double().numpy()
        some = list(at)
        if len(some) > 80:
            some = [some[int(x)] for x in c["rng"].integers(0, len(some), 80)]
        for row, h in some:
            ref, bound = _reference(c, q, row, h, at[row, h][0], softcap=softcap)
            assert np.all(np.abs(got[row, h] - ref) <= bound), (row, h, at[row, h], float(np.abs(got[row, h] - ref).max()))


@pytest.mark.parametrize("d", [64, 128])
def test_planted_mistakes_are_past_the_bound(d):
    """A 128-key tile lost, taken twice, or read from the place of another, and a 64-key step lost: each in turn
    at the tiles that a row points at."""
    c = _case([9000], [4], 4, 2, d, 9)
    q, at = _aim(c)
    for (row, h), (b, i, j) in at.items():
        seen = np.arange(c["lens"][0] - c["new"][0] + row + 1)
        ref, bound = _reference(c, q, row, h, b)
        for blk in {i, j}:
            tile, step = blk // 8, blk // 4
            inside = seen // 128 == tile
            other = (tile + 5) % (len(seen) // 128)
            one = i // 8 == j // 8  # both in one tile: losing or doubling it changes them alike
            planted = {"moved": np.where(inside, other * 128 + seen % 128, seen)}
            if not one:
                planted["lost"], planted["twice"] = seen[~inside], np.concatenate([seen, seen[inside]])
            if i // 4 != j // 4:
                planted["step lost"] = seen[seen // 64 != step]
            for name, keys in planted.items():
                wrong, _ = _reference(c, q, row, h, b, keys=keys)
                assert np.mean(np.abs(wrong - ref) > 2 * bound) > 0.5, (name, row, h, i, j)
