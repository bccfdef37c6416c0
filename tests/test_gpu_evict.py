"""Eviction by accumulated weight (pkv_kv_evict, pkv_kv_evict_q8) against a host model, exactly: fresh and earlier
shrunk sequences, ties, zeros of both signs, infinities and NaN, odd lengths and budgets, rows longer than shared memory
holds, outputs beside and in place of their inputs, bad lengths and blocks, full stacks, streams and graphs; and
the run of tables, append, decode with scores and eviction."""
import ctypes

import numpy as np
import pytest
import torch

import evict_model
import paged_kv_cache_mapped_gb300 as pkv
from paged_kv_cache_mapped_gb300 import _lib, header_constants

C = header_constants()
DEV = torch.device("cuda:0")


def _state(lens, hkv, d, mb, seed, q8=False, dropped=None, budget=0, extra=7, scores="exp"):
    """Numpy arrays of a cache of these lengths; sequences with dropped > 0 have explicit positions below `budget`."""
    rng = np.random.default_rng(seed)
    B = len(lens)
    lens = np.asarray(lens, dtype=np.int32)
    nblk = (lens + 15) // 16
    nb = int(nblk.sum()) + extra
    perm = rng.permutation(nb).astype(np.int32)
    bt = np.full((B, mb), -5, dtype=np.int32)
    at = 0
    for b in range(B):
        bt[b, :nblk[b]] = perm[at:at + nblk[b]]
        at += nblk[b]
    S = mb * 16
    dropped = np.zeros(B, dtype=np.int32) if dropped is None else np.asarray(dropped, dtype=np.int32)
    pos = np.full((B, hkv, S), -1, dtype=np.int32)
    for b in range(B):
        if dropped[b] > 0:
            old = int(dropped[b]) + budget   # positions from here on are in order, from slot `budget` on
            for g in range(hkv):
                pos[b, g, :budget] = rng.choice(old, budget, replace=False)
    sc = rng.exponential(size=(B, hkv, S)).astype(np.float32)
    if scores == "few":      # many equal ones
        sc = rng.integers(0, 3, size=sc.shape).astype(np.float32)
    elif scores == "zero":
        sc = np.where(rng.random(sc.shape) < 0.5, 0.0, -0.0).astype(np.float32)
    elif scores == "odd":    # infinities, negative and subnormal values, both zeros, wide exponents
        sc = (np.exp2(rng.uniform(-140, 120, sc.shape)) * rng.choice([-1, 1], sc.shape)).astype(np.float32)
        for x in (np.inf, -np.inf, 0.0, -0.0, 1e-45):
            sc[rng.random(sc.shape) < 0.05] = x
    if q8:
        pools = [rng.integers(0, 256, (nb, hkv, 16, d), dtype=np.uint8) for _ in range(2)]
        pools += [rng.random((nb, hkv, 16), dtype=np.float32) for _ in range(2)]
    else:
        pools = [rng.integers(-30000, 30000, (nb, hkv, 16, d), dtype=np.int16) for _ in range(2)]
    return dict(pools=pools, bt=bt, lens=lens, scores=sc, pos=pos, dropped=dropped, stack=[int(x) for x in perm[at:]], nb=nb)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _call(s, n_sink, k_top, n_recent, trigger=0, inplace=False, push=True, err=None, **kw):
    """The call on copies of the state; what it left, as numpy."""
    q8 = s["pools"][0].dtype == np.uint8
    pools = [_dev(p) if q8 else _dev(p).view(torch.bfloat16) for p in s["pools"]]
    lens, sc, pos, gone = _dev(s["lens"]), _dev(s["scores"]), _dev(s["pos"]), _dev(s["dropped"])
    free = torch.full((s["nb"],), -9, dtype=torch.int32, device=DEV)
    free[:len(s["stack"])] = torch.tensor(s["stack"], dtype=torch.int32, device=DEV)
    count = torch.tensor([len(s["stack"])], dtype=torch.int32, device=DEV)
    if push:
        kw.update(free_blocks=free, free_count=count)
    if inplace:
        kw.update(context_lens_out=lens, dropped_out=gone)
        so, po = sc, pos
        if push:
            kw.update(free_count_out=count)
    else:
        so, po = torch.full_like(sc, 77.0), torch.full_like(pos, -77)
        kw.update(scores_out=so, slot_pos_out=po)
    fn = pkv.kv_evict_q8 if q8 else pkv.kv_evict
    torch.cuda.synchronize()
    lo, go, co = fn(*pools, _dev(s["bt"]), lens, sc, pos, gone, n_sink, k_top, n_recent, trigger=trigger, error_word=err, **kw)
    torch.cuda.synchronize()
    assert (co is None) == (not push)
    got = [p.cpu().numpy() if q8 else p.view(torch.int16).cpu().numpy() for p in pools]
    stack = free[:int(co)].tolist() if push else None
    return got, lo.cpu().numpy(), so.cpu().numpy(), po.cpu().numpy(), go.cpu().numpy(), stack


def _check(s, got, n_sink, k_top, n_recent, trigger=0, inplace=False, push=True):
    want = evict_model.evict(s["pools"], [], s["bt"], s["lens"], s["scores"], s["pos"], s["dropped"], n_sink, k_top, n_recent, trigger,
                             s["stack"] if push else None)
    for a, b in zip(got[0], want[0]):
        assert np.array_equal(a, b)
    assert np.array_equal(got[1], want[1]) and np.array_equal(got[4], want[4])
    for b, L in enumerate(s["lens"].tolist()):
        assert np.array_equal(got[2][b, :, :L].view(np.int32), want[2][b, :, :L].view(np.int32)), b
        assert np.array_equal(got[3][b, :, :L], want[3][b, :, :L]), b
        if inplace:   # entries past the length stay
            assert np.array_equal(got[2][b, :, L:], s["scores"][b, :, L:]) and np.array_equal(got[3][b, :, L:], s["pos"][b, :, L:])
        else:
            assert (got[2][b, :, L:] == 77.0).all() and (got[3][b, :, L:] == -77).all()
    if push:
        assert got[5] == want[5]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,hkv,rules,kw", [
    ([300, 17, 0, 64, 65], 2, (4, 30, 30), {}),
    ([300, 290, 1], 1, (0, 1, 0), {}),
    ([100, 33, 32], 3, (0, 0, 0), {}),
    ([40, 41, 200], 2, (0, 0, 40), {}),
    ([40, 41, 200], 2, (40, 0, 0), {}),
    ([500, 499], 2, (3, 101, 57), dict(scores="few")),
    ([500, 499], 2, (3, 101, 57), dict(scores="zero")),
    ([777, 1200], 2, (5, 333, 7), dict(scores="odd")),
    ([2000, 1540, 1541], 8, (4, 512, 1024), {}),
    ([5000, 4097, 3000], 2, (1, 999, 31), dict(scores="few")),
    ([9000], 1, (4, 4000, 12), dict(scores="odd")),
])
@pytest.mark.parametrize("inplace", [False, True])
def test_fresh_sequences(lens, hkv, rules, kw, inplace):
    s = _state(lens, hkv, 64, (max(lens) + 15) // 16 + 2, 1, **kw)
    _check(s, _call(s, *rules, inplace=inplace), *rules, inplace=inplace)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("inplace", [False, True])
def test_shrunk_before(d, q8, inplace):
    rules, budget = (4, 60, 37), 101
    s = _state([150, 101, 102, 400, 180], 3, d, 30, 2, q8=q8, dropped=[70, 3, 1000, 1, 0], budget=budget, scores="few")
    for trigger in (0, 149, 150, 10**6):
        _check(s, _call(s, *rules, trigger=trigger, inplace=inplace), *rules, trigger=trigger, inplace=inplace)


@pytest.mark.gpu
def test_more_protected_than_the_budget_and_positions_at_their_ends():
    """Positions that name more protected tokens than there is room for (repeated ones): the lower slots stay."""
    s = _state([90, 90], 2, 64, 6, 3)
    s["pos"][:, :, :90] = 0
    s["pos"][1, 1, :] = 2**31 - 1
    _check(s, _call(s, 5, 10, 15), 5, 10, 15)
    s = _state([90], 2, 64, 6, 3, dropped=[2**31 - 91], budget=30)
    s["pos"][:] = -1
    _check(s, _call(s, 5, 10, 15), 5, 10, 15)


@pytest.mark.gpu
@pytest.mark.parametrize("q8", [False, True])
def test_rows_past_shared_memory(q8):
    lens = [50001, 49152, 60000]
    s = _state(lens, 1, 64, 3751, 4, q8=q8, scores="few")
    _check(s, _call(s, 4, 20000, 500), 4, 20000, 500)
    s = _state(lens, 1, 64, 3751, 5, q8=q8)
    _check(s, _call(s, 4, 333, 500), 4, 333, 500)


@pytest.mark.gpu
@pytest.mark.parametrize("scores", ["exp", "few"])
def test_the_longest_row(scores):
    most = C["PKV_MAX_EVICT_TOKENS"]
    s = _state([most], 1, 64, most // 16 + 3, 18, scores=scores)
    _check(s, _call(s, 4, 70001, 77), 4, 70001, 77)


@pytest.mark.gpu
def test_a_row_past_the_longest_is_refused():
    most = C["PKV_MAX_EVICT_TOKENS"]
    s = _state([most + 1, 500], 1, 64, most // 16 + 3, 18)
    err = pkv.new_error_word(DEV)
    got = _call(s, 4, 300, 77, err=err)
    assert pkv.read_error(err) == C["PKV_DEV_BAD_CONTEXT_LEN"]
    assert got[1].tolist() == [most + 1, 381] and got[4].tolist() == [0, 119]
    assert (got[2][0] == 77.0).all() and (got[3][0] == -77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[300, 290], [2000, 1999, 1733], [30011]])
def test_a_small_part_of_a_large_pool(lens):
    """Block ids far past the lengths: the lists of moves hold slots of the sequence, then slots of the pool."""
    s = _state(lens, 1, 64, max(lens) // 16 + 1, 21, extra=20000)
    for rules in ((4, 30, 41), (0, 137, 0)):
        _check(s, _call(s, *rules), *rules)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[20000, 9001], [33000], [8192, 8191, 16400, 4000]])
@pytest.mark.parametrize("scores", ["exp", "few", "zero", "odd"])
def test_rows_shared_by_clusters(lens, scores):
    s = _state(lens, 2, 64, max(lens) // 16 + 1, 19, scores=scores)
    for rules in ((4, 2000, 500), (0, 7999, 0)):
        _check(s, _call(s, *rules, inplace=True), *rules, inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[300, 290], [2001, 1999], [20003, 17001]])
@pytest.mark.parametrize("more", [0, 1, 2, 5])
def test_rows_of_odd_length(lens, more):
    """Rows of scores and positions that start anywhere."""
    s = _state(lens, 2, 64, max(lens) // 16 + 2, 22)
    for n in ("scores", "pos"):
        s[n] = s[n][:, :, :max(lens) + more].copy()
    for inplace in (False, True):
        _check(s, _call(s, 4, 60, 41, inplace=inplace), 4, 60, 41, inplace=inplace)


@pytest.mark.gpu
@pytest.mark.parametrize("mb,long", [(1100, [17600, 16384, 16385, 17001]), (2600, [41000, 16390, 33000]), (5000, [80000, 70001, 16385])])
@pytest.mark.parametrize("inplace", [False, True])
def test_many_sequences_in_wide_tables(mb, long, inplace):
    """More rows than CTAs at a time, most of them far shorter than the tables are wide, a few longer than one CTA takes."""
    rng = np.random.default_rng(mb)
    lens = rng.integers(0, 900, 82)
    lens[rng.choice(82, len(long), replace=False)] = long
    s = _state(lens.tolist(), 2, 64, mb, mb, scores="few" if inplace else "exp")
    for rules in ((4, 300, 41), (0, 9000, 0)):
        _check(s, _call(s, *rules, inplace=inplace), *rules, inplace=inplace)


@pytest.mark.gpu
def test_many_sequences():
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 90, 700).tolist()
    s = _state(lens, 2, 64, 6, 6)
    for push in (True, False):
        _check(s, _call(s, 2, 9, 20, trigger=40, push=push), 2, 9, 20, trigger=40, push=push)


@pytest.mark.gpu
def test_most_sequences_and_no_sequence():
    s = _state([20] * 4096, 1, 64, 2, 7)
    _check(s, _call(s, 1, 2, 3), 1, 2, 3)
    s = _state([], 1, 64, 2, 7)
    got = _call(s, 1, 2, 3)
    assert got[5] == s["stack"]


@pytest.mark.gpu
def test_nan_scores_are_the_lowest():
    s = _state([200, 150], 2, 64, 13, 8)
    s["scores"][0, 1, 30:80] = np.nan
    err = pkv.new_error_word(DEV)
    _check(s, _call(s, 4, 90, 16, err=err), 4, 90, 16)
    assert pkv.read_error(err) == C["PKV_DEV_BAD_SCORE"]
    s["scores"][:] = np.nan
    _check(s, _call(s, 4, 90, 16), 4, 90, 16)


@pytest.mark.gpu
def test_bad_lengths_leave_the_sequence_alone():
    s = _state([100, 90, 80, 70], 2, 64, 7, 9)
    lens, bad = s["lens"].copy(), {0: -1, 2: 7 * 16 + 1}
    for b, L in bad.items():
        s["lens"][b] = L
    s["dropped"][3] = -1
    err = pkv.new_error_word(DEV)
    got = _call(s, 4, 10, 16, err=err)
    assert pkv.read_error(err) == C["PKV_DEV_BAD_CONTEXT_LEN"]
    ok = dict(s, lens=np.array([0, 90, 0, 0], dtype=np.int32), dropped=np.zeros(4, dtype=np.int32))
    want = evict_model.evict(s["pools"], [], s["bt"], ok["lens"], s["scores"], s["pos"], ok["dropped"], 4, 10, 16, 0, s["stack"])
    for a, b in zip(got[0], want[0]):
        assert np.array_equal(a, b)
    assert got[1].tolist() == [-1, 30, 113, 70] and got[4].tolist() == [0, 60, 0, -1] and got[5] == want[5]
    for b in (0, 2, 3):
        assert (got[2][b] == 77.0).all() and (got[3][b] == -77).all()
    assert lens[1] == 90


@pytest.mark.gpu
def test_a_length_past_the_score_rows_is_refused():
    s = _state([100, 90], 2, 64, 7, 10)
    s["scores"], s["pos"] = s["scores"][:, :, :95].copy(), s["pos"][:, :, :95].copy()
    err = pkv.new_error_word(DEV)
    got = _call(s, 4, 10, 16, err=err)
    assert pkv.read_error(err) == C["PKV_DEV_BAD_CONTEXT_LEN"]
    assert got[1].tolist() == [100, 30] and (got[2][0] == 77.0).all()


@pytest.mark.gpu
def test_bad_blocks_are_skipped():
    s = _state([100, 120], 2, 64, 8, 11)
    want = evict_model.evict(s["pools"], [], s["bt"], s["lens"], s["scores"], s["pos"], s["dropped"], 4, 10, 16, 0, s["stack"])
    good = s["bt"].copy()
    s["bt"][0, 5] = s["nb"]       # behind the budget of 30: source of rows, and would be pushed
    s["bt"][1, 1] = -1            # takes rows
    err = pkv.new_error_word(DEV)
    got = _call(s, 4, 10, 16, err=err)
    assert pkv.read_error(err) == C["PKV_DEV_BAD_BLOCK_ID"]
    assert got[5] == [x for x in want[5] if x != good[0, 5]]
    assert np.array_equal(got[1], want[1])
    for b in range(2):
        L = int(s["lens"][b])
        assert np.array_equal(got[2][b, :, :L], want[2][b, :, :L]) and np.array_equal(got[3][b, :, :L], want[3][b, :, :L])
    for g, w, p in zip(got[0], want[0], s["pools"]):
        # a row is as the model has it or as it was
        same = (g == w).all(-1) | (g == p).all(-1)
        assert same.all()
        assert np.array_equal(g[good[1, 1]], p[good[1, 1]])
        assert np.array_equal(g[good[1, 0]], w[good[1, 0]])


@pytest.mark.gpu
def test_free_stack_that_overflows_or_is_out_of_range():
    s = _state([100, 120], 2, 64, 8, 12)
    want = evict_model.evict(s["pools"], [], s["bt"], s["lens"], s["scores"], s["pos"], s["dropped"], 4, 10, 16, 0, s["stack"])
    nb = s["nb"]
    s["stack"] = (s["stack"] * 20)[:nb - 3]
    err = pkv.new_error_word(DEV)
    got = _call(s, 4, 10, 16, err=err)
    assert pkv.read_error(err) == C["PKV_DEV_NO_BLOCKS"]
    assert len(got[5]) == nb and got[5][nb - 3:] == want[5][7:10]
    for count in (-1, nb + 1):
        free = torch.arange(nb, dtype=torch.int32, device=DEV)
        n = torch.tensor([count], dtype=torch.int32, device=DEV)
        err = pkv.new_error_word(DEV)
        pools = [_dev(p).view(torch.bfloat16) for p in s["pools"]]
        lo, _, co = pkv.kv_evict(*pools, _dev(s["bt"]), _dev(s["lens"]), _dev(s["scores"]), _dev(s["pos"]), _dev(s["dropped"]), 4, 10, 16,
                                 free_blocks=free, free_count=n, error_word=err)
        assert pkv.read_error(err) == C["PKV_DEV_NO_BLOCKS"]
        assert int(co) == count and free.tolist() == list(range(nb)) and lo.tolist() == [30, 30]


@pytest.mark.gpu
def test_guard_bands():
    """Nothing is written outside the arrays: they stand inside larger ones."""
    s = _state([300, 150], 2, 64, 19, 13)
    want = evict_model.evict(s["pools"], [], s["bt"], s["lens"], s["scores"], s["pos"], s["dropped"], 4, 30, 16, 0, s["stack"])
    pad = 64

    def inside(t):
        big = torch.full((t.numel() + 2 * pad,), 3, dtype=t.dtype, device=DEV)
        big[pad:-pad] = t.reshape(-1)
        return big, big[pad:-pad].view(t.shape)

    pools = [inside(_dev(p).view(torch.bfloat16)) for p in s["pools"]]
    sc, pos, lens, gone = (inside(_dev(s[n])) for n in ("scores", "pos", "lens", "dropped"))
    free = torch.full((s["nb"],), -9, dtype=torch.int32, device=DEV)
    free[:len(s["stack"])] = torch.tensor(s["stack"], dtype=torch.int32, device=DEV)
    free = inside(free)
    count = inside(torch.tensor([len(s["stack"])], dtype=torch.int32, device=DEV))
    ws = inside(torch.zeros(pkv.evict_workspace_bytes(2, 2, 4, 30, 16), dtype=torch.uint8, device=DEV))
    pkv.kv_evict(pools[0][1], pools[1][1], _dev(s["bt"]), lens[1], sc[1], pos[1], gone[1], 4, 30, 16, free_blocks=free[1],
                 free_count=count[1], context_lens_out=lens[1], dropped_out=gone[1], free_count_out=count[1], workspace=ws[1])
    torch.cuda.synchronize()
    for big, _ in pools + [sc, pos, lens, gone, free, count, ws]:
        assert (big[:pad] == 3).all() and (big[-pad:] == 3).all()
    assert np.array_equal(pools[0][1].view(torch.int16).cpu().numpy(), want[0][0])
    assert free[1][:int(count[1])].tolist() == want[5]


@pytest.mark.gpu
def test_other_stream_and_graph():
    rules = (4, 30, 16)
    s = _state([300, 150, 20], 2, 128, 19, 14)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _check(s, _call(s, *rules, stream=side), *rules)
    # captured once, replayed over other states in the same buffers
    ws = torch.zeros(pkv.evict_workspace_bytes(3, 2, *rules), dtype=torch.uint8, device=DEV)
    t = {n: _dev(s[n]) for n in ("bt", "lens", "scores", "pos", "dropped")}
    pools = [_dev(p).view(torch.bfloat16) for p in s["pools"]]
    free = torch.zeros(s["nb"], dtype=torch.int32, device=DEV)
    count = torch.zeros(1, dtype=torch.int32, device=DEV)

    def step():
        pkv.kv_evict(*pools, t["bt"], t["lens"], t["scores"], t["pos"], t["dropped"], *rules, trigger=60, free_blocks=free,
                     free_count=count, context_lens_out=t["lens"], dropped_out=t["dropped"], free_count_out=count, workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, lens in ((15, [300, 150, 20]), (16, [61, 60, 304]), (17, [0, 1, 2])):
        s = _state(lens, 2, 128, 19, seed, extra=t["bt"].shape[0] * 19)
        nb = pools[0].shape[0]
        s["bt"] = np.where(s["bt"] >= 0, s["bt"] % nb, s["bt"])
        used = s["bt"][s["bt"] >= 0]
        if len(set(used.tolist())) != len(used):   # blocks of one pool, each owned once
            perm = np.random.default_rng(seed).permutation(nb)
            s["bt"][s["bt"] >= 0] = perm[:len(used)]
        s["pools"] = [p[:nb] for p in s["pools"]]
        s["stack"], s["nb"] = [5, 3, 1], nb
        for n in t:
            t[n].copy_(_dev(s[n]))
        for p, q in zip(pools, s["pools"]):
            p.view(torch.int16).copy_(_dev(q))
        free[:3] = torch.tensor(s["stack"], dtype=torch.int32, device=DEV)
        count.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        got = ([p.view(torch.int16).cpu().numpy() for p in pools], t["lens"].cpu().numpy(), t["scores"].cpu().numpy(),
               t["pos"].cpu().numpy(), t["dropped"].cpu().numpy(), free[:int(count)].tolist())
        _check(s, got, *rules, trigger=60, inplace=True)


@pytest.mark.gpu
def test_run_of_tables_append_scores_and_eviction():
    """An engine's steps: every request decodes a token a step and is cut back each time it passes the trigger.  The output is that of
    64-bit attention over the kept tokens, blocks stay owned once, positions run on."""
    B, hq, hkv, d, mb, nb = 3, 4, 2, 64, 6, 12
    n_sink, k_top, n_recent, trigger = 2, 9, 10, 29
    budget, scale = n_sink + k_top + n_recent, 0.125
    g = torch.Generator(device=DEV).manual_seed(20)
    kc, vc = (torch.randn((nb, hkv, 16, d), generator=g, device=DEV).bfloat16() for _ in range(2))
    bt = torch.full((B, mb), -1, dtype=torch.int32, device=DEV)
    lens, gone = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2))
    free, count = torch.arange(nb, dtype=torch.int32, device=DEV), torch.tensor([nb], dtype=torch.int32, device=DEV)
    scores = torch.zeros((B, hkv, mb * 16), device=DEV)
    pos = torch.full((B, hkv, mb * 16), -1, dtype=torch.int32, device=DEV)
    held = [[{} for _ in range(hkv)] for _ in range(B)]   # position -> (K row, V row, score)
    err = pkv.new_error_word(DEV)
    cuts = 0
    for step in range(80):
        new = torch.tensor([1, 1 if step >= 7 else 0, 2 if step % 3 == 0 else 1], dtype=torch.int32, device=DEV)
        first = (lens + gone).tolist()
        lens, starts, slots, _, count = pkv.kv_step_tables(bt, lens, new, free, count, 4, error_word=err)
        k, v = (torch.randn((4, hkv, d), generator=g, device=DEV).bfloat16() for _ in range(2))
        pkv.kv_append(kc, vc, k, v, slots, error_word=err)
        q = torch.randn((B, hq, d), generator=g, device=DEV).bfloat16()
        out, lse = pkv.paged_decode_attention_scores(q, kc, vc, bt, lens, scale, scores, error_word=err)[:2]
        at, n = starts.tolist(), new.tolist()
        for b in range(B):
            for h in range(hkv):
                for i in range(n[b]):
                    held[b][h][first[b] + i] = [k[at[b] + i, h].double(), v[at[b] + i, h].double(), 0.0]
            if not held[b][0]:
                continue
            for h in range(hq):
                rows = held[b][h // 2]
                ks, vs = (torch.stack([r[j] for r in rows.values()]) for j in range(2))
                p = torch.softmax(ks @ q[b, h].double() * scale, 0)
                for r, x in zip(rows.values(), p.tolist()):
                    r[2] += x
                want = p @ vs
                # bf16 output: half a step of the value; weights of two bf16 terms: 2^-16 of what they carry; logits and sums in fp32
                tol = want.abs() * 2**-8 + (p @ vs.abs()) * (2**-16 + 64 * 2**-24) + 1e-9
                assert ((out[b, h].double() - want).abs() <= tol).all(), (step, b, h)
        lens_was = lens.tolist()
        lens, gone, count = pkv.kv_evict(kc, vc, bt, lens, scores, pos, gone, n_sink, k_top, n_recent, trigger=trigger, free_blocks=free,
                                         free_count=count, error_word=err)
        L, lost, sc, ps = lens.tolist(), gone.tolist(), scores.cpu().numpy(), pos.cpu().numpy()
        for b in range(B):
            seen = L[b] + lost[b]
            assert seen == first[b] + n[b]
            if lens_was[b] <= trigger:
                assert L[b] == lens_was[b]
                continue
            cuts += 1
            assert L[b] == budget
            for h in range(hkv):
                kept = ps[b, h, :budget].tolist()
                assert set(range(n_sink)) <= set(kept) and set(range(seen - n_recent, seen)) <= set(kept) and len(set(kept)) == budget
                # each kept token's score is what the steps gave it, and no evicted one's is clearly above a kept one's
                for i, t in enumerate(kept):
                    assert abs(sc[b, h, i] - held[b][h][t][2]) <= 1e-5 * (1 + held[b][h][t][2])
                rest = [r[2] for t, r in held[b][h].items() if t not in kept]
                free_kept = [held[b][h][t][2] for t in kept if n_sink <= t < seen - n_recent]
                assert max(rest) <= min(free_kept) + 1e-5
                held[b][h] = {t: held[b][h][t] for t in kept}
        owned = [int(x) for b in range(B) for x in bt[b, :(L[b] + 15) // 16].tolist()] + free[:int(count)].tolist()
        assert sorted(owned) == list(range(nb))
    assert pkv.read_error(err) == 0 and cuts >= 15


# ------------------------------------------------------------------------------------- refusals (no GPU)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_mapped_gb300 import _build
    _build.build()
    return _lib.load()


def test_header_is_exported(lib):
    names = _lib.header_functions(_lib.EVICT_HEADER)
    assert names == ["pkv_evict_workspace_bytes", "pkv_kv_evict", "pkv_kv_evict_q8"]
    for n in names:
        assert hasattr(lib, n), n


def test_host_validation_codes(lib):
    P = ctypes.c_void_p

    def dims(B=4, hkv=8, d=128, bs=16, nb=1000, mb=64):
        return ctypes.byref(_lib.PkvDims(B, 1, hkv, d, bs, nb, mb))

    def rules(a=4, b=8, c=8, trigger=0):
        return ctypes.byref(_lib.PkvEvictRules(a, b, c, trigger))

    def state(sc=0x10000, po=0x10000, gone=0x10000, stride=1024):
        return ctypes.byref(_lib.PkvEvictState(sc, sc, po, po, gone, gone, stride))

    def call(st=None, r=None, d=None, k=0x10000, bt=0x10000, free=0x10000, count=0x10000, ws=0x10000, n=1 << 30, err=None, q8=False):
        st, r, d = st or state(), r or rules(), d or dims()
        rest = (P(bt), P(0x10000), P(0x10000), st, r, P(free), P(count), P(count), P(ws), n, d, P(err), None)
        if q8:
            return lib.pkv_kv_evict_q8(P(k), P(k), P(0x10000), P(0x10008 if q8 == "odd" else 0x10000), *rest)
        return lib.pkv_kv_evict(P(k), P(k), *rest)

    assert call(r=rules(a=-1)) == call(r=rules(b=-1)) == call(r=rules(c=-1)) == C["PKV_ERR_ARGUMENT"]
    assert call(r=rules(b=2**30)) == call(r=rules(2**29, 2**29, 0)) == C["PKV_ERR_ARGUMENT"]
    assert call(d=dims(B=4097)) == call(d=dims(B=-1)) == call(d=dims(mb=1 << 28)) == call(d=dims(hkv=0)) == C["PKV_ERR_DIMS"]
    assert call(d=dims(hkv=1 << 23)) == call(d=dims(nb=1 << 27)) == call(st=state(stride=-1)) == C["PKV_ERR_DIMS"]
    assert call(d=dims(bs=8)) == C["PKV_ERR_BLOCK_SIZE"] and call(d=dims(d=96)) == C["PKV_ERR_HEAD_DIM"]
    for kw in (dict(k=None), dict(bt=None), dict(count=None), dict(st=state(sc=None)), dict(st=state(po=None)), dict(st=state(gone=None))):
        assert call(**kw) == C["PKV_ERR_NULL_POINTER"], kw
    assert call(ws=None) == call(n=16) == C["PKV_ERR_WORKSPACE"]
    for kw in (dict(k=0x10008), dict(bt=0x10002), dict(free=0x10001), dict(st=state(sc=0x10002)), dict(ws=0x10004), dict(err=0x10001),
               dict(q8="odd")):
        assert call(**kw) == C["PKV_ERR_ALIGNMENT"], kw
    assert call(d=dims(B=0), free=None) == C["PKV_OK"]
    assert lib.pkv_kv_evict(P(16), P(16), P(16), P(16), P(16), None, rules(), None, None, None, P(16), 1 << 30, dims(), None,
                            None) == C["PKV_ERR_NULL_POINTER"]
    assert lib.pkv_evict_workspace_bytes(dims(), None) == 0 and lib.pkv_evict_workspace_bytes(dims(B=4097), rules()) == 0
    n = lib.pkv_evict_workspace_bytes(dims(), rules())
    assert n >= 4 * 8 * 20 * 8 and n % 256 == 0 and lib.pkv_evict_workspace_bytes(dims(B=0), rules()) > 0


def test_binding_refusals():
    t = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_evict(t, t, i[None], i, torch.zeros(1, 2, 16), torch.zeros(1, 2, 16, dtype=torch.int32), i, 1, 1, 1)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_evict_q8(t.byte(), t.byte(), t[..., 0].float(), t[..., 0].float(), i[None], i, torch.zeros(1, 2, 16),
                        torch.zeros(1, 2, 16, dtype=torch.int32), i, 1, 1, 1)
    with pytest.raises(TypeError):
        pkv.kv_evict(t.float(), t, i[None], i, t, t, i, 1, 1, 1)
    for bad in ((-1, 1, 1), (1, 2**30, 1), (1, 1, 2**31), (2**32, 1, 1)):
        with pytest.raises(ValueError, match="within"):
            pkv.evict_workspace_bytes(2, 2, *bad)
    for sizes in ((5000, 2), (2**32 + 1, 2), (-1, 2), (2, 0)):
        with pytest.raises(ValueError):
            pkv.evict_workspace_bytes(*sizes, 1, 1, 1)


@pytest.mark.gpu
def test_binding_refuses_wrong_shapes_and_types():
    s = _state([40, 50], 2, 64, 4, 23)
    pools = [_dev(p).view(torch.bfloat16) for p in s["pools"]]
    t = dict(bt=_dev(s["bt"]), lens=_dev(s["lens"]), sc=_dev(s["scores"]), pos=_dev(s["pos"]), gone=_dev(s["dropped"]))
    free, count = torch.zeros(s["nb"], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    before = [p.clone() for p in pools]

    def call(n=(4, 10, 10), kw=None, **x):
        a = dict(t, **x)
        return pkv.kv_evict(*pools, a["bt"], a["lens"], a["sc"], a["pos"], a["gone"], *n, **(kw or {}))

    for x in (dict(lens=t["lens"][:1]), dict(gone=t["gone"][:1]), dict(sc=t["sc"][:, :1].contiguous()), dict(sc=t["sc"][:1]),
              dict(pos=t["pos"][:, :, :32].contiguous()), dict(bt=t["bt"].t()), dict(sc=t["sc"].cpu()), dict(bt=t["bt"][0])):
        with pytest.raises(ValueError):
            call(**x)
    for x in (dict(sc=t["sc"].double()), dict(pos=t["pos"].long()), dict(lens=None)):
        with pytest.raises(TypeError):
            call(**x)
    for kw in (dict(free_blocks=free), dict(free_count=count), dict(free_count_out=count), dict(free_blocks=free[:3], free_count=count),
               dict(free_blocks=free, free_count=free), dict(scores_out=t["sc"][:1]), dict(context_lens_out=count),
               dict(workspace=torch.zeros(16, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call(kw=kw)
    with pytest.raises(pkv.PkvError):
        call(kw=dict(workspace=torch.zeros(16, dtype=torch.uint8, device=DEV)))
    for n in ((-1, 1, 1), (1, 2**30, 1)):
        with pytest.raises(ValueError):
            call(n)
    with pytest.raises(pkv.PkvError):
        call((2**29, 2**29, 2**29))
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(pools, before))
