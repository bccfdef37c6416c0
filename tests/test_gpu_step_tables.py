"""pkv_kv_step_tables against a plain host model of the free stack, exactly: growth, release and
admission in one step, empty and idle sequences, exact fits, padding rows, in-place lengths, and the
all-or-nothing refusals; a run of steps keeps every block owned once; and a captured step replayed
with new counts."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
from paged_kv_cache_mapped_gb300 import header_constants

C = header_constants()
DEV = torch.device("cuda:0")


def _model(bt, lens, new, stack, T):
    """The step on host lists; `stack` is the live free list.  Returns copies after the step."""
    bt, stack = bt.copy(), list(stack)
    for b in range(len(lens)):
        if new[b] < 0:
            stack += [int(x) for x in bt[b, : (lens[b] + 15) // 16]]
    starts, slots, pos, out = [0], [], [], []
    for b in range(len(lens)):
        n = max(int(new[b]), 0)
        held, need = (lens[b] + 15) // 16, (lens[b] + n + 15) // 16
        if n > 0:
            for j in range(held, need):
                bt[b, j] = stack.pop()
        for i in range(n):
            t = lens[b] + i
            slots.append(int(bt[b, t // 16]) * 16 + t % 16)
            pos.append(t)
        starts.append(starts[-1] + n)
        out.append(0 if new[b] < 0 else lens[b] + n)
    pad = T - len(slots)
    return bt, out, starts, slots + [-1] * pad, pos + [-1] * pad, stack


def _state(lens, mb, nb, seed, free=None):
    rng = np.random.default_rng(seed)
    perm = rng.permutation(nb)
    bt = np.full((len(lens), mb), -7, dtype=np.int32)
    at = 0
    for b, L in enumerate(lens):
        h = (L + 15) // 16
        bt[b, :h] = perm[at:at + h]
        at += h
    stack = perm[at:] if free is None else perm[at:at + free]
    return bt, [int(x) for x in stack]


def _dev(a, dtype=torch.int32):
    return torch.as_tensor(np.asarray(a), dtype=dtype, device=DEV)


def _run(bt, lens, new, stack, nb, T, err=None, **kw):
    free = torch.full((nb,), -9, dtype=torch.int32, device=DEV)
    free[: len(stack)] = _dev(stack)
    t = _dev(bt)
    lens_out, starts, slots, pos, count = pkv.kv_step_tables(t, _dev(lens), _dev(new), free, _dev([len(stack)]), T,
                                                             error_word=err, **kw)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (t, lens_out, starts, slots, pos, count, free)]


def _check(got, want):
    t, lens_out, starts, slots, pos, count, free = got
    bt, out, st, sl, po, stack = want
    assert np.array_equal(t, bt)
    assert lens_out.tolist() == out and starts.tolist() == st
    assert slots.tolist() == sl and pos.tolist() == po
    assert count.tolist() == [len(stack)] and free[: len(stack)].tolist() == stack


CASES = {
    "one token": ([0], [1], 1),
    "idle": ([5, 0], [0, 0], 3),
    "block edges": ([15, 16, 17, 31, 32, 0], [1, 1, 1, 2, 16, 17], 64),
    "release and admit": ([40, 0, 16, 1, 100], [-1, 33, -1, 1, -1], 40),
    "release empty": ([0, 3], [-1, 1], 1),
    "long prompt": ([7, 0, 64], [1, 5000, 3], 5100),
    "nothing": ([], [], 4),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", CASES)
def test_step_matches_the_model(name):
    lens, new, T = CASES[name]
    mb = 320
    need = sum((L + 15) // 16 for L in lens) + sum((max(n, 0) + 31) // 16 for n in new) + 4
    bt, stack = _state(lens, mb, need, 3)
    err = pkv.new_error_word(DEV)
    got = _run(bt, lens, new, stack, need, T, err)
    assert pkv.read_error(err) == 0
    _check(got, _model(bt, lens, new, stack, T))


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 31, 1023, 1024, 1025, 4096])
def test_batch_sizes(B):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 300, B)
    kind = rng.random(B)
    new = np.where(kind < 0.6, 1, np.where(kind < 0.75, -1, np.where(kind < 0.85, 0, rng.integers(0, 90, B))))
    T = int(np.maximum(new, 0).sum())
    nb = int(((lens + 15) // 16).sum() + (np.maximum(new, 0) // 16 + 2).sum())
    bt, stack = _state(lens, 26, nb, B + 1)
    _check(_run(bt, lens, new, stack, nb, T), _model(bt, lens, new, stack, T))


@pytest.mark.gpu
def test_exact_fit_of_tokens_and_blocks():
    lens, new = [16, 0, 3], [16, 32, 13]
    bt, stack = _state(lens, 4, 2 + 3, 1)
    assert len(stack) == 3
    _check(_run(bt, lens, new, stack, 5, 61), _model(bt, lens, new, stack, 61))


def _refusals():
    ok = dict(lens=[20, 5, 0], new=[1, 12, 40], mb=4, nb=20, T=64)
    yield "too many tokens", dict(ok, T=52), C["PKV_DEV_BAD_QUERY_RANGE"]
    yield "count below -1", dict(ok, new=[1, -2, 3]), C["PKV_DEV_BAD_QUERY_RANGE"]
    yield "past the table", dict(ok, new=[45, 1, 1]), C["PKV_DEV_BAD_CONTEXT_LEN"]
    yield "huge count", dict(ok, new=[2**31 - 1, 1, 1]), C["PKV_DEV_BAD_CONTEXT_LEN"]
    yield "negative length", dict(ok, lens=[-1, 5, 0], held=[20, 5, 0]), C["PKV_DEV_BAD_CONTEXT_LEN"]
    yield "too few blocks", dict(ok, free=3), C["PKV_DEV_NO_BLOCKS"]
    yield "count past the stack", dict(ok, count=21), C["PKV_DEV_NO_BLOCKS"]
    yield "negative count", dict(ok, count=-1), C["PKV_DEV_NO_BLOCKS"]
    yield "freed twice", dict(ok, new=[-1, 0, 0], count=19), C["PKV_DEV_NO_BLOCKS"]
    yield "bad pushed block", dict(ok, new=[-1, 0, 0], put=(0, 1, 20)), C["PKV_DEV_BAD_BLOCK_ID"]
    yield "bad held block", dict(ok, put=(0, 1, -1)), C["PKV_DEV_BAD_BLOCK_ID"]
    yield "bad free block", dict(ok, top=20), C["PKV_DEV_BAD_BLOCK_ID"]


@pytest.mark.gpu
@pytest.mark.parametrize("name,c,code", list(_refusals()), ids=[r[0] for r in _refusals()])
def test_refusals_change_nothing(name, c, code):
    lens, new, nb, T = c["lens"], c["new"], c["nb"], c["T"]
    bt, stack = _state(c.get("held", lens), c["mb"], nb, 5, c.get("free"))
    if "put" in c:
        b, j, v = c["put"]
        bt[b, j] = v
    if "top" in c:
        stack[-1] = c["top"]
    free = torch.full((nb,), 11, dtype=torch.int32, device=DEV)
    free[: len(stack)] = _dev(stack)
    count = c.get("count", len(stack))
    t, ld, err = _dev(bt), _dev(lens), pkv.new_error_word(DEV)
    lo, starts, slots, pos, co = pkv.kv_step_tables(t, ld, _dev(new), free, _dev([count]), T, error_word=err)
    assert pkv.read_error(err) == code
    assert np.array_equal(t.cpu().numpy(), bt) and lo.tolist() == list(lens) and co.tolist() == [count]
    assert starts.tolist() == [0] * (len(lens) + 1)
    assert slots.tolist() == [-1] * T and pos.tolist() == [-1] * T
    assert free[: len(stack)].tolist() == stack


@pytest.mark.gpu
def test_steps_in_place_and_in_a_graph():
    """Thirty steps over one state, lengths and count updated in place, the step captured once and
    replayed with new counts; every block is owned once or free after each."""
    rng = np.random.default_rng(9)
    B, mb, nb, T = 24, 12, 150, 64
    bt, lens, stack = np.full((B, mb), -1, dtype=np.int32), [0] * B, list(rng.permutation(nb))
    t, ld, new, count = _dev(bt), _dev(lens), _dev([0] * B), _dev([nb])
    free = _dev(stack)
    starts = torch.empty(B + 1, dtype=torch.int32, device=DEV)
    slots, pos = torch.empty(T, dtype=torch.int64, device=DEV), torch.empty(T, dtype=torch.int32, device=DEV)
    err = pkv.new_error_word(DEV)

    def step():
        pkv.kv_step_tables(t, ld, new, free, count, T, context_lens_out=ld, free_count_out=count, query_starts=starts,
                           slot_mapping=slots, positions=pos, error_word=err)

    step()  # an idle step: one-time set-up before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(30):
        want, left, room = [], T, len(stack)
        for b in range(B):
            n = int(rng.choice([-1, 0, 1, 1, 1, 9])) if lens[b] else int(rng.integers(0, 30))
            n = min(n, left, mb * 16 - lens[b])
            cost = (lens[b] + max(n, 0) + 15) // 16 - (lens[b] + 15) // 16
            if cost > room:
                n, cost = 0, 0
            left, room = left - max(n, 0), room - cost
            want.append(n)
        bt, lens, st, sl, po, stack = _model(bt, lens, want, stack, T)
        new.copy_(_dev(want))
        g.replay()
        assert pkv.read_error(err) == 0
        assert np.array_equal(t.cpu().numpy(), bt) and ld.tolist() == lens and count.tolist() == [len(stack)]
        assert starts.tolist() == st and slots.tolist() == sl and pos.tolist() == po
        owned = [int(x) for b in range(B) for x in bt[b, : (lens[b] + 15) // 16]]
        assert sorted(owned + [int(x) for x in stack]) == list(range(nb))


@pytest.mark.gpu
def test_capacity_step_of_one_sequence():
    """The most tokens that one call takes, all of one sequence, on a stream of its own."""
    T = C["PKV_MAX_STEP_TOKENS"]
    bt, stack = _state([9], T // 16 + 1, T // 16 + 3, 2)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = _run(bt, [9], [T], stack, T // 16 + 3, T)
    _check(got, _model(bt, [9], [T], stack, T))


def test_host_refusals():
    t = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pkv.kv_step_tables(t, t[:, 0], t[:, 0], t[0], t[0, :1], 4)
    with pytest.raises(TypeError, match="int32"):
        pkv.kv_step_tables(t.long(), t[:, 0], t[:, 0], t[0], t[0, :1], 4)
    with pytest.raises(TypeError, match="Tensor"):
        pkv.kv_step_tables([[0]], t[:, 0], t[:, 0], t[0], t[0, :1], 4)
