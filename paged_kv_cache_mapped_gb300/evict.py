"""Binding of eviction from the paged cache (declared in include/pkv_evict.h): sequences past a limit shrink
in place to their sinks, their recent window and the tokens of the most accumulated attention weight.  As the
rest of the package: argument checks and marshalling only."""
from __future__ import annotations

import ctypes
import functools

import torch

from ._lib import PkvEvictRules, PkvEvictState, load
from .step import BLOCK_SIZE, _bf16_pools, _call, _dims, _give, _like, _need, _new, _sizes


@functools.lru_cache(maxsize=256)
def _record(n_sink, k_top, n_recent, trigger):
    return ctypes.pointer(PkvEvictRules(n_sink, k_top, n_recent, trigger))


def _rules(n_sink, k_top, n_recent, trigger=0):
    # (the record is kept by these numbers, not by the arguments: a tensor of one would be kept by its identity)
    n_sink, k_top, n_recent = int(n_sink), int(k_top), int(n_recent)
    for name, x in (("n_sink", n_sink), ("k_top", k_top), ("n_recent", n_recent)):
        if not 0 <= x < 2**30:
            raise ValueError(f"{name} must be within [0, 2**30), got {x}")
    return _record(n_sink, k_top, n_recent, max(0, min(int(trigger), 2**31 - 1)))


def evict_workspace_bytes(batch, num_kv_heads, n_sink, k_top, n_recent) -> int:
    """Workspace of kv_evict and kv_evict_q8 for these sizes."""
    n = int(load().pkv_evict_workspace_bytes(_sizes(batch, 1, num_kv_heads, 128, 0, 0), _rules(n_sink, k_top, n_recent)))
    if n == 0:
        raise ValueError("invalid sizes for an eviction")
    return n


def _evict(name, pools, hkv, d, nb, dev, block_tables, context_lens, scores, slot_pos, dropped, n_sink, k_top, n_recent, trigger,
           free_blocks, free_count, context_lens_out, scores_out, slot_pos_out, dropped_out, free_count_out, workspace, error_word,
           stream):
    bt = _need(block_tables, "block_tables", torch.int32, 2, dev)
    lens = _need(context_lens, "context_lens", torch.int32, 1, dev)
    sp = _need(scores, "scores", torch.float32, 3, dev)
    pp = _need(slot_pos, "slot_pos", torch.int32, 3, dev)
    dp = _need(dropped, "dropped", torch.int32, 1, dev)
    err = None if error_word is None else _need(error_word, "error_word", torch.int32, 1, dev)
    B, mb = block_tables.shape
    stride = scores.shape[2]
    if context_lens.shape[0] != B or dropped.shape[0] != B:
        raise ValueError("context_lens / dropped batch differs from block_tables'")
    if scores.shape != (B, hkv, stride) or slot_pos.shape != scores.shape:
        raise ValueError("scores and slot_pos must have one shape [batch, num_kv_heads, slots]")
    if stride >= 2**31:
        raise ValueError(f"sizes must be within [0, 2**31), got {stride}")
    if (free_blocks is None) != (free_count is None) or (free_count_out is not None and free_count is None):
        raise ValueError("free_blocks and free_count come together")
    rules = _rules(n_sink, k_top, n_recent, trigger)
    dims = _dims(B, 1, hkv, d, nb, mb)
    lens_out, lp = _like(context_lens_out, "context_lens_out", context_lens, dev, stream)
    gone_out, gp = _like(dropped_out, "dropped_out", dropped, dev, stream)
    sop = sp if scores_out is None else _give(scores_out, "scores_out", scores.shape, torch.float32, scores, dev, stream)[1]
    pop = pp if slot_pos_out is None else _give(slot_pos_out, "slot_pos_out", scores.shape, torch.int32, scores, dev, stream)[1]
    free = count = cp = count_out = None
    if free_blocks is not None:
        free = _need(free_blocks, "free_blocks", torch.int32, 1, dev)
        count = _need(free_count, "free_count", torch.int32, 1, dev)
        if free_blocks.shape[0] != nb or free_count.shape[0] != 1:
            raise ValueError("free_blocks must be [num_blocks] and free_count [1]")
        count_out, cp = _like(free_count_out, "free_count_out", free_count, dev, stream)
    if workspace is None:
        n = int(load().pkv_evict_workspace_bytes(dims, rules))
        workspace = _new((n,), torch.uint8, block_tables, stream)
    wp = _need(workspace, "workspace", torch.uint8, 1, dev)
    state = PkvEvictState(sp, sop, pp, pop, dp, gp, stride)
    _call(name, dev, stream, *pools, bt, lens, lp, ctypes.byref(state), rules, free, count, cp, wp, workspace.numel(),
          dims, err)
    return lens_out, gone_out, count_out


def kv_evict(k_cache, v_cache, block_tables, context_lens, scores, slot_pos, dropped, n_sink, k_top, n_recent, *, trigger=0,
             free_blocks=None, free_count=None, context_lens_out=None, scores_out=None, slot_pos_out=None, dropped_out=None,
             free_count_out=None, workspace=None, error_word=None, stream=None):
    """Shrink every sequence of more than max(trigger, budget) cached tokens to the budget n_sink + k_top +
    n_recent, in place: per kv head the tokens of position < n_sink, those of the last n_recent positions and the
    others of highest accumulated weight stay, and kept rows behind the budget move into the places of evicted ones.
    scores [B, Hkv, S] fp32 and slot_pos [B, Hkv, S] int32 (the position of each slot's token, -1: in order,
    slot + dropped[b]) go with them, in place unless scores_out / slot_pos_out are given.  dropped [B] int32
    counts the tokens lost; the positions of kv_step_tables are slots, to which dropped[b] adds up to a later token's own
    position.  With free_blocks [NB] and free_count [1] (the stack of kv_step_tables) the blocks
    behind the budget are pushed.  Returns (context_lens_out [B], dropped_out [B], free_count_out [1] or None); the
    outputs may be the inputs themselves."""
    nb, hkv, d, dev, kp, vp = _bf16_pools(k_cache, v_cache)
    return _evict("pkv_kv_evict", (kp, vp), hkv, d, nb, dev, block_tables, context_lens, scores, slot_pos, dropped, n_sink, k_top,
                  n_recent, trigger, free_blocks, free_count, context_lens_out, scores_out, slot_pos_out, dropped_out,
                  free_count_out, workspace, error_word, stream)


def kv_evict_q8(k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, scores, slot_pos, dropped, n_sink, k_top, n_recent,
                *, trigger=0, free_blocks=None, free_count=None, context_lens_out=None, scores_out=None, slot_pos_out=None,
                dropped_out=None, free_count_out=None, workspace=None, error_word=None, stream=None):
    """kv_evict over INT8 pools (codes [NB, Hkv, 16, d] uint8, row scales [NB, Hkv, 16] fp32)."""
    kp = _need(k_codes, "k_codes", torch.uint8, 4)
    dev = k_codes.get_device()
    vp = _need(v_codes, "v_codes", torch.uint8, 4, dev)
    ksp = _need(k_scales, "k_scales", torch.float32, 3, dev)
    vsp = _need(v_scales, "v_scales", torch.float32, 3, dev)
    nb, hkv, bs, d = k_codes.shape
    if v_codes.shape != k_codes.shape or bs != BLOCK_SIZE:
        raise ValueError(f"pools must have one shape [num_blocks, num_kv_heads, {BLOCK_SIZE}, head_dim]")
    if k_scales.shape != (nb, hkv, BLOCK_SIZE) or v_scales.shape != k_scales.shape:
        raise ValueError("scale pools must be [num_blocks, num_kv_heads, 16]")
    return _evict("pkv_kv_evict_q8", (kp, vp, ksp, vsp), hkv, d, nb, dev, block_tables, context_lens, scores, slot_pos, dropped,
                  n_sink, k_top, n_recent, trigger, free_blocks, free_count, context_lens_out, scores_out, slot_pos_out, dropped_out,
                  free_count_out, workspace, error_word, stream)
