"""Binding of the serving-step operators (declared in include/pkv_step.h): the step's block tables
and slots, the FP8 cache with one scale per (block, kv head), and attention with score rules for one
query token and for many.  As the rest of the package: argument checks and marshalling only, the
work runs in the library's CUDA kernels on the current stream of the tensors' device."""
from __future__ import annotations

import ctypes
import functools
import operator

import torch

from ._lib import PkvDims, PkvScoreRules, check, header_constants, load

BLOCK_SIZE = 16
_INPUTS_READY = header_constants()["PKV_DECODE_INPUTS_READY"]


def _need(t, name, dtype, ndim, device=-1):
    """The tensor's address, once it is what the kernels take: on CUDA device number `device` (-1: any)."""
    try:
        if (t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.dim() == ndim
                and (device < 0 or t.get_device() == device)):
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got shape {tuple(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{device}")


def _opt(t, name, dtype, ndim, device):
    return None if t is None else _need(t, name, dtype, ndim, device)


_functions = {}


def _call(name, device, stream, *args):
    """Calls pkv_<name>(*args, stream) with CUDA device number `device` current."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(load(), name)
    if torch._C._cuda_getDevice() == device:
        s = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
        status = fn(*args, s)
    else:
        with torch.cuda.device(device):
            s = torch._C._cuda_getCurrentRawStream(device) if stream is None else stream.cuda_stream
            status = fn(*args, s)
    if status:
        check(name, status)


@functools.lru_cache(maxsize=256)
def _dims(batch, hq, hkv, d, nb, mb):
    """The shape record's address (records of the same sizes are one; ctypes would cut a size to 32 bits)."""
    for x in (batch, hq, hkv, d, nb, mb):
        if not 0 <= x < 2**31:
            raise ValueError(f"sizes must be within [0, 2**31), got {x}")
    r = PkvDims(batch, hq, hkv, d, BLOCK_SIZE, nb, mb)
    return ctypes.pointer(r)


def _sizes(*sizes):
    """_dims of sizes that a caller names: the record is kept by the numbers (a tensor of one would be kept by its
    identity, and count as it once was)."""
    return _dims(*(operator.index(x) for x in sizes))


def _new(shape, dtype, like, stream, make=torch.empty):
    """A new tensor on `like`'s device, made (and zeroed) in the order of the call's own stream: a caching
    allocator may hand its memory out again once it is freed there."""
    if stream is None:
        return make(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=like.device)


def _give(t, name, shape, dtype, like, device, stream):
    """The output `t` after its checks, or a new one on `like`'s device; with its address."""
    if t is None:
        t = _new(shape, dtype, like, stream)
        return t, t.data_ptr()
    ptr = _need(t, name, dtype, len(shape), device)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t, ptr


def _like(t, name, like, device, stream):
    """The output `t` of `like`'s shape and type after its checks, or a new one; with its address."""
    if t is None and stream is None:
        t = torch.empty_like(like)
        return t, t.data_ptr()
    return _give(t, name, like.shape, like.dtype, like, device, stream)


def kv_step_tables(block_tables, context_lens, new_tokens, free_blocks, free_count, max_new_tokens, *,
                   context_lens_out=None, free_count_out=None, query_starts=None, slot_mapping=None, positions=None,
                   error_word=None, stream=None):
    """One step's block tables and slots: new_tokens[b] > 0 gives sequence b that many tokens, 0 leaves
    it, -1 ends it and frees its blocks.  block_tables [B, MB] and the free stack free_blocks [NB]
    (live: the first free_count [1] entries) are updated in place.  Returns (context_lens_out [B],
    query_starts [B + 1], slot_mapping [max_new_tokens] int64, positions [max_new_tokens],
    free_count_out [1]); rows past the step's last token have slot and position -1.  context_lens_out
    and free_count_out may be the inputs themselves.  All or nothing on a device error (see
    pkv_kv_step_tables)."""
    T = int(max_new_tokens)
    if not 0 <= T < 2**31:  # (the library refuses what is past its own limit)
        raise ValueError(f"max_new_tokens must be within [0, 2**31), got {T}")
    bt = _need(block_tables, "block_tables", torch.int32, 2)
    dev = block_tables.get_device()
    lens = _need(context_lens, "context_lens", torch.int32, 1, dev)
    new = _need(new_tokens, "new_tokens", torch.int32, 1, dev)
    free = _need(free_blocks, "free_blocks", torch.int32, 1, dev)
    count = _need(free_count, "free_count", torch.int32, 1, dev)
    err = _opt(error_word, "error_word", torch.int32, 1, dev)
    B, mb = block_tables.shape
    if context_lens.shape[0] != B or new_tokens.shape[0] != B:
        raise ValueError("context_lens / new_tokens batch differs from block_tables'")
    if free_count.shape[0] != 1:
        raise ValueError("free_count must be [1]")
    lens_out, lp = _give(context_lens_out, "context_lens_out", (B,), torch.int32, block_tables, dev, stream)
    count_out, cp = _give(free_count_out, "free_count_out", (1,), torch.int32, block_tables, dev, stream)
    starts, qp = _give(query_starts, "query_starts", (B + 1,), torch.int32, block_tables, dev, stream)
    slots, sp = _give(slot_mapping, "slot_mapping", (T,), torch.int64, block_tables, dev, stream)
    pos, pp = _give(positions, "positions", (T,), torch.int32, block_tables, dev, stream)
    _call("pkv_kv_step_tables", dev, stream, bt, lp, qp, sp, pp, cp, free, count, lens, new, T,
          _dims(B, 1, 1, 128, free_blocks.shape[0], mb), err)
    return lens_out, starts, slots, pos, count_out


def _f8_pools(k_codes, v_codes, k_scales, v_scales):
    kp = _need(k_codes, "k_codes", torch.float8_e4m3fn, 4)
    dev = k_codes.get_device()
    vp = _need(v_codes, "v_codes", torch.float8_e4m3fn, 4, dev)
    ksp = _need(k_scales, "k_scales", torch.float32, 2, dev)
    vsp = _need(v_scales, "v_scales", torch.float32, 2, dev)
    shape = k_codes.shape
    nb, hkv, bs, d = shape
    if v_codes.shape != shape:
        raise ValueError("k_codes and v_codes shapes differ")
    if bs != BLOCK_SIZE:
        raise ValueError(f"pool block size must be {BLOCK_SIZE}")
    if k_scales.shape != (nb, hkv) or v_scales.shape != (nb, hkv):
        raise ValueError("scale pools must be [num_blocks, num_kv_heads]")
    return nb, hkv, d, dev, kp, vp, ksp, vsp


def _bf16_pools(k_cache, v_cache):
    kp = _need(k_cache, "k_cache", torch.bfloat16, 4)
    dev = k_cache.get_device()
    vp = _need(v_cache, "v_cache", torch.bfloat16, 4, dev)
    nb, hkv, bs, d = k_cache.shape
    if v_cache.shape != k_cache.shape or bs != BLOCK_SIZE:
        raise ValueError(f"pools must have one shape [num_blocks, num_kv_heads, {BLOCK_SIZE}, head_dim]")
    return nb, hkv, d, dev, kp, vp


def kv_append_f8(k_codes, v_codes, k_scales, v_scales, k, v, slot_mapping, *, error_word=None, stream=None):
    """Write k, v [T, Hkv, d] (bf16) into FP8 pools at slot_mapping [T] (int64; < 0 skips): codes
    [NB, Hkv, 16, d] torch.float8_e4m3fn, one power-of-two fp32 scale per (block, kv head), [NB, Hkv].
    A block written at offset 0 starts anew; otherwise its scale only grows and its other rows move to
    it.  The tokens of one block are adjacent in slot_mapping, slots ascending (the order of
    kv_step_tables)."""
    nb, hkv, d, dev, kc, vc, ks, vs = _f8_pools(k_codes, v_codes, k_scales, v_scales)
    kp = _need(k, "k", torch.bfloat16, 3, dev)
    vp = _need(v, "v", torch.bfloat16, 3, dev)
    sp = _need(slot_mapping, "slot_mapping", torch.int64, 1, dev)
    err = _opt(error_word, "error_word", torch.int32, 1, dev)
    T = slot_mapping.shape[0]
    if k.shape != (T, hkv, d) or v.shape != (T, hkv, d):
        raise ValueError("k/v must be [num_tokens, num_kv_heads, head_dim]")
    _call("pkv_kv_append_f8", dev, stream, kc, vc, ks, vs, kp, vp, sp, T, _dims(0, 0, hkv, d, nb, 0), err)


def _rules(softcap, window, alibi_slopes, doc_starts, prefix_lens, hq, rows, batch, dev):
    softcap = float(softcap)
    if softcap != 0.0 and not 1e-30 <= softcap <= 1e30:
        raise ValueError("softcap must be 0 (none) or within [1e-30, 1e30]")
    a = _opt(alibi_slopes, "alibi_slopes", torch.float32, 1, dev)
    ds = _opt(doc_starts, "doc_starts", torch.int32, 1, dev)
    p = _opt(prefix_lens, "prefix_lens", torch.int32, 1, dev)
    if a is not None and alibi_slopes.shape[0] != hq:
        raise ValueError("alibi_slopes must be [num_q_heads]")
    if ds is not None and doc_starts.shape[0] != rows:
        raise ValueError("doc_starts must have one entry per query row")
    if p is not None and prefix_lens.shape[0] != batch:
        raise ValueError("prefix_lens must be [batch]")
    return PkvScoreRules(softcap, max(0, min(int(window), 2**31 - 1)), a, ds, p)


def _decode_common(q, nb, hkv, d, block_tables, context_lens, out, workspace, error_word, dev, stream):
    qp = _need(q, "q", torch.bfloat16, 3, dev)
    bp = _need(block_tables, "block_tables", torch.int32, 2, dev)
    lp = _need(context_lens, "context_lens", torch.int32, 1, dev)
    err = _opt(error_word, "error_word", torch.int32, 1, dev)
    B, hq, dq = q.shape
    rows, mb = block_tables.shape
    if dq != d:
        raise ValueError("q head_dim differs from the pools'")
    if rows != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens batch differs from q's")
    dims = _dims(B, hq, hkv, d, nb, mb)
    out, op = _give(out, "out", (B, hq, d), torch.bfloat16, q, dev, stream)
    if workspace is None:
        workspace = _new((int(load().pkv_decode_workspace_bytes(dims)),), torch.uint8, q, stream, torch.zeros)
    wp = _need(workspace, "workspace", torch.uint8, 1, dev)
    return B, hq, dims, qp, bp, lp, err, out, op, wp, workspace.numel()


def paged_decode_attention_rules(q, k_cache, v_cache, block_tables, context_lens, scale, window=0, *, softcap=0.0,
                                 alibi_slopes=None, doc_starts=None, prefix_lens=None, out=None, workspace=None,
                                 error_word=None, inputs_ready=False, stream=None):
    """paged_decode_attention with score rules: scores capped to softcap * tanh(x / softcap), a distance
    bias -alibi_slopes[h] * (L - 1 - t) (fp32 [Hq]), and the visible keys [max(0, L - window, doc_start), L)
    and [0, prefix_len) (int32 [B] each).  Returns out [B, Hq, d] bf16; a row that sees no key is zero."""
    nb, hkv, d, dev, kp, vp = _bf16_pools(k_cache, v_cache)
    B, hq, dims, qp, bp, lp, err, out, op, wp, ws_bytes = _decode_common(q, nb, hkv, d, block_tables, context_lens, out,
                                                                         workspace, error_word, dev, stream)
    rules = _rules(softcap, window, alibi_slopes, doc_starts, prefix_lens, hq, B, B, dev)
    _call("pkv_paged_decode_attention_rules", dev, stream, op, qp, kp, vp, bp, lp, scale, ctypes.byref(rules), wp, ws_bytes,
          dims, _INPUTS_READY if inputs_ready else 0, err)
    return out


def paged_decode_attention_f8(q, k_codes, v_codes, k_scales, v_scales, block_tables, context_lens, scale, window=0, *,
                              softcap=0.0, alibi_slopes=None, doc_starts=None, prefix_lens=None, out=None,
                              workspace=None, error_word=None, inputs_ready=False, stream=None):
    """paged_decode_attention over FP8 pools (codes [NB, Hkv, 16, d] torch.float8_e4m3fn times one fp32
    scale per (block, kv head), [NB, Hkv]), with the score rules of paged_decode_attention_rules."""
    nb, hkv, d, dev, kp, vp, ks, vs = _f8_pools(k_codes, v_codes, k_scales, v_scales)
    B, hq, dims, qp, bp, lp, err, out, op, wp, ws_bytes = _decode_common(q, nb, hkv, d, block_tables, context_lens, out,
                                                                         workspace, error_word, dev, stream)
    rules = None
    if softcap != 0 or window > 0 or alibi_slopes is not None or doc_starts is not None or prefix_lens is not None:
        rules = ctypes.byref(_rules(softcap, window, alibi_slopes, doc_starts, prefix_lens, hq, B, B, dev))
    _call("pkv_paged_decode_attention_f8", dev, stream, op, qp, kp, vp, ks, vs, bp, lp, scale, rules, wp, ws_bytes, dims,
          _INPUTS_READY if inputs_ready else 0, err)
    return out


def prefill_workspace_bytes(total_tokens, batch, num_q_heads, num_kv_heads, head_dim, num_blocks, max_blocks_per_seq) -> int:
    """Workspace of paged_prefill_attention for these sizes and at most total_tokens query rows."""
    dims = _sizes(batch, num_q_heads, num_kv_heads, head_dim, num_blocks, max_blocks_per_seq)
    T = int(total_tokens)
    n = int(load().pkv_prefill_workspace_bytes(dims, T)) if 0 <= T < 2**31 else 0
    if n == 0:
        raise ValueError("invalid dims for paged prefill")
    return n


def paged_prefill_attention(q, k_cache, v_cache, block_tables, context_lens, query_starts, scale, window=0, *, softcap=0.0,
                            alibi_slopes=None, doc_starts=None, prefix_lens=None, out=None, workspace=None,
                            error_word=None, stream=None):
    """Causal attention of many query tokens per sequence over the paged cache, with score rules.
    q [T, Hq, d] bf16 packs the queries of every sequence: rows query_starts[b] .. query_starts[b+1]
    (int32 [B + 1]) are sequence b's last positions, context_lens [B] counts its keys with the step's own.
    The pools are bf16 (there is no form over the FP8 cache).  The rules are those of
    paged_decode_attention_rules, doc_starts one int32 per packed row [T].  Returns
    out [T, Hq, d]; rows from query_starts[B] on are left as they were (unset when `out` is made here)."""
    nb, hkv, d, dev, kp, vp = _bf16_pools(k_cache, v_cache)
    qp = _need(q, "q", torch.bfloat16, 3, dev)
    bp = _need(block_tables, "block_tables", torch.int32, 2, dev)
    lp = _need(context_lens, "context_lens", torch.int32, 1, dev)
    sp = _need(query_starts, "query_starts", torch.int32, 1, dev)
    err = _opt(error_word, "error_word", torch.int32, 1, dev)
    T, hq, dq = q.shape
    B, mb = block_tables.shape
    if dq != d:
        raise ValueError("q head_dim differs from the pools'")
    if context_lens.shape[0] != B or query_starts.shape[0] != B + 1:
        raise ValueError("context_lens must be [B] and query_starts [B + 1]")
    rules = _rules(softcap, window, alibi_slopes, doc_starts, prefix_lens, hq, T, B, dev)
    dims = _dims(B, hq, hkv, d, nb, mb)
    out, op = _give(out, "out", (T, hq, d), torch.bfloat16, q, dev, stream)
    if workspace is None:
        workspace = _new((int(load().pkv_prefill_workspace_bytes(dims, T)),), torch.uint8, q, stream)
    wp = _need(workspace, "workspace", torch.uint8, 1, dev)
    _call("pkv_paged_prefill_attention", dev, stream, op, qp, kp, vp, bp, lp, sp, T, scale, ctypes.byref(rules), wp,
          workspace.numel(), dims, err)
    return out
