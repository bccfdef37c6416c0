"""Binding of differential attention over the paged cache (declared in include/pkv_diff.h): a head's output is
the difference of two softmax maps with a learned factor.  As the rest of the package: argument checks and
marshalling only."""
from __future__ import annotations

import ctypes

import torch

from ._lib import PkvDiffParams, header_constants, load
from .step import _bf16_pools, _call, _dims, _give, _like, _need, _new, _opt, _rules, _sizes

_INPUTS_READY = header_constants()["PKV_DECODE_INPUTS_READY"]


def _params(lambdas, norm_weight, norm_eps, rows, hq, d, dev):
    per_row = getattr(lambdas, "ndim", 0) == 2
    lp = _need(lambdas, "lambdas", torch.float32, 2 if per_row else 1, dev)
    if lambdas.shape != ((rows, hq) if per_row else (hq,)):
        raise ValueError(f"lambdas must be [num_q_heads] or [rows of q, num_q_heads], got {tuple(lambdas.shape)}")
    wp = None
    if norm_weight is not None:
        wp = _need(norm_weight, "norm_weight", torch.float32, 1, dev)
        if norm_weight.shape[0] != d:
            raise ValueError("norm_weight must be [head_dim]")
        if not 1e-45 <= norm_eps < 3.4e38:  # (finite and positive in fp32)
            raise ValueError("norm_eps must be finite and positive")
    return PkvDiffParams(lp, 1 if per_row else 0, norm_eps, wp)


def diff_decode_workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, num_blocks, max_blocks_per_seq, *, score_stride=0) -> int:
    """Workspace of paged_diff_decode_attention, or with the scores' row length of paged_diff_decode_attention_scores.
    Zero-filled before its first use."""
    dims = _sizes(batch, num_q_heads, num_kv_heads, head_dim, num_blocks, max_blocks_per_seq)
    stride = int(score_stride)
    n = int(load().pkv_diff_decode_workspace_bytes(dims, stride)) if 0 <= stride < 2**31 else 0
    if n == 0:
        raise ValueError("invalid sizes for a differential decode")
    return n


def _decode(name, lead, stride, q, k_cache, v_cache, block_tables, context_lens, lambdas, scale, window, norm_weight, norm_eps,
            softcap, alibi_slopes, doc_starts, prefix_lens, out, workspace, error_word, inputs_ready, stream):
    nb, hkv, d, dev, kp, vp = _bf16_pools(k_cache, v_cache)
    qp = _need(q, "q", torch.bfloat16, 3, dev)
    bp = _need(block_tables, "block_tables", torch.int32, 2, dev)
    lp = _need(context_lens, "context_lens", torch.int32, 1, dev)
    err = None if error_word is None else _need(error_word, "error_word", torch.int32, 1, dev)
    B, hq, dq = q.shape
    rows, mb = block_tables.shape
    if dq != d:
        raise ValueError("q head_dim differs from the pools'")
    if rows != B or context_lens.shape[0] != B:
        raise ValueError("block_tables / context_lens batch differs from q's")
    params = _params(lambdas, norm_weight, norm_eps, B, hq, d, dev)
    rules = None
    if softcap != 0 or window > 0 or alibi_slopes is not None or doc_starts is not None or prefix_lens is not None:
        rules = ctypes.byref(_rules(softcap, window, alibi_slopes, doc_starts, prefix_lens, hq, B, B, dev))
    dims = _dims(B, hq, hkv, d, nb, mb)
    out, op = _like(out, "out", q, dev, stream)
    if workspace is None:
        workspace = _new((int(load().pkv_diff_decode_workspace_bytes(dims, stride)),), torch.uint8, q, stream, torch.zeros)
    wp = _need(workspace, "workspace", torch.uint8, 1, dev)
    _call(name, dev, stream, op, *lead, qp, kp, vp, bp, lp, scale, ctypes.byref(params), rules, wp, workspace.numel(), dims,
          _INPUTS_READY if inputs_ready else 0, err)
    return out


def paged_diff_decode_attention(q, k_cache, v_cache, block_tables, context_lens, lambdas, scale, window=0, *, norm_weight=None,
                                norm_eps=1e-5, softcap=0.0, alibi_slopes=None, doc_starts=None, prefix_lens=None, out=None,
                                workspace=None, error_word=None, inputs_ready=False, stream=None):
    """Differential attention of one token per sequence: q [B, Hq, d] and the K rows hold the two maps' queries and
    keys in their halves, out = sum_t (a_1,t - lambda a_2,t) V_t with a_m = softmax(scale q_m . k_m,t), lambdas
    fp32 [Hq] or [B, Hq]; with norm_weight (fp32 [d]) followed by a root-mean-square norm of each head.  The score
    rules are those of paged_decode_attention_rules.  Returns out [B, Hq, d] bf16; a row that sees no key is zero."""
    return _decode("pkv_paged_diff_decode_attention", (), 0, q, k_cache, v_cache, block_tables, context_lens, lambdas, scale, window,
                   norm_weight, norm_eps, softcap, alibi_slopes, doc_starts, prefix_lens, out, workspace, error_word, inputs_ready,
                   stream)


def paged_diff_decode_attention_scores(q, k_cache, v_cache, block_tables, context_lens, lambdas, scores, scale, window=0, *,
                                       scores_out=None, norm_weight=None, norm_eps=1e-5, softcap=0.0, alibi_slopes=None,
                                       doc_starts=None, prefix_lens=None, out=None, workspace=None, error_word=None,
                                       inputs_ready=False, stream=None):
    """paged_diff_decode_attention that also adds each seen key's |a_1 - lambda a_2|, summed over the query heads of
    its kv head, into scores [B, Hkv, S] fp32 (into scores_out with the other keys' values, where that is given): what
    kv_evict and kv_select_topk go by.  Returns out."""
    dev = scores.get_device() if isinstance(scores, torch.Tensor) else -1
    sp = _need(scores, "scores", torch.float32, 3, k_cache.get_device() if isinstance(k_cache, torch.Tensor) else -1)
    if isinstance(q, torch.Tensor) and isinstance(k_cache, torch.Tensor) and tuple(scores.shape[:2]) != (q.shape[0], k_cache.shape[1]):
        raise ValueError("scores must be [batch, num_kv_heads, slots]")
    stride = scores.shape[2]
    if stride >= 2**31:
        raise ValueError(f"sizes must be within [0, 2**31), got {stride}")
    sop = sp if scores_out is None else _give(scores_out, "scores_out", scores.shape, torch.float32, scores, dev, stream)[1]
    return _decode("pkv_paged_diff_decode_attention_scores", (sp, sop, stride), stride, q, k_cache, v_cache, block_tables,
                   context_lens, lambdas, scale, window, norm_weight, norm_eps, softcap, alibi_slopes, doc_starts, prefix_lens, out,
                   workspace, error_word, inputs_ready, stream)


def diff_prefill_workspace_bytes(total_tokens, batch, num_q_heads, num_kv_heads, head_dim, num_blocks, max_blocks_per_seq) -> int:
    """Workspace of paged_diff_prefill_attention for these sizes and at most total_tokens query rows."""
    dims = _sizes(batch, num_q_heads, num_kv_heads, head_dim, num_blocks, max_blocks_per_seq)
    T = int(total_tokens)
    n = int(load().pkv_diff_prefill_workspace_bytes(dims, T)) if 0 <= T < 2**31 else 0
    if n == 0:
        raise ValueError("invalid dims for paged prefill")
    return n


def paged_diff_prefill_attention(q, k_cache, v_cache, block_tables, context_lens, query_starts, lambdas, scale, window=0, *,
                                 norm_weight=None, norm_eps=1e-5, softcap=0.0, alibi_slopes=None, doc_starts=None,
                                 prefix_lens=None, out=None, workspace=None, error_word=None, stream=None):
    """Differential attention of many query tokens per sequence, causal, over the paged cache: q [T, Hq, d] packs the
    queries of every sequence as in paged_prefill_attention (query_starts int32 [B + 1]), heads, norm and rules are those of
    paged_diff_decode_attention with lambdas fp32 [Hq] or [T, Hq] and doc_starts one int32 per packed row.  Returns
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
    params = _params(lambdas, norm_weight, norm_eps, T, hq, d, dev)
    rules = _rules(softcap, window, alibi_slopes, doc_starts, prefix_lens, hq, T, B, dev)
    dims = _dims(B, hq, hkv, d, nb, mb)
    out, op = _like(out, "out", q, dev, stream)
    if workspace is None:
        workspace = _new((int(load().pkv_diff_prefill_workspace_bytes(dims, T)),), torch.uint8, q, stream)
    wp = _need(workspace, "workspace", torch.uint8, 1, dev)
    _call("pkv_paged_diff_prefill_attention", dev, stream, op, qp, kp, vp, bp, lp, sp, T, scale, ctypes.byref(params),
          ctypes.byref(rules), wp, workspace.numel(), dims, err)
    return out
