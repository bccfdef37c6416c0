"""ctypes handle on libpkv.so: loads the in-tree library and declares the C signatures of
include/pkv.h, pkv_step.h, pkv_evict.h and pkv_diff.h.  No arithmetic happens here."""
from __future__ import annotations

import ctypes
import os
import re
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libpkv.so")
HEADER = os.path.join(os.path.dirname(PKG), "include", "pkv.h")
STEP_HEADER = os.path.join(os.path.dirname(PKG), "include", "pkv_step.h")
EVICT_HEADER = os.path.join(os.path.dirname(PKG), "include", "pkv_evict.h")
DIFF_HEADER = os.path.join(os.path.dirname(PKG), "include", "pkv_diff.h")

_lock = threading.Lock()
_lib = None


class PkvDims(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
    ]


class PkvScoreRules(ctypes.Structure):
    _fields_ = [
        ("softcap", ctypes.c_float),
        ("window", ctypes.c_int32),
        ("alibi_slopes", ctypes.c_void_p),
        ("doc_starts", ctypes.c_void_p),
        ("prefix_lens", ctypes.c_void_p),
    ]


class PkvDiffParams(ctypes.Structure):
    _fields_ = [
        ("lambdas", ctypes.c_void_p),
        ("lambda_rows", ctypes.c_int32),
        ("norm_eps", ctypes.c_float),
        ("norm_weight", ctypes.c_void_p),
    ]


class PkvEvictRules(ctypes.Structure):
    _fields_ = [
        ("n_sink", ctypes.c_int32),
        ("k_top", ctypes.c_int32),
        ("n_recent", ctypes.c_int32),
        ("trigger", ctypes.c_int32),
    ]


class PkvEvictState(ctypes.Structure):
    _fields_ = [
        ("scores", ctypes.c_void_p),
        ("scores_out", ctypes.c_void_p),
        ("slot_pos", ctypes.c_void_p),
        ("slot_pos_out", ctypes.c_void_p),
        ("dropped", ctypes.c_void_p),
        ("dropped_out", ctypes.c_void_p),
        ("stride", ctypes.c_int32),
    ]


class PkvError(RuntimeError):
    """A call into libpkv returned a non-zero status."""

    def __init__(self, func: str, status: int, text: str):
        super().__init__(f"{func}: status {status}: {text}")
        self.status = status


def header_constants() -> dict:
    """#define NAME value pairs of the public headers (status and device-error codes, flags, limits)."""
    out = {}
    for path in (HEADER, STEP_HEADER, EVICT_HEADER):
        with open(path) as f:
            for m in re.finditer(r"^#define\s+(PKV_\w+)\s+([-+*() 0-9]+?)\s*(?:/\*.*)?$", f.read(), re.M):
                out[m.group(1)] = int(eval(m.group(2), {"__builtins__": {}}, {}))  # integer literal arithmetic only
    return out


def header_functions(path: str = HEADER) -> list:
    """Names of the functions include/pkv.h (or the header at `path`) declares."""
    with open(path) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\*?\s+\*?(pkv_\w+)\s*\(", text, re.M)))


def load():
    """Load libpkv.so; raises if it was not built (there is no fallback path)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`"
                " (the CUDA library is required; there is no CPU fallback)")
        lib = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
        U32 = ctypes.c_uint32
        D = ctypes.POINTER(PkvDims)
        R = ctypes.POINTER(PkvScoreRules)
        DP = ctypes.POINTER(PkvDiffParams)
        ER, ES = ctypes.POINTER(PkvEvictRules), ctypes.POINTER(PkvEvictState)
        sig = {
            "pkv_kv_append": (I32, [P, P, P, P, P, I64, D, P, P]),
            "pkv_kv_append_q8": (I32, [P, P, P, P, P, P, P, I64, D, P, P]),
            "pkv_prefill_window_scores": (I32, [P, I32, P, I32, P, P, P, P, I32, F32, D, P, P]),
            "pkv_decode_workspace_bytes": (SZ, [D]),
            "pkv_paged_decode_attention_q8": (I32, [P, P, P, P, P, P, P, P, F32, I32, P, SZ, D, U32, P, P]),
            "pkv_paged_decode_attention": (I32, [P, P, P, P, P, P, F32, I32, P, SZ, D, U32, P, P]),
            "pkv_paged_decode_attention_append": (I32, [P, P, P, P, P, P, P, P, F32, I32, P, SZ, D, U32, P, P]),
            "pkv_paged_decode_attention_scores": (I32, [P, P, P, P, I32, P, P, P, P, P, P, P, F32, I32, P, SZ,
                                                        D, U32, P, P]),
            "pkv_kv_rolling_admit": (I32, [P, P, P, P, P, P, P, P, P, I32, I32, I32, D, U32, P, P]),
            "pkv_paged_decode_attention_scores_q8": (I32, [P, P, P, P, I32, P, P, P, P, P, P, P, F32, I32, P,
                                                           SZ, D, U32, P, P]),
            "pkv_paged_decode_attention_append_q8": (I32, [P, P, P, P, P, P, P, P, P, P, F32, I32, P, SZ, D, U32,
                                                           P, P]),
            "pkv_sparse_decode_attention_q8": (I32, [P, P, P, P, P, P, P, P, P, P, I32, F32, P, SZ, D, U32, P, P]),
            "pkv_kv_compact_q8": (I32, [P, P, P, P, P, I32, I32, P, P, P, P, P, P, P, P, I32, D, U32, P, P]),
            "pkv_kv_rolling_admit_q8": (I32, [P, P, P, P, P, P, P, P, P, P, P, I32, I32, I32, D, U32, P, P]),
            "pkv_sparse_decode_workspace_bytes": (SZ, [D, I32]),
            "pkv_sparse_decode_attention": (I32, [P, P, P, P, P, P, P, P, I32, F32, P, SZ, D, U32, P, P]),
            "pkv_kv_select_topk": (I32, [P, P, P, I32, P, I32, I32, I32, D, U32, P, P]),
            "pkv_kv_compact": (I32, [P, P, P, I32, I32, P, P, P, P, P, P, I32, D, U32, P, P]),
            "pkv_paged_decode_attention_fixed_scratch": (I32, [P, P, P, P, P, P, F32, I32, D, P, P]),
            "pkv_kv_step_tables": (I32, [P, P, P, P, P, P, P, P, P, P, I32, D, P, P]),
            "pkv_paged_decode_attention_rules": (I32, [P, P, P, P, P, P, F32, R, P, SZ, D, U32, P, P]),
            "pkv_paged_decode_attention_f8": (I32, [P, P, P, P, P, P, P, P, F32, R, P, SZ, D, U32, P, P]),
            "pkv_prefill_workspace_bytes": (SZ, [D, I32]),
            "pkv_paged_prefill_attention": (I32, [P, P, P, P, P, P, P, I32, F32, R, P, SZ, D, P, P]),
            "pkv_kv_append_f8": (I32, [P, P, P, P, P, P, P, I64, D, P, P]),
            "pkv_diff_decode_workspace_bytes": (SZ, [D, I32]),
            "pkv_paged_diff_decode_attention": (I32, [P, P, P, P, P, P, F32, DP, R, P, SZ, D, U32, P, P]),
            "pkv_paged_diff_decode_attention_scores": (I32, [P, P, P, I32, P, P, P, P, P, F32, DP, R, P, SZ, D, U32, P,
                                                             P]),
            "pkv_diff_prefill_workspace_bytes": (SZ, [D, I32]),
            "pkv_paged_diff_prefill_attention": (I32, [P, P, P, P, P, P, P, I32, F32, DP, R, P, SZ, D, P, P]),
            "pkv_evict_workspace_bytes": (SZ, [D, ER]),
            "pkv_kv_evict": (I32, [P, P, P, P, P, ES, ER, P, P, P, P, SZ, D, P, P]),
            "pkv_kv_evict_q8": (I32, [P, P, P, P, P, P, P, ES, ER, P, P, P, P, SZ, D, P, P]),
            "pkv_read_error": (I32, [P, I32, P]),
            "pkv_device_alias": (I32, [P, ctypes.POINTER(ctypes.c_void_p)]),
            "pkv_status_string": (ctypes.c_char_p, [I32]),
            "pkv_device_error_string": (ctypes.c_char_p, [I32]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def check(func: str, status: int) -> None:
    if status != 0:
        text = load().pkv_status_string(status).decode()
        raise PkvError(func, status, text)
