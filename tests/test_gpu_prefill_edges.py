"""The prefill attention where there is nothing to do, and where its result is worked out twice."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
import test_gpu_prefill_attention as prefill
from paged_kv_cache_mapped_gb300 import header_constants
from test_gpu_guard_bands import Guarded, _check

C = header_constants()
DEV = torch.device("cuda:0")


@pytest.mark.gpu
@pytest.mark.parametrize("B,hkv", [(1, 1), (3, 8), (600, 2), (4096, 1)])
@pytest.mark.parametrize("what", ["idle", "idle and empty", "refused"])
def test_steps_without_an_entry(what, B, hkv):
    """No sequence has a row to compute: the output stays as it was, and a call with rows on the same workspace
    is as ever (the plan of the empty one has no items and no splits)."""
    c = prefill._case([40, 17, 16] * (B // 3) + [33] * (B % 3), [0] * B, 2 * hkv, hkv, 64, 60, pad=50)
    c["bt"][:, :] = c["bt"][:, :].clamp(min=0)
    want_err = 0
    if what == "idle and empty":
        c["lens"] = [0] * B
    if what == "refused":  # more rows than keys, for the last, and the others behind its start
        c["starts"] = np.array([0] * B + [50], dtype=np.int32)
        c["lens"][-1] = 20
        want_err = C["PKV_DEV_BAD_CONTEXT_LEN"]
    err = pkv.new_error_word(DEV)
    out = Guarded((50, 2 * hkv, 64), torch.bfloat16)
    ws = Guarded((pkv.prefill_workspace_bytes(50, B, 2 * hkv, hkv, 64, c["pools"][0].shape[0], c["bt"].shape[1]),), torch.uint8)
    for r in ({}, dict(softcap=5.0, window=9)):
        out.t.fill_(3.0)
        prefill._call(c, out=out.t, workspace=ws.t, error_word=err, **r)
        assert pkv.read_error(err, clear=True) == want_err
        assert bool((out.t == 3.0).all())
        _check(("out", out), ("workspace", ws))
    rows = dict(c, starts=np.array([0] + [min(9, c["lens"][0] or 9)] * B, dtype=np.int32), lens=[40] + [17] * (B - 1))
    want = prefill._call(rows)[:9]
    out.t.fill_(3.0)
    prefill._call(rows, out=out.t, workspace=ws.t, error_word=err)
    assert pkv.read_error(err) == 0
    # bit for bit: a length past the sequence's own reads the pools' NaN fill
    assert torch.equal(out.t[:9].view(torch.int16), want.view(torch.int16)) and bool((out.t[9:] == 3.0).all())
