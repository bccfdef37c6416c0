"""Sizes past 32 bits given to the serving-step binding: refused, not cut to the low word.  (No GPU needed: sizes are
looked at before the tensors.)"""
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
from paged_kv_cache_mapped_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


def test_prefill_workspace_of_sizes_past_32_bits():
    ok = (64, 4, 32, 8, 128, 1000, 64)
    assert pkv.prefill_workspace_bytes(*ok) > 0
    for at in range(len(ok)):
        for x in (2**32 + ok[at], 2**31, -1, -(2**32) + ok[at]):
            with pytest.raises(ValueError):
                pkv.prefill_workspace_bytes(*ok[:at], x, *ok[at + 1:])


@pytest.mark.parametrize("n", [2**31, 2**32, 2**32 + 4, -1, -(2**32) + 4])
def test_step_tables_of_token_counts_past_32_bits(n):
    t = torch.zeros((2, 3), dtype=torch.int32)
    with pytest.raises(ValueError, match="max_new_tokens"):
        pkv.kv_step_tables(t, t[:, 0], t[:, 0], t[0], t[0, :1], n)
