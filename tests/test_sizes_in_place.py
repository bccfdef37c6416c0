"""The workspace sizes follow the values that their arguments have at the call, a tensor's of one number too."""
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
from paged_kv_cache_mapped_gb300 import _build

CALLS = {
    "prefill": (pkv.prefill_workspace_bytes, (300, 4, 32, 8, 128, 1000, 64), {3: 4, 4: 64}),
    "differential prefill": (pkv.diff_prefill_workspace_bytes, (300, 4, 32, 8, 128, 1000, 64), {3: 4, 4: 64}),
    "differential decode": (pkv.diff_decode_workspace_bytes, (4, 32, 8, 128, 1000, 64), {2: 4, 3: 64}),
    "eviction": (pkv.evict_workspace_bytes, (4, 8, 4, 100, 10), {}),
}


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


@pytest.mark.parametrize("name", CALLS)
def test_an_argument_changed_in_place_counts_as_it_is_now(name):
    fn, sizes, values = CALLS[name]
    for at, x in enumerate(sizes):
        other = values.get(at, 2 * x)
        t = torch.tensor(x)
        args = [*sizes[:at], t, *sizes[at + 1:]]
        assert fn(*args) == fn(*sizes)
        t.fill_(other)
        assert fn(*args) == fn(*sizes[:at], other, *sizes[at + 1:]), at


@pytest.mark.parametrize("name", CALLS)
def test_sizes_that_are_no_whole_numbers_are_refused(name):
    fn, sizes, _ = CALLS[name]
    first = 1 if "prefill" in name else 0   # (the number of tokens is cut to an int)
    with pytest.raises(TypeError):
        fn(*sizes[:first], 2.5, *sizes[first + 1:])
