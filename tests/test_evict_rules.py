"""What an eviction keeps, as the binding hands it on: the values that the arguments have at the call."""
import numpy as np
import pytest
import torch

import paged_kv_cache_mapped_gb300 as pkv
from paged_kv_cache_mapped_gb300 import _build, evict


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()


def _values(*args):
    r = evict._rules(*args).contents
    return r.n_sink, r.k_top, r.n_recent, r.trigger


@pytest.mark.parametrize("make", [lambda x: torch.tensor(x), lambda x: np.array(x)], ids=["tensor", "array"])
def test_an_argument_changed_in_place_counts_as_it_is_now(make):
    args = [make(4), make(100), make(10), make(50)]
    for at, x in enumerate((7, 4000, 33, 500)):
        want = list(_values(*(int(a) for a in args)))
        assert list(_values(*args)) == want
        args[at].fill(x) if isinstance(args[at], np.ndarray) else args[at].fill_(x)
        want[at] = x
        assert list(_values(*args)) == want


def test_the_workspace_follows_an_argument_changed_in_place():
    k_top = torch.tensor(100)
    for n in (100, 4000, 100):
        k_top.fill_(n)
        assert pkv.evict_workspace_bytes(3, 2, 4, k_top, 10) == pkv.evict_workspace_bytes(3, 2, 4, n, 10)


def test_the_trigger_is_any_number():
    assert _values(1, 2, 3, -5) == (1, 2, 3, 0) and _values(1, 2, 3, 2**40) == (1, 2, 3, 2**31 - 1)
    assert _values(1, 2, 3, True) == (1, 2, 3, 1) and _values(1, 2, 3) == (1, 2, 3, 0)
