"""The host checks of the paged cache keep away from a GPU: what hands the library made-up
pointers is refused before a launch, or does not run where there is a GPU."""
import ctypes

import pytest
import torch

import conftest
import test_cache_cpu as host
from order_retrieval_gb300 import ZetaCache
from order_retrieval_gb300 import binding as zb


def test_calls_that_read_the_order_refuse_pools_without_pages():
    L = zb.lib()
    P, Q = ctypes.byref(host._prob()), ctypes.byref(host._cache(order_pages=0))
    a = [host.FAKE] * 13
    assert L.zeta_cache_order(P, Q, *a[:7], None, None) == 1
    assert L.zeta_cache_attend(P, Q, *a, None, None) == 1


class _Item:
    def __init__(self, name):
        self.name, self.marks = name, []

    def add_marker(self, mark):
        self.marks.append(mark.name)


def test_a_call_that_would_launch_is_skipped_where_there_is_a_gpu(monkeypatch):
    for gpu, want in ((True, ["skip"]), (False, [])):
        monkeypatch.setattr(torch.cuda, "is_available", lambda: gpu)
        items = [_Item("test_pools_without_pages"), _Item("test_invalid_problems")]
        conftest.pytest_collection_modifyitems(items)
        assert [x.marks for x in items] == [want, []]


def test_no_other_host_check_reaches_the_runtime(monkeypatch):
    """Every status that the refusal tests see is a refusal; 4 would be a launch."""
    real, seen = zb.lib(), []

    class Spy:
        def __getattr__(self, name):
            f = getattr(real, name)

            def call(*args):
                seen.append(f(*args))
                return seen[-1]
            return call

    for kw in (dict(page=0), dict(pages=-1), dict(n=-1), dict(table_len=15)):
        host.test_invalid_caches(Spy(), kw)
    host.test_invalid_problems(Spy())
    host.test_null_and_unaligned_pointers(Spy())
    host.test_empty_calls_are_no_ops(Spy())
    assert seen and 4 not in seen


def test_pools_of_other_dimensions_are_refused():
    k, v = torch.zeros(4, 2, 16, 3), torch.zeros(4, 2, 16, 64)
    for codes in (torch.zeros(8), torch.zeros(2, 4, 2)):
        with pytest.raises(ValueError):
            ZetaCache(k, v, codes, codes, 64, 32, 4)
