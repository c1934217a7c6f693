"""Host-side checks of the drafting calls (nothing reaches the CUDA runtime) and the plain
forms that the GPU tests use."""
import ctypes

import numpy as np
import pytest

from order_retrieval_gb300 import binding as zb

from draft_util import line, reserve_plain, tree
from test_cache_cpu import FAKE, _cache, _prob

CALLS = {"zeta_cache_attend_tree": (16, (15,)), "zeta_cache_accept": (11, (10,)),
         "zeta_cache_reserve": (8, (7,))}         # pointers before the status, optional ones


@pytest.fixture(scope="module")
def L():
    return zb.lib()


def _all(L, p, c):
    P, Q = (ctypes.byref(x) if x is not None else None for x in (p, c))
    return [getattr(L, f)(P, Q, *[FAKE] * n, None, None) for f, (n, _) in CALLS.items()]


@pytest.mark.parametrize("kw", [dict(page=0), dict(page=24), dict(pages=-1), dict(order_pages=-1),
                                dict(n=-1), dict(table_len=15), dict(table_len=-1),
                                dict(pages=0)])
def test_invalid_caches(L, kw):
    assert _all(L, _prob(), _cache(**kw)) == [1, 1, 1]


def test_invalid_problems(L):
    for kw in (dict(N=1000), dict(k=0), dict(k=129), dict(d_K=0), dict(B=-1)):
        assert _all(L, _prob(**kw), _cache()) == [1, 1, 1]
    assert _all(L, None, _cache()) == [1, 1, 1]
    assert _all(L, _prob(), None) == [1, 1, 1]


@pytest.mark.parametrize("pk,ck", [(dict(), dict(n=129)), (dict(), dict(page=1 << 17)),
                                   (dict(N=16384, C=16384), dict(table_len=256)),
                                   (dict(), dict(pages=1 << 30)), (dict(d_V=512), dict()),
                                   (dict(flags=4), dict())])
def test_unsupported_caches(L, pk, ck):
    assert _all(L, _prob(**pk), _cache(**ck)) == [2, 2, 2]


def test_drafts_of_more_nodes_than_there_may_be(L):
    p, c = _prob(N=4096, C=2048), _cache(n=1025, table_len=64)
    assert _all(L, p, _cache(n=1025, table_len=64))[:2] == [2, 2]
    P, Q = ctypes.byref(p), ctypes.byref(c)
    assert L.zeta_cache_reserve(P, Q, *[None] * 10) == 1      # n bounds no tree there


def test_the_tree_wants_order_pools(L):
    P, Q = ctypes.byref(_prob()), ctypes.byref(_cache(order_pages=0))
    assert L.zeta_cache_attend_tree(P, Q, *[FAKE] * 16, None, None) == 1


def test_null_and_unaligned_pointers(L):
    P, Q = ctypes.byref(_prob()), ctypes.byref(_cache())
    for f, (n, optional) in CALLS.items():
        for pos in range(n):
            a = [FAKE] * n
            a[pos] = None
            if pos not in optional:
                assert getattr(L, f)(P, Q, *a, None, None) == 1, (f, pos)
    odd = ctypes.c_void_p(0x1008)
    for f, places in (("zeta_cache_attend_tree", (2, 9, 13)), ("zeta_cache_accept", (1, 8))):
        for pos in places:                           # v, v_pages, out
            a = [FAKE] * CALLS[f][0]
            a[pos] = odd
            assert getattr(L, f)(P, Q, *a, None, None) == 1, (f, pos)


@pytest.mark.parametrize("f,out,inputs", [("zeta_cache_attend_tree", 13, (2,)),
                                           ("zeta_cache_accept", 9, (2, 3, 5)),
                                           ("zeta_cache_accept", 10, (4,)),
                                           ("zeta_cache_reserve", 6, (0, 3)),
                                           ("zeta_cache_reserve", 3, (0, 1))])
def test_outputs_in_the_place_of_inputs(L, f, out, inputs):
    """What other blocks still read must not be written: refused before a launch."""
    P, Q = ctypes.byref(_prob()), ctypes.byref(_cache())
    for pos in inputs:
        a = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(CALLS[f][0])]
        a[out] = a[pos]
        assert getattr(L, f)(P, Q, *a, None, None) == 1, (f, out, pos)


def test_empty_calls_are_no_ops(L):
    for p, c in ((_prob(B=0), _cache()), (_prob(H=0), _cache()), (_prob(), _cache(n=0))):
        P, Q = ctypes.byref(p), ctypes.byref(c)
        for f, (n, _) in CALLS.items():
            assert getattr(L, f)(P, Q, *[None] * (n + 2)) == 0
    # the binding's marshalling matches the C signatures
    p, c = _prob(B=0), _cache()
    zb.zeta_cache_attend_tree(p, c, *[None] * 15, stream=0)
    zb.zeta_cache_accept(p, c, *[None] * 10, stream=0)
    zb.zeta_cache_reserve(p, c, *[None] * 7, stream=0)


def test_trees_of_the_tests():
    rng = np.random.default_rng(0)
    for kind in ("tree", "bushy", "chain", "star"):
        for n in (0, 1, 2, 5, 40):
            p = tree(rng, n, kind)
            assert len(p) == n and all(-1 <= p[t] < t for t in range(n))
            for t in range(n):
                x = line(p, t)
                assert x[-1] == t and p[x[0]] == -1 and all(p[b] == a for a, b in zip(x, x[1:]))
    assert line(tree(rng, 5, "chain"), 4) == [0, 1, 2, 3, 4]


def test_plain_reserve_keeps_the_pages():
    """Over many steps no page is lost or given twice, a step that is taken back restores the
    list, and who is granted holds what it needs."""
    rng = np.random.default_rng(1)
    B, page, pages, N, n = 7, 4, 60, 80, 20
    table, held = np.full((B, N // page), -1), np.zeros(B, np.int64)
    free, F = rng.permutation(pages), pages
    length = np.zeros(B, np.int64)
    refused = 0
    for _ in range(60):
        length[rng.random(B) < 0.2] = 0
        count = np.minimum(rng.integers(0, n + 1, B), N - length)
        before = (table.copy(), held.copy(), free[:F].copy())
        had = held.copy()
        granted, slots, F = reserve_plain(table, held, free, F, length, count, n, page, pages, N)
        out = np.concatenate([free[:F]] + [table[b, :held[b]] for b in range(B)])
        assert sorted(out.tolist()) == list(range(pages))
        refused += int((granted < count).sum())
        for b in range(B):
            assert (table[b, held[b]:] == -1).all()
            if granted[b] == count[b] and count[b]:
                assert held[b] == -(-(length[b] + count[b]) // page)
                i = length[b] + np.arange(count[b])
                assert np.array_equal(slots[b, :count[b]], table[b, i // page] * page + i % page)
        _, _, F = reserve_plain(table, held, free, F, had * page, 0 * count, n, page, pages, N)
        assert np.array_equal(table, before[0]) and np.array_equal(held, before[1])
        assert np.array_equal(free[:F], before[2])
        granted, _, F = reserve_plain(table, held, free, F, length, count, n, page, pages, N)
        length += granted
    assert refused > 5
