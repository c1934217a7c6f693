"""Host-side checks of the drafting calls' further forms (nothing reaches the CUDA runtime)."""
import ctypes

import pytest

from order_retrieval_gb300 import binding as zb

from test_cache_cpu import FAKE, _cache, _prob

GRANTED = 12                                          # pointers of accept_granted before the status


@pytest.fixture(scope="module")
def L():
    return zb.lib()


def test_accept_granted_checks_as_accept_does(L):
    P, Q = ctypes.byref(_prob()), ctypes.byref(_cache())
    call = L.zeta_cache_accept_granted
    for pos in range(GRANTED - 1):                   # all but path; granted among them
        a = [FAKE] * GRANTED
        a[pos] = None
        assert call(P, Q, *a, None, None) == 1, pos
    for pos in (1, 9):                               # v, v_pages
        a = [FAKE] * GRANTED
        a[pos] = ctypes.c_void_p(0x1008)
        assert call(P, Q, *a, None, None) == 1, pos
    a = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(GRANTED)]
    for out in (10, 11):                             # accepted, path in the place of granted
        b = list(a)
        b[out] = b[6]
        assert call(P, Q, *b, None, None) == 1, out
    for kw in (dict(N=1000), dict(d_K=0)):
        assert call(ctypes.byref(_prob(**kw)), Q, *[FAKE] * GRANTED, None, None) == 1
    big = _prob(N=4096, C=2048), _cache(n=1025, table_len=64)
    assert call(*map(ctypes.byref, big), *[FAKE] * GRANTED, None, None) == 2
    for p, c in ((_prob(B=0), _cache()), (_prob(H=0), _cache()), (_prob(), _cache(n=0))):
        assert call(ctypes.byref(p), ctypes.byref(c), *[None] * (GRANTED + 2)) == 0
    zb.zeta_cache_accept_granted(_prob(B=0), _cache(), *[None] * 11, stream=0)


def test_reserve_without_rows_wants_its_arrays(L):
    """It has pages to give back; without any array it is the empty call."""
    for p, c in ((_prob(), _cache(n=0)), (_prob(H=0), _cache())):
        P, Q = ctypes.byref(p), ctypes.byref(c)
        assert L.zeta_cache_reserve(P, Q, *[None] * 10) == 0
        for pos in range(7):
            a = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(7)] + [None] * 3
            a[pos] = None
            assert L.zeta_cache_reserve(P, Q, *a) == 1, pos
