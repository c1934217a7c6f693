"""Host-side checks of the drafting calls' further forms (nothing reaches the CUDA runtime)."""
import ctypes

import pytest
import torch

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


# f: the outputs and inputs among the pointers, with elements of 4 bytes for _prob(**ONE), n = 1
ONE = dict(B=3, H=1, d_K=1, d_V=4, k=1, v_dtype="f32")
SPANS = {
    "zeta_cache_attend_tree": ({13: 12, 14: 3, 15: 3},
                               {0: 3, 1: 3, 2: 12, 3: 1, 4: 3, 5: 3, 6: 3, 7: 48, 10: 48}),
    "zeta_cache_accept": ({9: 3, 10: 3}, {0: 3, 1: 12, 2: 3, 3: 3, 4: 3, 5: 3, 6: 48}),
    "zeta_cache_accept_granted": ({10: 3, 11: 3},
                                  {0: 3, 1: 12, 2: 3, 3: 3, 4: 3, 5: 3, 6: 3, 7: 48}),
    "zeta_cache_reserve": ({2: 48, 3: 3, 4: 40, 5: 1, 6: 3, 7: 3}, {0: 3, 1: 3}),
}
POINTERS = {"zeta_cache_attend_tree": 16, "zeta_cache_accept": 11, "zeta_cache_accept_granted": 12,
            "zeta_cache_reserve": 8}


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up pointers: only without a GPU")
@pytest.mark.parametrize("f", SPANS)
def test_outputs_that_meet_other_arrays(L, f):
    """Every output in the place of, across the begin and across the end of every input and every
    other output is refused before a launch.  (granted in count's place is meant to be.)"""
    P, Q = ctypes.byref(_prob(**ONE)), ctypes.byref(_cache(n=1, pages=40))
    outs, ins = SPANS[f]
    at = [0x1000000 * (i + 1) for i in range(POINTERS[f])]

    def code(places):
        return getattr(L, f)(P, Q, *[ctypes.c_void_p(x) for x in places], None, None)

    for o, size in outs.items():
        for i, other in {**ins, **{x: y for x, y in outs.items() if x != o}}.items():
            moves = [0, 4 * (other - 1), -4 * (size - 1)]
            if f == "zeta_cache_attend_tree" and o == 13:            # out on 16 bytes
                moves = [int(m / 16) * 16 for m in moves]
            for m in moves:
                if f == "zeta_cache_reserve" and (o, i, m) == (6, 1, 0):
                    continue
                places = list(at)
                places[o] = at[i] + m
                assert code(places) == 1, (f, o, i, m)
