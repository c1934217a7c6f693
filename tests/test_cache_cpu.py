"""Host-side checks of the paged-cache calls (nothing reaches the CUDA runtime),
and the plain forms that the GPU tests use against the oracle."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from order_retrieval_gb300 import ZetaCache
from order_retrieval_gb300 import binding as zb
from order_retrieval_gb300 import workloads as W

from cache_util import Sequence

FAKE = ctypes.c_void_p(0x1000)            # never dereferenced: the checks fail first


@pytest.fixture(scope="module")
def L():
    return zb.lib()


def _prob(**kw):
    base = dict(B=2, H=2, N=1024, d_K=3, d_V=64, k=16, C=128, bits=10)
    base.update(kw)
    return zb.problem(**base)


def _cache(**kw):
    base = dict(n=4, page=64, pages=100, order_pages=100, table_len=16)
    base.update(kw)
    return zb.zeta_cache_t(**base)


def _all(L, p, c, args=None):
    """Status of the three calls with non-null fakes."""
    P, Q = (ctypes.byref(x) if x is not None else None for x in (p, c))
    a = [FAKE] * 15
    return [L.zeta_cache_append(P, Q, *a[:7], None, None), L.zeta_cache_order(P, Q, *a[:7], None,
                                                                            None),
            L.zeta_cache_attend(P, Q, *a[:13], None, None)]


@pytest.mark.parametrize("kw", [dict(page=0), dict(page=24), dict(page=-16), dict(pages=-1),
                                dict(order_pages=-1), dict(n=-1), dict(table_len=15),
                                dict(table_len=-1)])
def test_invalid_caches(L, kw):
    assert _all(L, _prob(), _cache(**kw)) == [1, 1, 1]


@pytest.mark.parametrize("pk,ck", [(dict(), dict(n=129)), (dict(), dict(page=1 << 17)),
                                   (dict(N=16384, C=16384), dict(table_len=256)),
                                   (dict(), dict(pages=1 << 30)),
                                   (dict(), dict(order_pages=1 << 30)),
                                   (dict(d_V=512), dict()), (dict(flags=4), dict())])
def test_unsupported_caches(L, pk, ck):
    assert _all(L, _prob(**pk), _cache(**ck)) == [2, 2, 2]


def test_pools_without_pages(L):
    assert _all(L, _prob(), _cache(pages=0)) == [1, 1, 1]
    assert _all(L, _prob(), _cache(order_pages=0))[1:] == [1, 1]


def test_invalid_problems(L):
    for kw in (dict(N=1000), dict(k=0), dict(k=129), dict(d_K=0)):
        assert _all(L, _prob(**kw), _cache()) == [1, 1, 1]
    assert _all(L, None, _cache()) == [1, 1, 1]
    assert _all(L, _prob(), None) == [1, 1, 1]


def test_null_and_unaligned_pointers(L):
    P, Q = ctypes.byref(_prob()), ctypes.byref(_cache())
    for fn, count, optional in ((L.zeta_cache_append, 7, ()), (L.zeta_cache_order, 7, ()),
                                (L.zeta_cache_attend, 13, (12,))):
        for pos in range(count):
            a = [FAKE] * count
            a[pos] = None
            if pos not in optional:
                assert fn(P, Q, *a, None, None) == 1, (fn, pos)
    odd = ctypes.c_void_p(0x1008)
    for pos in (1, 6):                     # v, v_pages
        a = [FAKE] * 7
        a[pos] = odd
        assert L.zeta_cache_append(P, Q, *a, None, None) == 1
    for pos in (5, 6):                     # order_codes, order_idx
        a = [FAKE] * 7
        a[pos] = odd
        assert L.zeta_cache_order(P, Q, *a, None, None) == 1
    for pos in (6, 10):                    # v_pages, out
        a = [FAKE] * 13
        a[pos] = odd
        assert L.zeta_cache_attend(P, Q, *a, None, None) == 1


def test_empty_calls_are_no_ops(L):
    for p, c in ((_prob(B=0), _cache()), (_prob(H=0), _cache()), (_prob(), _cache(n=0))):
        P, Q = ctypes.byref(p), ctypes.byref(c)
        assert L.zeta_cache_append(P, Q, *[None] * 9) == 0
        assert L.zeta_cache_order(P, Q, *[None] * 9) == 0
        assert L.zeta_cache_attend(P, Q, *[None] * 15) == 0
    # the binding's marshalling matches the C signatures
    p, c = _prob(B=0), _cache()
    zb.zeta_cache_append(p, c, *[None] * 7, stream=0)
    zb.zeta_cache_order(p, c, *[None] * 7, stream=0)
    zb.zeta_cache_attend(p, c, *[None] * 12, stream=0)


def test_the_handle_wants_cuda_pools():
    with pytest.raises(ValueError):
        ZetaCache.empty(4, 16, 2, 3, 64, 64, 32, 4, device="cpu")
    k = torch.zeros(4, 2, 16, 3)
    with pytest.raises(ValueError):
        ZetaCache(k, torch.zeros(4, 2, 8, 64), k, k, 64, 32, 4)
    with pytest.raises(TypeError):
        ZetaCache(k, torch.zeros(4, 2, 16, 64).half(), k, k, 64, 32, 4)


@pytest.mark.parametrize("weight,kind", [("cauchy", oracle.CAUCHY), ("softmax", oracle.SOFTMAX),
                                         ("inv_euclid", oracle.INV_EUCLID)])
def test_plain_forms_equal_the_oracle(weight, kind):
    """The rows that the GPU tests compare with are the oracle's rows of the whole
    sequence: windows equal, sums to 1e-12."""
    w = W.TINY.replace(name="cache_plain", H=2, N=256, C=64, k=11, bits=4, d_V=8,
                       gamma=(0.4, 0.9))
    g = W.generate(w)
    seq = Sequence(g["q"][0], g["k"][0], g["v"][0].astype(np.float64), w.C, w.k, w.bits,
                   g["gamma"], weight)
    for h in range(w.H):
        idx = oracle.select(seq.qc[h][None], seq.kc[h][None], w.C, w.k)[0]
        out, rs = oracle.attend_fwd(g["q"][0, h], g["k"][0, h], g["v"][0, h],
                                    float(g["gamma"][h]), idx, w.C, kind=kind)
        for i in range(0, w.N, 5):
            win, o, s, bo, bs = seq.row(h, i, 0.0, 2.0 ** -24)
            assert np.array_equal(win if len(win) else np.full(w.k, -1), idx[i])
            assert np.abs(o - out[i]).max() <= 1e-12 * max(1, np.abs(out[i]).max())
            assert abs(s - rs[i]) <= 1e-12 * rs[i]
            assert (bo > 0).all() and bo.max() < 1e-3 and 0 < bs < 1e-3 * s
        t, tok = oracle.prefix_table(seq.kc[h][None], w.C)
        for c in range(1, w.N // w.C):
            lo = w.C * c * (c - 1) // 2
            z, j = seq.prefix(h, c)
            assert np.array_equal(z, t[0, lo:lo + c * w.C])
            assert np.array_equal(j, tok[0, lo:lo + c * w.C])
