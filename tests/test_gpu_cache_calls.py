"""GPU tests of the paged cache's handle: which lengths its calls take, and what it does
when its pools change under it."""
import pytest
import torch

from order_retrieval_gb300 import ZetaCache, ZetaError
from test_gpu_cache import PAD, _fresh, _small

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]


def _pools(c):
    return [x.clone() for x in (c.k_pages, c.v_pages, c.order_codes, c.order_idx)]


@pytest.mark.parametrize("n", [1, 4])
def test_more_tokens_than_rows_are_skipped_by_every_call(n):
    """A count of n + 1 that would complete a chunk: append, order and attend of the step all
    skip the sequence and say so; the other sequence goes on."""
    w, sv, _ = _small()
    start = torch.tensor([w.C + w.C - n, w.C + w.C - n], dtype=torch.int32).cuda()
    count = torch.tensor([n + 1, n], dtype=torch.int32).cuda()
    q, k, v = (x[:, :, w.C:w.C + n].contiguous() for x in (sv.q, sv.k, sv.v))
    out, rs = _fresh(w, n)
    c = sv.cache
    before = _pools(c)
    for call in (lambda: c.append(k, v, start, count, sv.table),
                 lambda: c.order(start, count, sv.table, n=n),
                 lambda: c.attend(q, sv.gamma, start, count, sv.table, out, rs)):
        c.status.zero_()
        call()
        assert int(c.status.item()) == 6
    mine = sv.table[0].long()
    mine = mine[mine >= 0]
    for old, new, dim in zip(before, _pools(c), (0, 0, 1, 1)):
        assert torch.equal(old.index_select(dim, mine), new.index_select(dim, mine))
    assert not torch.equal(before[3], c.order_idx)           # sequence 1 has its prefix
    assert (out[0] == PAD).all() and (rs[0] == PAD).all() and (rs[1] != PAD).all()


def test_order_takes_the_step_rows():
    w, sv, n = _small()
    c = sv.cache
    st = torch.full((2,), 32, dtype=torch.int32).cuda()
    ct = torch.full((2,), 32, dtype=torch.int32).cuda()
    sv.step([32, 32])
    want = _pools(c)
    c.order_idx[0] = 0
    c.order(st, ct, sv.table)                                # default: up to C
    assert torch.equal(want[3], c.order_idx)
    c.order_idx[0] = 0
    c.order(st, ct, sv.table, n=32)
    assert torch.equal(want[3], c.order_idx)
    for bad, code in ((w.C + 1, 2), (-1, 1)):
        with pytest.raises(ZetaError) as e:
            c.order(st, ct, sv.table, n=bad)
        assert e.value.code == code
    assert int(c.status.item()) == 0


def _step(w, sv, c, n, table):
    start, count, q, k, v = sv.batch([n, n], n)
    out, rs = _fresh(w, n)
    c.append(k, v, start, count, table)
    c.order(start, count, table, n=n)
    c.attend(q, sv.gamma, start, count, table, out, rs)
    return out, rs


@pytest.mark.parametrize("name", ["k_pages", "v_pages", "order_codes", "order_idx", "status", "k",
                                  "C", "N", "bits", "pages"])
def test_pools_and_sizes_cannot_be_assigned(name):
    """An assigned pool used to be ignored: the calls went on with the old memory."""
    c = ZetaCache.empty(4, 16, 2, 3, 64, 64, 32, 4)
    old = getattr(c, name)
    with pytest.raises(AttributeError):
        setattr(c, name, old.clone() if torch.is_tensor(old) else old + 1)
    assert getattr(c, name) is old


def test_a_cache_may_carry_what_its_user_adds():
    class Named(ZetaCache):
        def __init__(self, *args, **kw):
            super().__init__(*args, **kw)
            self.name = "one"

    c = Named.empty(4, 16, 2, 3, 64, 64, 32, 4)
    c.name = "two"
    c.step = 1
    c.step = 2
    assert (c.name, c.step) == ("two", 2)
    with pytest.raises(AttributeError):
        c.order_pages = 8


@pytest.mark.parametrize("how", ["data", "set_"])
def test_pools_that_move_are_followed(how):
    """New memory under the same tensors, as they hold it at the call: outputs and pools are
    those of a cache that stayed."""
    w, sv, n = _small()
    c = sv.cache
    twin = ZetaCache(*_pools(c), w.N, w.C, w.k, w.bits)
    kept = []
    for t in (c.k_pages, c.v_pages, c.order_codes, c.order_idx, c.status):
        kept.append(t.detach().view(t.shape))                # the old memory, still there
        new = t.clone()
        if how == "data":
            t.data = new
        else:
            t.set_(new)
        kept[-1].zero_()
    got, want = _step(w, sv, c, n, sv.table), _step(w, sv, twin, n, sv.table)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for a, b in zip(_pools(c), _pools(twin)):
        assert torch.equal(a, b)
    assert int(c.status.item()) == 0
    for t in kept:
        assert not t.any()                                   # nobody wrote there


def test_pools_that_no_longer_fit_are_refused():
    """Released or resized memory is an error of the call, on the host."""
    w, sv, n = _small()
    c = sv.cache
    c.v_pages.untyped_storage().resize_(0)
    with pytest.raises(ZetaError) as e:                      # no memory: a null pointer
        _step(w, sv, c, n, sv.table)
    assert e.value.code == 1
    w, sv, n = _small()
    sv.cache.k_pages.data = sv.cache.k_pages[:2].clone()
    with pytest.raises(ValueError):
        _step(w, sv, sv.cache, n, sv.table)
    w, sv, n = _small()
    sv.cache.order_idx.data = sv.cache.order_idx.cpu()
    with pytest.raises(ValueError):
        _step(w, sv, sv.cache, n, sv.table)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dims", [(64,), (2, 64), (2, 4, 3), (2, 2, 4, 3, 1)])
def test_rows_of_other_dimensions_are_refused(dims):
    w, sv, n = _small()
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    x = torch.zeros(dims, device="cuda")
    out, rs = _fresh(w, n)
    v = torch.zeros(2, w.H, n, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        sv.cache.append(x, v, st, st, sv.table)
    with pytest.raises(ValueError):
        sv.cache.attend(x, sv.gamma, st, st, sv.table, out, rs)
