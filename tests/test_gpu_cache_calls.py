"""GPU tests of the paged cache's handle: which lengths its calls take, and what it does
when its pools change under it."""
import pytest
import torch

from order_retrieval_gb300 import ZetaError
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
