"""GPU tests of the tile kernel's blocks of 16, 32 and 64 rows at the edges of what the
paged cache's calls allow, against the plain 64-bit form.

The rule that chooses the block: 64 rows from sequences x heads x rows of 65,536 on,
32 rows from 7,296 on, else 16."""
import numpy as np
import pytest
import torch

from cache_util import attend_row, window
from gpu_util import in_threads
from test_gpu_cache import PAD, Serving, _work
from test_gpu_cache_bits import HALF_OUT, TILE

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

WEIGHTS = pytest.mark.parametrize("weight", ["cauchy", "softmax", "inv_euclid"])
BLOCKS = [dict(H=2), dict(H=8), dict(B=16, H=8), dict(B=16, H=8, d_V=128)]


def _name(kw):
    return "-".join(f"{a}{b}" for a, b in kw.items())


def _large(**kw):
    return _work(**{**dict(B=5, N=1536, C=512, k=24, gamma=(0.3, 1.0)), **kw})


def rows_without(sv, b, h, i, gone, weight):
    """(out, rowsum, bounds) of position i when the tokens of gone are left out; None when
    nothing is left."""
    s, w = sv.seqs[b], sv.w
    win = window(s.qc[h, i], s.kc[h], i, w.C, w.k)
    j = np.array([x for x in [*win, *range(i // w.C * w.C, i + 1)] if x not in gone], np.int64)
    if not len(j):
        return None
    none = np.empty(0, np.int64)
    return attend_row(s.q[h, i], s.k[h][j], s.v[h][j], s.gamma[h], none, len(j) - 1, len(j),
                      weight, TILE, HALF_OUT)


@WEIGHTS
@pytest.mark.parametrize("kw", BLOCKS, ids=_name)
def test_pages_out_of_range_in_the_own_chunk(kw, weight):
    """Pages of 16 tokens, so that half a warp's lanes meet the missing page while the
    others do not: the first, a middle and the last page of the own chunk, and one that
    only windows reach."""
    w = _large(**kw)
    sv = Serving(w, 16, weight)
    sv.step([512] * w.B)
    start, count, q, k, v = sv.batch([512] * w.B, 512)
    sv.cache.append(k, v, start, count, sv.table)
    gone = {b: set() for b in range(w.B)}
    bad = sv.table.clone()
    for b, t in ((0, 512), (1, 768 + 16), (2, 1008), (3, 192), (4, 512 + 48), (4, 512 + 80)):
        bad[b, t // 16] = -1 if b % 2 else 10 ** 6
        gone[b] |= set(range(t, t + 16))
    out = torch.full((w.B, w.H, 512, w.d_V), PAD, dtype=torch.bfloat16, device="cuda")
    rs = torch.full((w.B, w.H, 512), PAD, device="cuda")
    sv.cache.attend(q, sv.gamma, start, count, bad, out, rs, sv.table)
    assert int(sv.cache.status.item()) == 6
    out, rs = out.double().cpu().numpy(), rs.cpu().numpy()

    def one(bt):
        b, t = bt
        for h in (0, w.H - 1):
            want = rows_without(sv, b, h, 512 + t, gone[b], weight)
            if want is None:
                assert rs[b, h, t] == 0 and np.isnan(out[b, h, t]).all()
                continue
            o, s, bo, bs = want
            assert abs(rs[b, h, t] - s) <= bs, (b, h, t, rs[b, h, t], s)
            assert (np.abs(out[b, h, t] - o) <= bo).all(), (b, h, t)

    in_threads(one, [(b, t) for b in [*range(5), w.B - 1]
                     for t in (0, 15, 16, 63, 64, 100, 271, 290, 300, 495, 511)])


@WEIGHTS
@pytest.mark.parametrize("B,v_dtype", [(2, "bf16"), (2, "f32"), (600, "bf16")])
def test_pages_out_of_range_under_single_tokens(B, v_dtype, weight):
    """The row kernel, a cluster of blocks a token and one block a token: half a warp's
    lanes meet a missing page in the own chunk, more than one segment of 1024 keys long."""
    w = _work(B=2, H=2, N=4096, C=2048, k=24, v_dtype=v_dtype, gamma=(0.3, 1.0))
    sv = Serving(w, 16, weight)
    sv.step([2048] * 2)
    sv.step([1500] * 2)
    gone = {0: set(), 1: set()}
    bad = sv.table.clone()
    for b, t in ((0, 2048), (0, 2048 + 1040), (1, 2048 + 1488), (1, 304)):
        bad[b, t // 16] = -1 if b else 10 ** 6
        gone[b] |= set(range(t, t + 16))
    start, count, q, k, v = sv.batch([1, 1], 1)
    sv.cache.append(k, v, start, count, sv.table)
    many = [x.repeat(B // 2, *[1] * (x.dim() - 1)) for x in (q, start, count, bad, sv.table)]
    out = torch.full((B, w.H, 1, w.d_V), PAD, dtype=sv.vdt, device="cuda")
    rs = torch.full((B, w.H, 1), PAD, device="cuda")
    sv.cache.attend(many[0], sv.gamma, many[1], many[2], many[3], out, rs, many[4])
    assert int(sv.cache.status.item()) == 6
    for x in (out, rs):                                     # copies of two rows
        assert torch.equal(x.view(B // 2, 2, -1), x[:2].reshape(1, 2, -1).expand(B // 2, -1, -1))
    out, rs = out.double().cpu().numpy(), rs.cpu().numpy()
    for b in range(2):
        for h in range(w.H):
            o, s, bo, bs = rows_without(sv, b, h, 3548, gone[b], weight)
            assert abs(rs[b, h, 0] - s) <= bs
            assert (np.abs(out[b, h, 0] - o) <= bo).all()
