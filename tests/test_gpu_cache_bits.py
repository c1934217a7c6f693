"""GPU tests of how many bits the paged cache's attention keeps: bf16 results within the
rounding of the stored value itself, whichever kernel the size of the batch chooses.

Bounds are those of tests/cache_util.py.  The row kernel rounds no weight.  The tile
kernel carries a weight as a bf16 half and the bf16 of what that leaves: the half is off
by at most 2^-8 of the weight, its rest by 2^-8 of that, 2^-16 together."""
import numpy as np
import pytest
import torch

from gpu_util import in_threads
from test_gpu_cache import Serving, _work

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

HALF_OUT = 2.0 ** -8
TILE, ROW = 2.0 ** -16, 0.0


def hold(sv, half_w, rows=None, heads=None):
    """Collected rows (of the positions in rows) against the plain form; bf16 values."""
    w = sv.w

    def one(bi):
        b, i = bi
        idx, out, rs = sv.got[b][i]
        for h in range(w.H) if heads is None else heads:
            win, o, s, bo, bs = sv.seqs[b].row(h, i, half_w, HALF_OUT)
            assert np.array_equal(idx[h], win if len(win) else np.full(w.k, -1)), (b, h, i)
            off = np.abs(out[h] - o) - bo
            assert (off <= 0).all(), (b, h, i, off.max(), bo[off.argmax()])
            assert abs(rs[h] - s) <= bs, (b, h, i, rs[h], s)

    todo = [(b, i) for b in range(w.B) for i in sv.got[b] if rows is None or i in rows]
    assert todo
    in_threads(one, todo)


def sampled(w, first, count, seed):
    rng = np.random.default_rng(seed)
    return set(rng.integers(first, w.N, count).tolist()) | {first, w.N - 1}


# Pieces of 512 rows: blocks of 16 rows (8 slices), 32 (10 slices) and 64 (32 for values
# wider than 64).
@pytest.mark.parametrize("weight", ["cauchy", "softmax", "inv_euclid"])
@pytest.mark.parametrize("kw", [dict(B=8, H=1), dict(B=8, H=1, d_V=128), dict(H=2), dict(B=16, H=8),
                                dict(B=16, H=8, d_V=128)],
                         ids=lambda x: "-".join(f"{a}{b}" for a, b in x.items()))
def test_large_pieces_keep_the_weights_bits(kw, weight):
    w = _work(**{**dict(B=5, N=1536, C=512, k=24, gamma=(0.3, 1.0)), **kw})
    sv = Serving(w, 64, weight)
    for _ in range(3):
        sv.step([512] * w.B)
    hold(sv, TILE, sampled(w, 0, 24, 7), heads=(0, w.H - 1))


@pytest.mark.parametrize("weight", ["cauchy", "softmax", "inv_euclid"])
@pytest.mark.parametrize("counts", [[1, 1, 1], [5, 3, 4], [7, 0, 7]])
def test_few_tokens_keep_the_weights_bits(counts, weight):
    """Up to seven rows a sequence: no weight is rounded to fewer bits."""
    w = _work(B=3, H=2, N=640, C=128, k=24, gamma=(0.3, 1.0))
    sv = Serving(w, 32, weight)
    while sv.len.min() < 560:
        sv.step([min(128, 560 - int(m)) for m in sv.len])
    sv.got = [dict() for _ in range(w.B)]
    while sv.len.max() < 630:
        sv.step(counts)
    hold(sv, ROW)
