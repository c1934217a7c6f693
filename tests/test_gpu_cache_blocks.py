"""GPU tests of the tile kernel's blocks of 16, 32 and 64 rows at the edges of what the
paged cache's calls allow, against the plain 64-bit form.  Pieces of 512 rows of eight
slices run in blocks of 16 rows, of ten slices in blocks of 32, of forty and more in blocks
of 64 rows (32 where values are wider than 64)."""
import numpy as np
import pytest
import torch

from cache_util import EPS, Sequence, attend_row, window
from gpu_util import in_threads
from test_gpu_cache import PAD, Serving, _work
from test_gpu_cache_bits import HALF_OUT, TILE, hold

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

WEIGHTS = pytest.mark.parametrize("weight", ["cauchy", "softmax", "inv_euclid"])
BLOCKS = [dict(B=8, H=1), dict(B=8, H=1, d_V=128), dict(H=2), dict(B=16, H=8),
          dict(B=16, H=8, d_V=128)]


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
    halves = (TILE, HALF_OUT) if w.v_dtype == "bf16" else (0.0, EPS)
    return attend_row(s.q[h, i], s.k[h][j], s.v[h][j], s.gamma[h], none, len(j) - 1, len(j),
                      weight, *halves)


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


# The largest blocks: sixteen sequences, eight heads, pieces of 512 rows.
WIDE = [
    dict(), dict(d_V=8), dict(d_V=40, k=65), dict(d_V=96), dict(d_V=128, k=100),
    dict(d_K=1, bits=21, d_V=32), dict(d_K=4, bits=8, d_V=128), dict(d_K=2, bits=21, d_V=72),
    dict(bits=1), dict(dist="clusters", bits=12), dict(C=520, N=2600, k=33),
]


@WEIGHTS
@pytest.mark.parametrize("kw", WIDE, ids=lambda x: _name(x) or "base")
def test_the_largest_blocks(kw, weight):
    """Whole pieces (no window, then windows), then ragged pieces across a chunk's end with
    idle sequences and single tokens beside them."""
    w = _large(**{**dict(B=16, H=8, N=2560), **kw})
    sv = Serving(w, 64, weight)
    c = w.C
    sv.step([c] * 16)
    sv.step([c, c - 60] * 8, n=c)
    sv.step([c, c, 100, 0, c - 1, 17, 1, 333] * 2, n=c)
    sv.check_order()
    rng = np.random.default_rng(5)
    rows = {0, 1, 62, 63, 64, c - 1, c, c + 1, 2 * c - 61, 2 * c - 60, 2 * c, 2 * c + 16}
    hold(sv, TILE, rows | set(rng.integers(0, 3 * c, 8).tolist()), heads=(0, 7))


@pytest.mark.parametrize("d_V", [64, 128])
def test_the_largest_blocks_with_values_that_are_not_finite(d_V):
    """Infinities and NaN in later tokens of the own chunk and in keys of other rows'
    windows reach only the rows that attend to them."""
    w = _large(B=16, H=8, d_V=d_V)
    sv = Serving(w, 64)
    bad = {0: 700, 1: 1200, 2: 100, 9: 1535}
    for b, t in bad.items():
        sv.v[b, :, t] = float("inf") if b else float("nan")
    for _ in range(3):
        sv.step([512] * 16)
    for b, t in bad.items():
        for i in range(3, w.N, 7):
            win, o, r = (x[7] for x in sv.got[b][i])
            sees = t in win.tolist() or (t // 512 == i // 512 and t <= i)
            assert np.isfinite(o).all() != sees, (b, i)
            assert np.isfinite(r)
    sv.seqs = [Sequence(s.q, s.k, np.nan_to_num(s.v, nan=0.0, posinf=0.0), s.C, s.ksel, w.bits,
                        s.gamma, "cauchy") for s in sv.seqs]
    for b in bad:
        sv.got[b] = {i: x for i, x in sv.got[b].items() if np.isfinite(x[1]).all()}
    hold(sv, TILE, set(range(0, w.N, 61)), heads=(0, 7))


def test_captured_largest_blocks():
    """A step captured into a graph and replayed equals the eager one, bit for bit."""
    w = _large(B=16, H=8)
    sv, twin = Serving(w, 64), Serving(w, 64)
    for x in (sv, twin):
        x.step([512] * 16)
    start, count, q, k, v = sv.batch([512, 400] * 8, 512)
    got = []
    for x, graph in ((sv, True), (twin, False)):
        c = x.cache
        out = torch.full((16, 8, 512, 64), PAD, dtype=torch.bfloat16, device="cuda")
        rs = torch.full((16, 8, 512), PAD, device="cuda")

        def step():
            c.append(k, v, start, count, x.table)
            c.order(start, count, x.table, n=512)
            c.attend(q, x.gamma, start, count, x.table, out, rs)

        if graph:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step()
            for _ in range(2):
                g.replay()
        else:
            step()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        got.append((out, rs, c.order_idx.clone()))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert (got[0][0][1, :, 400:] == PAD).all()


@WEIGHTS
@pytest.mark.parametrize("d_V", [64, 128])
def test_blocks_of_a_few_rows(d_V, weight):
    """Up to seven rows of many sequences under chunks of 1000, enough to share them: idle
    sequences, single rows and rows on both sides of a chunk's end."""
    w = _large(B=32, H=8, N=3000, C=1000, d_V=d_V)
    sv = Serving(w, 64, weight)
    sv.step([1000] * 32)
    sv.step([996, 995, 997, 700] * 8, n=1000)
    sv.got = [dict() for _ in range(32)]
    sv.step([7, 7, 0, 5, 1, 6, 7, 2] * 4, n=7)
    sv.check_order()
    sv.step([7, 3, 7, 7] * 8, n=7)
    hold(sv, TILE, heads=(0, 7))
