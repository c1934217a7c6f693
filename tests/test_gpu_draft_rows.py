"""GPU tests of attend_tree's row kernel (values wider than 128 or no multiple of 16 bytes, more than
four coordinates): its weights over several segments of keys, and everything that may be wrong with
parents, pages, order entries and values."""
import numpy as np
import pytest
import torch

from order_retrieval_gb300 import workloads as W

from draft_util import Drafting, line

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

FORMS = [dict(d_V=33), dict(d_V=256), dict(d_V=33, v_dtype="f32"), dict(d_K=5, bits=12),
         dict(d_K=8, bits=8, d_V=136, v_dtype="f32"), dict(d_V=1)]


def _work(**kw):
    base = dict(name="draft", B=2, H=2, N=512, d_K=3, d_V=64, k=16, C=64, bits=10, v_dtype="bf16",
                gamma=(0.3, 0.8), dist="uniform", v_dist="normal", seed=41)
    base.update(kw)
    return W.Workload(**base)


def _name(kw):
    return "-".join(f"{a}{b}" for a, b in kw.items())


@pytest.mark.parametrize("weight", ["softmax", "inv_euclid"])
@pytest.mark.parametrize("kw", FORMS, ids=_name)
def test_weight_kernels(kw, weight):
    w = _work(B=4, C=96, N=480, k=20, dist="clusters", **kw)
    d = Drafting(w, 32, [200, 480 - 7, 50, 300], [30, 12, 33, 1], 33, weight)
    d.attend()
    d.check()


@pytest.mark.parametrize("weight", ["cauchy", "softmax", "inv_euclid"])
@pytest.mark.parametrize("kw", FORMS, ids=_name)
def test_segments_of_keys(kw, weight):
    """More than 1024 and 2048 keys a node.  Sequence 0: the nearest is the node itself, in the last
    segment; 1: a key in the first one, in the place of the query; 2: a node of the line."""
    w = _work(B=3, H=1, C=2048, N=8192, k=200, **kw)
    d = Drafting(w, 64, [2048 + 2000, 4096 + 900, 2048 + 1500], [3, 3, 12], 12, weight, kind="chain")
    d.qn[0, :, :3] = d.kn[0, :, :3]
    d.q[0, :, :3] = d.k[0, :, :3]
    for t in range(3):                               # a token of the own chunk's beginning
        d.qn[1, :, t] = d.g["k"][1, :, 4096 + 40 * t]
        d.q[1, :, t] = torch.from_numpy(d.g["k"][1, :, 4096 + 40 * t]).cuda()
    d.qn[2, :, 11] = d.kn[2, :, 6]
    d.q[2, :, 11] = d.k[2, :, 6]
    d.attend()
    d.check()


@pytest.mark.parametrize("kw", FORMS, ids=_name)
@pytest.mark.parametrize("n", [10, 40])
def test_bad_parents(n, kw):
    w = _work(B=4, **kw)
    d = Drafting(w, 16, [100, 200, 300, 150], [n] * 4, n)
    parents = [p.copy() for p in d.parents]
    lost = set()
    for b, (t, p) in {0: (3, 3), 1: (4, 7), 2: (0, -2), 3: (5, -2 ** 31)}.items():
        lost |= {(b, u) for u in range(n) if t in line(parents[b], u)}
        d.parent[b, t] = p
    d.attend(status=6)
    d.check(skip=lost)


@pytest.mark.parametrize("kw", FORMS, ids=_name)
@pytest.mark.parametrize("page_id", [-1, 10 ** 6, -2 ** 31])
def test_bad_pages(page_id, kw):
    w = _work(C=128, N=1024, k=20, **kw)
    d = Drafting(w, 16, [700, 600], [30, 20], 30, split_tables=True)
    d.table[0, 650 // 16] = page_id                  # tokens 640..655, chunk from 640
    d.table[1, 100 // 16] = page_id                  # tokens 96..111
    d.attend(status=6)
    lost = [set(range(640, 656)), set(range(96, 112))]
    d.check(gone=lambda b: lost[b])


@pytest.mark.parametrize("weight", ["cauchy", "softmax"])
@pytest.mark.parametrize("kw", FORMS, ids=_name)
@pytest.mark.parametrize("entry", [256, -1, 2 ** 31 - 1])
def test_bad_order_entries(entry, kw, weight):
    w = _work(**kw)
    d = Drafting(w, 16, [300, 200], [12, 12], 12, weight)
    plane, e = 300 // 64 & 1, 100
    p = int(d.table_np[0][e // 16])
    token = d.cache.order_idx[plane, p, :, e % 16].tolist()
    d.cache.order_idx[plane, p, :, e % 16] = entry   # not in [0, 256), the prefix's length
    # who looks at it: nodes whose window holds the token
    seen = any(token[h] in d.plain(0, t, h)[0] for t in range(12) for h in range(w.H)
               if d.has_result(0, t))
    out, rs, idx = d.attend(status=6 if seen else 0)
    for b in range(2):
        for t in range(12):
            for h in range(w.H):
                gone = {token[h]} if b == 0 else set()
                win, o, s, bo, bs = d.plain(b, t, h, gone)
                want = np.where(np.isin(win, list(gone)), -1, win)
                assert np.array_equal(idx[b, h, t].cpu().numpy(), want)
                assert (np.abs(out[b, h, t].double().cpu().numpy() - o) <= bo).all()
                assert abs(float(rs[b, h, t]) - s) <= bs


@pytest.mark.parametrize("kw", FORMS, ids=_name)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite(bad, kw):
    w = _work(C=256, N=1024, k=20, **kw)
    d = Drafting(w, 64, [600, 700], [40, 30], 40)
    d.v[0, :, 11] = bad                              # a node
    d.k[0, :, 11] = float("nan")
    e = 300                                          # a token of the prefix
    d.cache.v_pages[d.table_np[1][e // 64], :, e % 64] = bad
    t = torch.arange(600, 640, device="cuda")        # rows behind the sequence's end
    d.cache.v_pages[d.table[0].long()[t // 64], :, t % 64] = bad
    d.cache.k_pages[d.table[0].long()[t // 64], :, t % 64] = float("nan")
    out, rs, idx = d.attend()
    good = set()
    for b in range(2):
        for t in range(d.counts[b]):
            for h in range(w.H):
                sees = b == 0 and 11 in line(d.parents[0], t) or b == 1 and e in idx[b, h, t].tolist()
                assert bool(torch.isfinite(out[b, h, t].float()).all()) != sees, (b, t, h)
            if all(torch.isfinite(out[b, h, t].float()).all() for h in range(w.H)):
                good.add((b, t))
    assert good
    d.values[1][:, e] = 0                            # any value: it is in none of their sets
    d.check(good)


@pytest.mark.parametrize("kw", FORMS, ids=_name)
def test_the_chunks_end_and_empty_sequences(kw):
    """Nodes behind the chunk's end and padding are left as they were; sequences out of range too."""
    w = _work(B=5, **kw)
    d = Drafting(w, 16, [511, 0, 63, 64, 100], [7, 7, 0, 1, 7], 7, kind="chain")
    d.start[4], d.starts[4], d.counts[4] = 600, 0, 0
    d.attend(status=6)
    d.check()
