"""GPU tests of attend_tree's block layouts (groups of 8 nodes, clusters), of memory that is
aligned no better than it must be, and of what batches of unequal sequences leave alone."""
import numpy as np
import pytest
import torch

from order_retrieval_gb300 import ZetaCache
from order_retrieval_gb300 import workloads as W

from draft_util import Drafting

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]


def _work(**kw):
    base = dict(name="draft", B=4, H=2, N=1024, d_K=3, d_V=64, k=20, C=256, bits=10,
                v_dtype="bf16", gamma=(0.4, 1.0), dist="uniform", v_dist="normal", seed=23)
    base.update(kw)
    return W.Workload(**base)


def _name(kw):
    return "-".join(f"{a}{b}" for a, b in kw.items()) or "base"


# Slices: 2, 24, 60, 160 and 400; with chunks of 256 a tree has one block or two (wider clusters:
# below and in test_gpu_draft_layouts.py).
@pytest.mark.parametrize("weight", ["cauchy", "softmax", "inv_euclid"])
@pytest.mark.parametrize("kw", [dict(), dict(v_dtype="f32"), dict(d_V=128), dict(d_V=72, k=70),
                                dict(v_dtype="f32", d_V=100), dict(d_K=2, bits=21, d_V=40)],
                         ids=_name)
@pytest.mark.parametrize("B,H,n", [(1, 2, 8), (1, 2, 33), (3, 8, 17), (15, 4, 40), (20, 8, 8),
                                   (20, 8, 19), (50, 8, 3), (50, 8, 24)])
def test_block_layouts(B, H, n, kw, weight):
    w = _work(B=B, H=H, **kw)
    rng = np.random.default_rng(B + n)
    starts = rng.integers(w.C, w.N, B)
    starts[0] = 700
    d = Drafting(w, 64, starts, np.maximum(1, rng.integers(n // 2, n + 1, B)), n, weight,
                 kind="bushy")
    d.attend()
    picks = {(int(b), int(t)) for b in rng.integers(0, B, 12) for t in rng.integers(0, n, 3)}
    d.check(picks | {(0, 0), (0, n - 1)}, heads=(0, H - 1))


@pytest.mark.parametrize("weight", ["cauchy", "softmax", "inv_euclid"])
@pytest.mark.parametrize("kw", [dict(), dict(d_V=128), dict(d_V=72), dict(v_dtype="f32", d_V=128),
                                dict(v_dtype="f32", d_V=20)], ids=_name)
@pytest.mark.parametrize("B,H,n", [(1, 1, 5), (2, 1, 16), (3, 5, 30), (9, 7, 8)])
def test_long_chunks_over_many_blocks(B, H, n, kw, weight):
    """Chunks long enough that up to eight blocks share a tree's keys, some of them none."""
    w = _work(B=B, H=H, C=4096, N=8192, **kw)
    starts = [8000, 4096 + 3, 4095][:B] + [5000] * (B - 3)
    d = Drafting(w, 64, starts, [n] * B, n, weight)
    d.attend()
    d.check({(b, t) for b in range(min(B, 4)) for t in range(0, n, 3)}, heads=(0, H - 1))


def _moved(t, elements):
    """The same tensor some elements behind an aligned address."""
    buf = torch.empty(t.numel() + elements, dtype=t.dtype, device=t.device)
    out = buf[elements:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("v_dtype,d_V", [("bf16", 64), ("bf16", 48), ("bf16", 128), ("f32", 64)])
@pytest.mark.parametrize("page", [16, 64, 4])
def test_memory_that_is_barely_aligned(v_dtype, d_V, page):
    """Values on 16 bytes but not 32, coordinates and the other arrays on 4."""
    w = _work(v_dtype=v_dtype, d_V=d_V)
    d = Drafting(w, page, [700, 300, 513, 1000], [12, 20, 3, 20], 20)
    want = [x.clone() for x in d.attend()]
    c, off = d.cache, 8 if v_dtype == "bf16" else 4
    d.cache = ZetaCache(_moved(c.k_pages, 1), _moved(c.v_pages, off), c.order_codes, c.order_idx,
                        w.N, w.C, w.k, w.bits)
    d.v, d.k, d.q = _moved(d.v, off), _moved(d.k, 1), _moved(d.q, 1)
    d.parent, d.table = _moved(d.parent, 1), _moved(d.table, 3)
    outputs = d.outputs
    d.outputs = lambda: (_moved(outputs()[0], off), _moved(outputs()[1], 1), _moved(outputs()[2], 1))
    out, rs, idx = d.attend()
    d.check()
    assert torch.equal(idx, want[2])
    # accept writes to the same places; reserve takes lists anywhere
    acc, path = d.ints([0] * 4), _moved(d.ints(np.zeros((4, 20))), 1)
    d.cache.accept(d.k, d.v, d.start, d.count, d.parent, d.ints([11, 19, 2, 19]), d.table, acc,
                   path)
    assert int(d.cache.status.item()) == 0 and acc.min() > 0
    for b in range(4):
        for j in range(int(acc[b])):
            i = d.starts[b] + j
            p = int(d.table_np[b][i // page])
            assert torch.equal(d.cache.v_pages[p, :, i % page], d.v[b, :, int(path[b, j])])
            assert torch.equal(d.cache.k_pages[p, :, i % page], d.k[b, :, int(path[b, j])])
    table, held = _moved(d.ints(np.full((4, 70), -1)), 1), _moved(d.ints([0] * 4), 1)
    pages = c.pages
    free, fc = _moved(d.ints(np.arange(pages)), 1), _moved(d.ints([pages]), 1)
    got, slots = _moved(d.ints([0] * 4), 1), _moved(d.ints(np.zeros((4, 20))), 1)
    d.cache.status.zero_()
    if page > 4:
        d.cache.reserve(d.start, d.count, table, held, free, fc, got, slots)
        assert int(d.cache.status.item()) == 0
        assert held.tolist() == [-(-(s + n) // page) for s, n in zip(d.starts, d.counts)]
        for b in range(4):
            i = d.starts[b] + np.arange(d.counts[b])
            t = table[b].cpu().numpy()
            assert np.array_equal(slots[b, :d.counts[b]].cpu().numpy(), t[i // page] * page + i % page)


@pytest.mark.parametrize("v_dtype,B", [("bf16", 3), ("bf16", 40), ("f32", 3)])
def test_a_batch_of_unequal_sequences(v_dtype, B):
    """Empty texts, full ones, idle slots and trees of one node side by side: the rows of each
    are what they are alone, and nothing else is written."""
    w = _work(B=B, H=4, v_dtype=v_dtype)
    rng = np.random.default_rng(7)
    starts = rng.choice([0, 1, w.C - 1, w.C, 500, w.N - 1], B)
    counts = rng.choice([0, 1, 2, 9, 18], B)
    counts[0] = 18
    d = Drafting(w, 32, starts, counts, 18)
    out, rs, idx = (x.clone() for x in d.attend())
    d.check({(b, t) for b in range(B) for t in range(18)}, heads=(3,))
    one = ZetaCache(d.cache.k_pages, d.cache.v_pages, d.cache.order_codes, d.cache.order_idx, w.N,
                    w.C, w.k, w.bits)
    for b in range(0, B, max(1, B // 3)):
        o, r, i = (x[b:b + 1].clone() for x in d.outputs())
        args = [x[b:b + 1].contiguous() for x in (d.q, d.k, d.v)]
        more = [x[b:b + 1].contiguous() for x in (d.start, d.count, d.parent, d.table)]
        one.attend_tree(*args, d.gamma, *more, o, r, idx=i)
        assert torch.equal(i[0], idx[b])
        # another layout joins the same float32 sums in another order
        ok = r[0] != 7.0
        assert torch.equal(ok, rs[b] != 7.0)
        assert ((r[0] - rs[b]).abs() <= 2 * (w.C + w.k + 18) * 2.0 ** -24 * rs[b].abs())[ok].all()
        big = out[b].float().abs().amax(-1, keepdim=True).clamp(min=1e-6)
        step = torch.finfo(out.dtype).eps * (1 if v_dtype == "bf16" else 2 * (w.C + w.k + 18))
        assert ((o[0].float() - out[b].float()).abs() <= step * big)[ok].all()
    assert int(one.status.item()) == 0
