"""GPU tests of the drafting calls (attend_tree, accept, reserve) against their plain forms:
selections, tables and copies bit for bit, sums within bounds counted from the roundings
(tests/cache_util.py)."""
import numpy as np
import pytest
import torch

from order_retrieval_gb300 import ZetaCache, ZetaError
from order_retrieval_gb300 import binding as zb
from order_retrieval_gb300 import workloads as W

from draft_util import PAD, Drafting, line, reserve_plain, tree

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]


def _work(**kw):
    base = dict(name="draft", B=4, H=2, N=512, d_K=3, d_V=64, k=16, C=64, bits=10, v_dtype="bf16",
                gamma=(0.5, 1.0), dist="uniform", v_dist="normal", seed=17)
    base.update(kw)
    return W.Workload(**base)


def _name(kw):
    return "-".join(f"{a}{b}" for a, b in kw.items()) or "base"


SHAPES = [
    (dict(), 16), (dict(v_dtype="f32"), 16), (dict(C=40, N=400, k=7), 16),
    (dict(C=100, N=500, k=33, d_V=40), 32), (dict(C=128, k=128, d_V=32, v_dtype="f32"), 8),
    (dict(d_K=1, bits=21, d_V=128), 64), (dict(d_K=2, bits=21, v_dtype="f32", d_V=128), 1),
    (dict(d_K=4, bits=8, d_V=96), 256), (dict(d_K=8, bits=8, d_V=256, H=1), 512),
    (dict(d_K=5, bits=12, d_V=256, v_dtype="f32", H=1), 16), (dict(d_V=1), 16),
    (dict(d_V=33, v_dtype="f32"), 16), (dict(d_V=250, H=1), 16), (dict(bits=1), 16),
    (dict(dist="clusters", bits=12, H=5), 32), (dict(C=8, N=96, k=3), 16),
    (dict(C=512, N=512), 64), (dict(C=256, k=100, d_V=8), 16), (dict(d_V=4, v_dtype="f32"), 16),
    (dict(d_V=100, v_dtype="f32", k=65, C=128), 16), (dict(d_V=8, H=3, k=1), 16),
]


@pytest.mark.parametrize("kind", ["tree", "bushy", "chain"])
@pytest.mark.parametrize("kw,page", SHAPES, ids=lambda x: str(x) if isinstance(x, int) else
                         _name(x))
def test_trees(kw, page, kind):
    """In the middle of a chunk, next to its end, in the first chunk, an idle sequence."""
    w = _work(**kw)
    C, last = w.C, w.N - w.C
    n = min(C, 37)
    d = Drafting(w, page, [last + C // 2, last - 1 if last else C - 2, C // 3, C],
                 [n, min(n, 9), max(1, n - 5), 0] if last else [n, 9, 1, 0], n, kind=kind)
    d.attend()
    d.check()


@pytest.mark.parametrize("weight", ["softmax", "inv_euclid"])
@pytest.mark.parametrize("v_dtype,d_V", [("bf16", 64), ("f32", 64), ("bf16", 24), ("bf16", 128)])
def test_weight_kernels(weight, v_dtype, d_V):
    w = _work(v_dtype=v_dtype, d_V=d_V, C=96, N=480, k=20, dist="clusters")
    d = Drafting(w, 32, [200, 480 - 7, 50, 300], [30, 12, 33, 1], 33, weight)
    d.attend()
    d.check()


@pytest.mark.parametrize("v_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("start", [0, 1, 63, 64, 65, 127, 128, 448, 511])
def test_lengths(start, v_dtype):
    """From no token at all to the last place there is; one node and some."""
    w = _work(v_dtype=v_dtype)
    d = Drafting(w, 16, [start] * 4, [1, 2, 17, 33], 40)
    d.attend()
    d.check()


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 64, 200, 512, 1024])
def test_numbers_of_nodes(n):
    w = _work(B=2, C=1024, N=4096, k=40)
    d = Drafting(w, 64, [3500, 700], [n, max(1, n - 3)], n, kind="bushy")
    d.attend()
    rng = np.random.default_rng(n)
    d.check({(b, int(t)) for b in range(2) for t in rng.integers(0, n, 60)}, heads=(1,))


@pytest.mark.parametrize("n", [64, 1024])
def test_long_lines(n):
    w = _work(B=2, C=2048, N=4096, k=40)
    d = Drafting(w, 64, [2100, 2048 - 30], [n, n], n, kind="chain")
    d.attend()
    d.check({(b, t) for b in range(2) for t in range(0, n, max(1, n // 50))}, heads=(0,))


@pytest.mark.parametrize("v_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,n", [(1, 4), (40, 5), (150, 24)])
def test_numbers_of_sequences(B, n, v_dtype):
    rng = np.random.default_rng(B)
    w = _work(B=B, H=4, v_dtype=v_dtype, N=1024, C=256, k=24)
    starts = rng.integers(0, w.N, B)
    d = Drafting(w, 64, starts, rng.integers(0, n + 1, B), n)
    d.attend()
    d.check({(int(b), int(t)) for b in rng.integers(0, B, 40) for t in rng.integers(0, n, 4)})


@pytest.mark.parametrize("v_dtype", ["bf16", "f32"])
def test_long_prefixes(v_dtype):
    w = _work(B=2, H=1, N=1 << 17, C=1024, k=64, v_dtype=v_dtype)
    d = Drafting(w, 64, [(1 << 17) - 700, 70000], [20, 8], 20)
    d.attend()
    d.check()


@pytest.mark.parametrize("kw", [dict(), dict(v_dtype="f32", d_V=24), dict(d_K=8, bits=8)],
                         ids=_name)
def test_longest_chunks(kw):
    w = _work(**{**dict(B=2, H=1, N=16384, C=8192, k=200), **kw})
    d = Drafting(w, 128, [16384 - 100, 8191], [12, 5], 12)
    d.attend()
    d.check()


@pytest.mark.parametrize("v_dtype", ["bf16", "f32"])
def test_a_line_is_what_attend_gives(v_dtype):
    """The nodes of one line against the same tokens appended and attended."""
    w = _work(B=3, C=256, N=1024, k=32, v_dtype=v_dtype)
    n = 48
    d = Drafting(w, 64, [300, 0, 256 + 230], [n, n, n], n, kind="chain")
    out, rs, idx = d.attend()
    o2, r2, i2 = d.outputs()
    d.cache.append(d.k, d.v, d.start, d.count, d.table)
    d.cache.order(d.start, d.count, d.table, n=n)
    d.cache.attend(d.q, d.gamma, d.start, d.count, d.table, o2, r2, idx=i2)
    assert int(d.cache.status.item()) == 0
    ok = torch.zeros(3, n, dtype=torch.bool, device="cuda")
    for b in range(3):
        for t in range(n):
            ok[b, t] = d.has_result(b, t)
    assert ok[:2].all() and not ok[2].all()
    ok = ok[:, None].expand(-1, w.H, -1)
    assert torch.equal(idx[ok], i2[ok])
    # float32 sums of up to C + k terms in two orders; out one step of its type apart
    assert ((rs - r2).abs() <= 2 * (w.C + w.k) * 2.0 ** -24 * r2)[ok].all()
    step = torch.finfo(out.dtype).eps * (1 if v_dtype == "bf16" else 2 * (w.C + w.k))
    big = out.float().abs().amax(-1, keepdim=True)
    assert ((out.float() - o2.float()).abs() <= step * big)[ok].all()


def test_an_order_table_of_its_own():
    d = Drafting(_work(), 16, [200, 130, 20, 400], [9, 8, 7, 6], 10, split_tables=True)
    d.attend()
    d.check()


@pytest.mark.parametrize("v_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite(bad, v_dtype):
    """They reach only the nodes that attend to them: a node off the line, tokens in no window,
    the unused end of a page."""
    w = _work(B=2, C=256, N=1024, k=20, v_dtype=v_dtype)
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
    assert 40 < len(good) < 70
    d.values[1][:, e] = 0                            # any value: it is in none of their sets
    d.check(good)


@pytest.mark.parametrize("n", [10, 40])
def test_bad_parents_cost_their_lines(n):
    """A parent that is the node itself, a later one, below -1: the lines through it have no
    result and are not accepted; all others have theirs."""
    w = _work(B=4)
    d = Drafting(w, 16, [100, 200, 300, 150], [n, n, n, n], n)
    parents = [p.copy() for p in d.parents]
    bad = {0: (3, 3), 1: (4, 7), 2: (0, -2), 3: (5, -2 ** 31)}
    lost = set()
    for b, (t, p) in bad.items():
        lost |= {(b, u) for u in range(n) if t in line(parents[b], u)}
        d.parent[b, t] = p
    d.attend(status=6)
    d.check(skip=lost)
    before = d.cache.k_pages.clone()
    d.cache.status.zero_()
    leaf = d.ints([t for t, _ in bad.values()])
    acc, path = d.ints([9] * 4), d.ints(np.full((4, n), 9))
    d.cache.accept(d.k, d.v, d.start, d.count, d.parent, leaf, d.table, acc, path)
    assert int(d.cache.status.item()) == 6
    assert acc.tolist() == [0] * 4 and (path == -1).all()
    assert torch.equal(before, d.cache.k_pages)


@pytest.mark.parametrize("start,count", [(-1, 2), (513, 0), (512, 1), (40, -1), (40, 6),
                                         (2 ** 31 - 1, 3), (-2 ** 31, 1)])
def test_bad_lengths_skip_the_sequence(start, count):
    w = _work(B=2)
    d = Drafting(w, 16, [100, 200], [5, 5], 5)
    d.start[0], d.count[0] = start, count
    d.starts[0], d.counts[0] = 0, 0
    d.attend(status=6)
    d.check()
    d.cache.status.zero_()
    acc = d.ints([9, 9])
    d.cache.accept(d.k, d.v, d.start, d.count, d.parent, d.ints([0, 4]), d.table, acc)
    assert int(d.cache.status.item()) == 6
    assert acc.tolist() == [0, len(line(d.parents[1], 4))]


def test_the_last_place():
    """start = N without drafts is a sequence that is full; start = N - 1 takes one token."""
    w = _work(B=3)
    d = Drafting(w, 16, [512, 511, 511], [0, 3, 1], 3, kind="chain")
    d.attend()
    d.check()
    acc = d.ints([9] * 3)
    d.cache.accept(d.k, d.v, d.start, d.count, d.parent, d.ints([-1, 2, 0]), d.table, acc)
    assert acc.tolist() == [0, 1, 1] and int(d.cache.status.item()) == 0


@pytest.mark.parametrize("v_dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page_id", [-1, 10 ** 6, -2 ** 31])
def test_bad_pages_drop_their_keys(page_id, v_dtype):
    """A page of the own chunk and one of the prefix, an order table of its own."""
    w = _work(B=2, C=128, N=1024, k=20, v_dtype=v_dtype)
    d = Drafting(w, 16, [700, 600], [30, 20], 30, split_tables=True)
    d.table[0, 650 // 16] = page_id                  # tokens 640..655, chunk from 640
    d.table[1, 100 // 16] = page_id                  # tokens 96..111
    d.attend(status=6)
    lost = [set(range(640, 656)), set(range(96, 112))]
    d.check(gone=lambda b: lost[b])


def test_bad_order_entries_are_dropped():
    w = _work(B=2, C=64, N=512, k=16)
    d = Drafting(w, 16, [300, 200], [12, 12], 12)
    plane, e = 300 // 64 & 1, 100
    p = int(d.table_np[0][e // 16])
    token = d.cache.order_idx[plane, p, :, e % 16].tolist()
    d.cache.order_idx[plane, p, :, e % 16] = 256     # not below the prefix's length
    out, rs, idx = d.attend(status=6)
    hit = 0
    for b in range(2):
        for t in range(12):
            for h in range(w.H):
                gone = {token[h]} if b == 0 else set()
                win, o, s, bo, bs = d.plain(b, t, h, gone)
                want = np.where(np.isin(win, list(gone)), -1, win)
                hit += int((want == -1).any())
                assert np.array_equal(idx[b, h, t].cpu().numpy(), want)
                assert (np.abs(out[b, h, t].double().cpu().numpy() - o) <= bo).all()
                assert abs(float(rs[b, h, t]) - s) <= bs
    assert hit > 0


@pytest.mark.parametrize("v_dtype,d_V", [("bf16", 256), ("bf16", 128), ("f32", 64)])
def test_pools_past_32_bit_offsets(v_dtype, d_V):
    """Pages whose bytes lie past 2^32 of the pools."""
    w = _work(B=1, H=8, N=1024, C=256, d_V=d_V, k=20, v_dtype=v_dtype)
    d = Drafting(w, 64, [700], [11], 11)
    want = d.attend()
    pages = 40000                                    # x 8 x 64 rows of at least 256 bytes: 5.2 GB
    ids = torch.arange(16, device="cuda") * 7 + pages - 140
    big = [torch.empty(pages, 8, 64, 3, device="cuda"),
           torch.empty(pages, 8, 64, d_V, dtype=d.vdt, device="cuda")]
    order = [torch.empty(2, pages, 8, 64, dtype=x.dtype, device="cuda")
             for x in (d.cache.order_codes, d.cache.order_idx)]
    old = d.table[0, :16].long()
    for new, x in zip(big, (d.cache.k_pages, d.cache.v_pages)):
        new[ids] = x[old]
    for new, x in zip(order, (d.cache.order_codes, d.cache.order_idx)):
        new[:, ids] = x[:, old]
    c = ZetaCache(*big, *order, w.N, w.C, w.k, w.bits)
    table = torch.full((1, 17), -1, dtype=torch.int32, device="cuda")
    table[0, :16] = ids.int()
    out, rs, idx = d.outputs()
    c.attend_tree(d.q, d.k, d.v, d.gamma, d.start, d.count, d.parent, table, out, rs, idx=idx)
    acc = d.ints([0])
    c.accept(d.k, d.v, d.start, d.count, d.parent, d.ints([10]), table, acc)
    assert int(c.status.item()) == 0
    for a, b in zip((out, rs, idx), want):
        assert torch.equal(a, b)
    path = line(d.parents[0], 10)
    e = 700 + torch.arange(len(path), device="cuda")
    assert acc.tolist() == [len(path)]
    assert torch.equal(big[1][ids[e // 64], :, e % 64], d.v[0][:, path].transpose(0, 1))


# ------------------------------------------------------------------ accept ---

@pytest.mark.parametrize("kw,page", [(dict(), 16), (dict(v_dtype="f32"), 1),
                                     (dict(d_V=33, v_dtype="f32"), 64), (dict(d_V=250), 16),
                                     (dict(d_V=1, d_K=8, bits=8), 16),
                                     (dict(d_V=256, v_dtype="f32", H=1), 8)],
                         ids=lambda x: str(x) if isinstance(x, int) else _name(x))
@pytest.mark.parametrize("kind", ["tree", "chain", "star"])
def test_accept(kw, page, kind):
    """Lines of every length, cut at the chunk's end; every other row of the pools stays."""
    w = _work(**{**dict(B=6, C=64), **kw})
    n = 50
    d = Drafting(w, page, [100, 120, 0, 63, 64, 300], [n, n, 30, 5, 0, 1], n, kind=kind)
    kp, vp = d.cache.k_pages.clone(), d.cache.v_pages.clone()
    leaf = [n - 1, n - 1, -1, 4, 7, 0]
    want_path = np.full((6, n), -1)
    for b, t in enumerate(leaf):
        nodes = line(d.parents[b], t) if d.counts[b] else []
        for j, u in enumerate(nodes[:w.C - d.starts[b] % w.C]):
            i = d.starts[b] + j
            kp[d.table_np[b][i // page], :, i % page] = d.k[b, :, u]
            vp[d.table_np[b][i // page], :, i % page] = d.v[b, :, u]
            want_path[b, j] = u
    for _ in range(2):                               # a second time changes nothing
        acc, path = d.ints([9] * 6), d.ints(np.full((6, n), 9))
        d.cache.accept(d.k, d.v, d.start, d.count, d.parent, d.ints(leaf), d.table, acc, path)
        assert int(d.cache.status.item()) == 0
        assert acc.tolist() == (want_path >= 0).sum(1).tolist()
        assert np.array_equal(path.cpu().numpy(), want_path)
        assert torch.equal(kp, d.cache.k_pages) and torch.equal(vp, d.cache.v_pages)
    assert acc.tolist()[2] == 0 and (kind != "chain" or acc.tolist()[1] == 8)


@pytest.mark.parametrize("n", [1, 1024])
def test_accept_many_nodes(n):
    w = _work(B=2, C=2048, N=4096)
    d = Drafting(w, 64, [2048 + 100, 2048 - 200], [n, n], n, kind="chain")
    acc, path = d.ints([9] * 2), d.ints(np.full((2, n), 9))
    d.cache.accept(d.k, d.v, d.start, d.count, d.parent, d.ints([n - 1] * 2), d.table, acc, path)
    assert int(d.cache.status.item()) == 0
    for b, m in enumerate((n, min(n, 200))):
        assert acc[b] == m and path[b, :m].tolist() == list(range(m)) and (path[b, m:] == -1).all()
        e = d.starts[b] + torch.arange(m, device="cuda")
        got = d.cache.v_pages[d.table[b].long()[e // 64], :, e % 64]
        assert torch.equal(got, d.v[b, :, :m].transpose(0, 1))


@pytest.mark.parametrize("leaf", [-2, 5, 2 ** 31 - 1, -2 ** 31])
def test_bad_leaves_accept_nothing(leaf):
    d = Drafting(_work(B=2), 16, [100, 200], [5, 5], 8)
    before = d.cache.v_pages.clone()
    acc, path = d.ints([9, 9]), d.ints(np.full((2, 8), 9))
    d.cache.accept(d.k, d.v, d.start, d.count, d.parent, d.ints([leaf, -1]), d.table, acc, path)
    assert int(d.cache.status.item()) == 6
    assert acc.tolist() == [0, 0] and (path == -1).all()
    assert torch.equal(before, d.cache.v_pages)


def test_accept_into_a_missing_page_skips_its_rows():
    d = Drafting(_work(B=1), 16, [70], [20], 20, kind="chain")
    d.table[0, 5] = -1                               # tokens 80..95
    before = d.cache.v_pages.clone()
    acc = d.ints([0])
    d.cache.accept(d.k, d.v, d.start, d.count, d.parent, d.ints([19]), d.table, acc)
    assert int(d.cache.status.item()) == 6 and acc.tolist() == [20]
    p = int(d.table_np[0][4])
    before[p, :, 6:] = d.v[0, :, :10]                # tokens 70..79
    assert torch.equal(before, d.cache.v_pages)


# ----------------------------------------------------------------- reserve ---

def _pool_cache(pages, page, N, C=64, H=1):
    return ZetaCache.empty(pages, page, H, 1, 8, N, C, 1, 8, order_pages=1)


class Lists:
    """Tables and a list on both sides."""

    def __init__(self, B, page, pages, N, seed, width=None):
        rng = np.random.default_rng(seed)
        self.page, self.pages, self.N = page, pages, N
        self.table = np.full((B, width or -(-N // page)), -1, np.int64)
        self.held, self.free, self.F = np.zeros(B, np.int64), rng.permutation(pages), pages
        up = Drafting.ints
        self.d = [up(self.table), up(self.held), up(self.free), up([self.F])]

    def step(self, cache, start, count, n, slots=True, status=0):
        B = len(self.held)
        granted, want, self.F = reserve_plain(self.table, self.held, self.free, self.F, start,
                                              count, n, self.page, self.pages, self.N)
        up = Drafting.ints
        g, s = up([99] * B), up(np.full((B, n), 99))
        cache.reserve(up(start), up(count), *self.d, g, s if slots else None, n=n)
        assert int(cache.status.item()) == status
        for a, b in zip(self.d, (self.table, self.held, self.free, [self.F])):
            assert np.array_equal(a.cpu().numpy(), b)
        assert np.array_equal(g.cpu().numpy(), granted)
        if slots:
            assert np.array_equal(s.cpu().numpy(), want)
        return granted


@pytest.mark.parametrize("B,page,pages,N,n", [(1, 16, 8, 128, 5), (7, 4, 50, 64, 20),
                                              (64, 1, 1500, 64, 64), (300, 64, 700, 1024, 64),
                                              (1000, 16, 5000, 320, 1), (5000, 2, 40000, 64, 3),
                                              (9, 256, 500, 65536, 64)])
def test_reserve_over_many_steps(B, page, pages, N, n):
    rng = np.random.default_rng(B)
    cache, x = _pool_cache(pages, page, N), Lists(B, page, pages, N, 3)
    length = np.zeros(B, np.int64)
    refused = 0
    for i in range(12):
        length[rng.random(B) < 0.2] = 0              # ended
        jump = rng.random(B) < 0.3                   # a request with many tokens already
        length[jump] = rng.integers(0, N + 1, jump.sum())
        count = np.minimum(rng.integers(0, n + 1, B), N - length)
        granted = x.step(cache, length, count, n, slots=i % 3 < 2)
        refused += int((granted < count).sum())
        short = (granted < count) | (x.held * page < length)
        length = np.where(short, np.minimum(length, x.held * page), length + granted)
    assert refused > 0 or B == 1


def test_a_step_taken_back_restores_the_list():
    x = Lists(33, 8, 900, 512, 5)
    cache = _pool_cache(900, 8, 512)
    rng = np.random.default_rng(2)
    start = rng.integers(0, 200, 33)
    x.step(cache, start, 0 * start, 64)
    before = [t.clone() for t in x.d]
    x.step(cache, np.where(np.arange(33) % 4 == 0, 0, start), 50 * (np.arange(33) % 4 > 0), 64)
    assert not torch.equal(before[0], x.d[0])
    x.step(cache, start, 0 * start, 64)
    for i in (0, 1, 3):
        assert torch.equal(before[i], x.d[i])
    assert torch.equal(before[2][:x.F], x.d[2][:x.F])


def test_reserve_lets_granted_be_the_count():
    cache = _pool_cache(10, 4, 64)
    up = Drafting.ints
    table, held = up(np.full((3, 16), -1)), up([0, 0, 0])
    free, fc = up(np.arange(10)), up([10])
    count = up([20, 30, 8])
    cache.reserve(up([0, 0, 0]), count, table, held, free, fc, count, n=30)
    assert count.tolist() == [20, 0, 0] and held.tolist() == [5, 0, 0] and fc.tolist() == [5]
    assert table[0, :6].tolist() == [9, 8, 7, 6, 5, -1] and (table[1:] == -1).all()


@pytest.mark.parametrize("start,count,held", [(-1, 1, 0), (60, 5, 0), (0, 6, 0), (0, -1, 0),
                                              (4, 1, -1), (4, 1, 17), (2 ** 31 - 1, 1, 0)])
def test_reserve_skips_bad_lengths(start, count, held):
    x, cache = Lists(3, 4, 40, 64, 1), _pool_cache(40, 4, 64)
    x.held[1] = held
    x.d[1][1] = held
    x.step(cache, np.array([3, start, 9]), np.array([5, count, 5]), 5, status=6)


@pytest.mark.parametrize("F", [-1, 39, 41, 2 ** 31 - 1])
def test_reserve_refuses_a_list_that_cannot_be(F):
    """More free places than there are pages, counting those that come back: nothing changes."""
    x, cache = Lists(3, 4, 40, 64, 1), _pool_cache(40, 4, 64)
    x.step(cache, np.array([20, 3, 0]), np.array([5, 5, 0]), 5)
    x.F = F
    x.d[3][0] = F
    granted = x.step(cache, np.array([0, 10, 0]), np.array([0, 1, 1]), 5, status=6)
    assert not granted.any() and x.held.tolist() == [7, 2, 0]


def test_reserve_passes_bad_page_numbers_on():
    cache = _pool_cache(8, 4, 64)
    up = Drafting.ints
    table, held = up(np.full((1, 16), -1)), up([0])
    free, fc, g, s = up([1, 2, 77, -5, 3, 0, 0, 0]), up([5]), up([0]), up(np.zeros((1, 16)))
    cache.reserve(up([0]), up([16]), table, held, free, fc, g, s)
    assert int(cache.status.item()) == 6 and fc.tolist() == [1] and g.tolist() == [16]
    assert table[0, :4].tolist() == [3, -5, 77, 2]
    assert s[0].tolist() == [12, 13, 14, 15] + [-1] * 8 + [8, 9, 10, 11]


# ---------------------------------------------------------------- together ---

@pytest.mark.parametrize("v_dtype,weight", [("bf16", "cauchy"), ("f32", "softmax")])
def test_drafting_steps_write_a_text(v_dtype, weight):
    """Texts written by drafting: every step reserves pages, tries a tree in which the true
    continuation is one branch, accepts as much of it as was guessed, completes chunks; the
    accepted nodes' outputs are those of the whole text, and so are the pages afterwards."""
    w = _work(B=5, H=2, N=256, C=32, k=12, v_dtype=v_dtype)
    n, page = 11, 16
    d = Drafting(w, page, [0] * 5, [0] * 5, n, weight)         # texts, codes, an empty cache
    rng = np.random.default_rng(4)
    full_k = torch.from_numpy(d.g["k"]).cuda()
    full_q = torch.from_numpy(d.g["q"]).cuda()
    full_v = torch.from_numpy(np.stack(d.values).astype(np.float32)).cuda().to(d.vdt)
    pages = d.pages
    table, held = d.ints(np.full((5, w.N // page), -1)), d.ints([0] * 5)
    free, fc = d.ints(rng.permutation(pages)), d.ints([pages])
    at = np.zeros(5, np.int64)
    checked = 0
    for step in range(200):
        if (at >= w.N - n).all():
            break
        count = np.where(at < w.N - n, rng.integers(0, n + 1, 5), 0)
        par, true = np.full((5, n), 99), [[] for _ in range(5)]
        for b in range(5):
            p = tree(rng, count[b], "tree")
            par[b, :count[b]] = p
            if count[b]:
                true[b] = line(p, int(rng.integers(0, count[b])))
        q, k = (torch.rand(5, w.H, n, w.d_K, device="cuda") * 2 - 1 for _ in range(2))
        v = torch.randn(5, w.H, n, w.d_V, device="cuda").to(d.vdt)
        for b in range(5):
            for j, t in enumerate(true[b]):
                for x, y in ((q, full_q), (k, full_k), (v, full_v)):
                    x[b, :, t] = y[b, :, at[b] + j]
        start, cnt, parent = d.ints(at), d.ints(count), d.ints(par)
        leaf = d.ints([x[-1] if x else -1 for x in true])
        out, rs, idx = d.outputs()
        acc, path, granted = d.ints([0] * 5), d.ints(np.zeros((5, n))), d.ints([0] * 5)
        c = d.cache
        c.reserve(start, cnt, table, held, free, fc, granted, n=n)
        c.attend_tree(q, k, v, d.gamma, start, granted, parent, table, out, rs, idx=idx)
        c.accept(k, v, start, granted, parent, leaf, table, acc, path)
        c.order(start, acc, table, n=n)
        assert int(c.status.item()) == 0 and granted.tolist() == count.tolist()
        for b in range(5):
            m = int(acc[b])
            assert m == min(len(true[b]), w.C - at[b] % w.C if true[b] else 0)
            for j in range(m):
                i, t, h = int(at[b]) + j, true[b][j], j % w.H
                d.parents[b], d.starts[b] = [-1], i
                d.qn[b, h, 0], d.kn[b, h, 0] = d.g["q"][b, h, i], d.g["k"][b, h, i]
                d.vn[b, h, 0] = d.values[b][h][i]
                win, o, s, bo, bs = d.plain(b, 0, h)
                assert np.array_equal(idx[b, h, t].cpu().numpy(), win if len(win) else [-1] * w.k)
                assert (np.abs(out[b, h, t].double().cpu().numpy() - o) <= bo).all()
                assert abs(float(rs[b, h, t]) - s) <= bs
                checked += 1
            at[b] += m
        c.reserve(d.ints(at), d.ints([0] * 5), table, held, free, fc, granted, n=n)
        assert held.tolist() == (-(-at // page)).tolist()
    assert checked > 500 and (at >= w.N - n).all()
    for b in range(5):
        e = torch.arange(int(at[b]), device="cuda")
        ids = table[b].long()[e // page]
        assert torch.equal(d.cache.k_pages[ids, :, e % page], full_k[b, :, e].transpose(0, 1))
        assert torch.equal(d.cache.v_pages[ids, :, e % page], full_v[b, :, e].transpose(0, 1))
    # pages: none lost, none twice
    used = sum((table[b, :int(held[b])].tolist() for b in range(5)), [])
    assert sorted(used + free[:int(fc)].tolist()) == list(range(pages))


def test_captured_steps_equal_eager_ones():
    """One captured step, replayed with other lengths (in the same chunks), trees and lists in
    the same buffers."""
    w = _work(B=40, H=4, N=1024, C=128, k=24)
    n = 20
    rng = np.random.default_rng(0)
    d = Drafting(w, 64, rng.integers(0, w.N - n, 40), rng.integers(0, n + 1, 40), n)
    other = np.minimum(np.array(d.starts) // w.C * w.C + rng.integers(0, w.C, 40), w.N - n)
    e = Drafting(w, 64, other, rng.integers(0, n + 1, 40), n, seed=5)
    e.table.copy_(d.table)
    leaf = d.ints(np.zeros(40))
    lists = [d.ints(np.full((40, 17), -1)), d.ints([0] * 40), d.ints(np.arange(d.pages)),
             d.ints([d.pages])]

    def step(x, outs, acc, path, lists, granted, slots):
        c = d.cache
        c.reserve(x.start, x.count, *lists, granted, slots)
        c.attend_tree(x.q, x.k, x.v, x.gamma, x.start, x.count, x.parent, x.table, outs[0],
                      outs[1], idx=outs[2])
        c.accept(x.k, x.v, x.start, x.count, x.parent, leaf, x.table, acc, path)

    def fresh():
        return (d.outputs(), d.ints([9] * 40), d.ints(np.zeros((40, n))),
                [x.clone() for x in lists], d.ints([0] * 40), d.ints(np.zeros((40, n))))

    kept = [x.clone() for x in (d.cache.k_pages, d.cache.v_pages)]

    def eager(x):
        for a, b in zip((d.cache.k_pages, d.cache.v_pages), kept):
            a.copy_(b)
        got = fresh()
        step(x, *got)
        return [*got[0], *got[1:3], *got[3], *got[4:], d.cache.k_pages.clone(),
                d.cache.v_pages.clone()]

    want = [eager(x) for x in (d, e)]
    got = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(d, *got)
    first = [x.clone() for x in (d.start, d.count, d.parent, d.q, d.k, d.v)]
    for i, x in enumerate((e, None, e)):
        new = (x.start, x.count, x.parent, x.q, x.k, x.v) if x else first
        for a, b in zip((d.start, d.count, d.parent, d.q, d.k, d.v), new):
            a.copy_(b)
        for a, b in zip((d.cache.k_pages, d.cache.v_pages), kept):
            a.copy_(b)
        clean = fresh()
        for a, b in zip([*got[0], *got[1:3], *got[3], *got[4:]],
                        [*clean[0], *clean[1:3], *clean[3], *clean[4:]]):
            a.copy_(b)
        graph.replay()
        flat = [*got[0], *got[1:3], *got[3], *got[4:], d.cache.k_pages, d.cache.v_pages]
        for a, b in zip(flat, want[0] if x is None else want[1]):
            assert torch.equal(a, b), i
    assert int(d.cache.status.item()) == 0


def test_two_streams_at_once():
    w = _work(B=8, H=4, N=1024, C=256, k=24)
    x = [Drafting(w, 64, np.arange(8) * 100 + 60, [16] * 8, 16, seed=i) for i in range(2)]
    want = [[t.clone() for t in y.attend()] for y in x]
    outs = [y.outputs() for y in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for y, o, s in zip(x, outs, streams):
            y.cache.attend_tree(y.q, y.k, y.v, y.gamma, y.start, y.count, y.parent, y.table, o[0],
                                o[1], idx=o[2], stream=s)
    torch.cuda.synchronize()
    for o, a in zip(outs, want):
        assert all(torch.equal(p, q) for p, q in zip(o, a))


def test_same_bits_each_run():
    w = _work(B=16, H=8, N=2048, C=512, k=48)
    d = Drafting(w, 64, np.arange(16) * 120 + 30, [24] * 16, 24)
    want = [x.clone() for x in d.attend()]
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(want, d.attend()))


def test_refused_arguments():
    w = _work(B=2)
    d = Drafting(w, 16, [100, 200], [5, 5], 5)
    out, rs, idx = d.outputs()
    c, leaf, acc = d.cache, d.ints([0, 0]), d.ints([0, 0])

    def tree_call(**kw):
        a = dict(q=d.q, k=d.k, v=d.v, gamma=d.gamma, start=d.start, count=d.count,
                 parent=d.parent, page_table=d.table, out=out, rowsum=rs)
        c.attend_tree(**{**a, **kw})

    def accept_call(**kw):
        a = dict(k=d.k, v=d.v, start=d.start, count=d.count, parent=d.parent, leaf=leaf,
                 page_table=d.table, accepted=acc)
        c.accept(**{**a, **kw})

    lists = Lists(2, 16, d.pages, w.N, 0)
    table, held, free, fc = lists.d

    def reserve_call(**kw):
        a = dict(start=d.start, count=d.count, page_table=table, held=held, free=free,
                 free_count=fc, granted=acc)
        c.reserve(**{**a, **kw})

    for call in (tree_call, accept_call):
        for bad in (d.parent[:, :4], d.parent[:1], d.parent.t().contiguous().t(), d.parent.cpu()):
            with pytest.raises(ValueError):
                call(parent=bad)
        for bad in (d.parent.long(), d.parent.float()):
            with pytest.raises(TypeError):
                call(parent=bad)
        with pytest.raises(ValueError):
            call(k=d.k[:, :, :4])
        with pytest.raises(ValueError):
            call(k=d.k.clone().requires_grad_())
        with pytest.raises(TypeError):
            call(v=d.v.float())
        with pytest.raises(ValueError):
            call(start=d.start[:1])
    with pytest.raises(ValueError):
        tree_call(q=d.q[0])
    with pytest.raises(ValueError):
        tree_call(out=out.transpose(1, 2))
    with pytest.raises(TypeError):
        tree_call(idx=idx.long())
    with pytest.raises(ValueError):
        accept_call(path=d.ints([0, 0]))
    with pytest.raises(ValueError):
        accept_call(leaf=leaf[:1])
    with pytest.raises(ValueError):
        reserve_call(free=free[:-1])
    with pytest.raises(ValueError):
        reserve_call(slots=d.ints(np.zeros((3, 5))))
    with pytest.raises(TypeError):
        reserve_call(held=held.long())
    with pytest.raises(ValueError):
        reserve_call(free_count=d.ints([0, 0]))
    with pytest.raises(ZetaError) as err:
        reserve_call(n=w.C + 1)
    assert err.value.code == 2
    big = _work(B=1, C=2048, N=2048)
    with pytest.raises(ZetaError) as err:
        cc = ZetaCache.empty(40, 64, 2, 3, 64, 2048, 2048, 16)
        z = torch.zeros(1, 2, 1025, 3, device="cuda")
        vv = torch.zeros(1, 2, 1025, 64, dtype=torch.bfloat16, device="cuda")
        cc.attend_tree(z, z, vv, d.gamma, d.ints([0]), d.ints([1]), d.ints(np.zeros((1, 1025))),
                       d.ints(np.zeros((1, 32))), vv.clone(), z[..., 0].contiguous())
    assert err.value.code == 2 and big.C == 2048
    torch.cuda.synchronize()
    assert (out == PAD).all()


def test_the_binding_runs_the_same_calls():
    w = _work(B=2)
    d = Drafting(w, 16, [100, 200], [5, 5], 5)
    want = [x.clone() for x in d.attend()]
    c = d.cache
    p = zb.problem(w.B, w.H, w.N, w.d_K, w.d_V, w.k, w.C, w.bits, w.v_dtype)
    cc = zb.zeta_cache_t(5, 16, c.pages, c.order_pages, d.table.shape[1])
    out, rs, idx = d.outputs()
    zb.zeta_cache_attend_tree(p, cc, d.q, d.k, d.v, d.gamma, d.start, d.count, d.parent, d.table,
                              c.k_pages, c.v_pages, d.table, c.order_codes, c.order_idx, out, rs,
                              idx)
    assert all(torch.equal(a, b) for a, b in zip(want, (out, rs, idx)))
    leaf, acc, acc2 = d.ints([4, 3]), d.ints([0, 0]), d.ints([0, 0])
    zb.zeta_cache_accept(p, cc, d.k, d.v, d.start, d.count, d.parent, leaf, d.table, c.k_pages,
                         c.v_pages, acc)
    pages = [c.k_pages.clone(), c.v_pages.clone()]
    c.accept(d.k, d.v, d.start, d.count, d.parent, leaf, d.table, acc2)
    assert torch.equal(acc, acc2) and acc.min() > 0
    assert torch.equal(pages[0], c.k_pages) and torch.equal(pages[1], c.v_pages)
    x = [Lists(2, 16, c.pages, w.N, 0).d for _ in range(2)]
    width = x[0][0].shape[1]
    cc = zb.zeta_cache_t(5, 16, c.pages, c.order_pages, width)
    zb.zeta_cache_reserve(p, cc, d.start, d.count, *x[0], acc)
    c.reserve(d.start, d.count, *x[1], acc2, n=5)
    assert torch.equal(acc, acc2) and all(torch.equal(a, b) for a, b in zip(*x))


def test_empty_calls():
    w = _work(B=2)
    d = Drafting(w, 16, [100, 200], [0, 0], 1)
    c, e = d.cache, torch.empty
    i32 = dict(dtype=torch.int32, device="cuda")
    none, table = e(0, **i32), e(0, d.table.shape[1], **i32)
    z, vv = e(0, w.H, 3, 3, device="cuda"), e(0, w.H, 3, 64, dtype=torch.bfloat16, device="cuda")
    c.attend_tree(z, z, vv, d.gamma, none, none, e(0, 3, **i32), table, vv, z[..., 0].contiguous())
    c.accept(z, vv, none, none, e(0, 3, **i32), none, table, none)
    free, fc = d.ints(np.arange(d.pages)), d.ints([d.pages])
    c.reserve(none, none, table, none, free, fc, none)
    d.attend()                                        # sequences without drafts
    d.check()
    assert fc.tolist() == [d.pages]
