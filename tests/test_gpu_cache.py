"""GPU tests of the paged-cache calls (append, order, attend) against their plain
64-bit forms: selections bit for bit, sums within bounds counted from the
roundings (tests/cache_util.py)."""
import numpy as np
import pytest
import torch

from order_retrieval_gb300 import ZetaCache, ZetaError, zeta_attention
from order_retrieval_gb300 import binding as zb
from order_retrieval_gb300 import workloads as W

from cache_util import EPS, Sequence, window
from gpu_util import in_threads

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]

PAD = 7.0          # what padding rows hold before and after


class Serving:
    """Sequences of one workload read through a cache in steps of given counts."""

    def __init__(self, w, page, weight="cauchy", seed=0, shuffle=True, spare=3, split_tables=False):
        self.w, self.page, self.weight = w, page, weight
        g = W.generate(w)
        self.vdt = torch.bfloat16 if w.v_dtype == "bf16" else torch.float32
        vt = torch.from_numpy(np.ascontiguousarray(g["v"]))
        self.q = torch.from_numpy(g["q"]).cuda()
        self.k = torch.from_numpy(g["k"]).cuda()
        self.v = (vt.view(torch.bfloat16) if w.v_dtype == "bf16" else vt).cuda()
        self.gamma = torch.from_numpy(g["gamma"]).cuda()
        self.seqs = [Sequence(g["q"][b], g["k"][b], W.values_f64(w, g["v"][b]), w.C, w.k, w.bits,
                              g["gamma"], weight) for b in range(w.B)]
        per = -(-w.N // page)
        rng = np.random.default_rng(seed)

        def tables():
            ids = np.arange(w.B * per + spare)
            if shuffle:
                rng.shuffle(ids)
            t = np.full((w.B, per + 1), -1, np.int32)      # one entry nobody reads
            t[:, :per] = ids[:w.B * per].reshape(w.B, per)
            return t

        self.table_np = tables()
        self.otable_np = tables() if split_tables else self.table_np
        self.table = torch.from_numpy(self.table_np).cuda()
        self.otable = torch.from_numpy(self.otable_np).cuda() if split_tables else None
        self.pages = w.B * per + spare
        self.cache = ZetaCache.empty(self.pages, page, w.H, w.d_K, w.d_V, w.N, w.C, w.k, w.bits,
                                     self.vdt, weight)
        self.len = np.zeros(w.B, np.int64)
        self.got = [dict() for _ in range(w.B)]            # position -> (idx, out, rowsum) [H, ...]

    def batch(self, counts, n):
        """start, count and padded k, v, q of the next tokens; padding is NaN."""
        w = self.w
        start = torch.from_numpy(self.len.astype(np.int32)).cuda()
        count = torch.tensor(counts, dtype=torch.int32).cuda()

        def rows(x):
            r = torch.full((w.B, w.H, n, x.shape[-1]), float("nan"), dtype=x.dtype, device="cuda")
            for b, c in enumerate(counts):
                s = int(self.len[b])
                r[b, :, :c] = x[b, :, s:s + c]
            return r

        return start, count, rows(self.q), rows(self.k), rows(self.v)

    def step(self, counts, n=None):
        w = self.w
        n = max(max(counts), 1) if n is None else n
        start, count, q, k, v = self.batch(counts, n)
        out = torch.full((w.B, w.H, n, w.d_V), PAD, dtype=self.vdt, device="cuda")
        rs = torch.full((w.B, w.H, n), PAD, device="cuda")
        idx = torch.full((w.B, w.H, n, w.k), 77, dtype=torch.int32, device="cuda")
        self.cache.append(k, v, start, count, self.table)
        self.cache.order(start, count, self.table, self.otable)
        self.cache.attend(q, self.gamma, start, count, self.table, out, rs, self.otable, idx)
        assert int(self.cache.status.item()) == 0
        for b, c in enumerate(counts):
            assert (out[b, :, c:] == PAD).all() and (rs[b, :, c:] == PAD).all()
            assert (idx[b, :, c:] == 77).all()
            o, r, i = out[b].double().cpu().numpy(), rs[b].cpu().numpy(), idx[b].cpu().numpy()
            for t in range(c):
                self.got[b][int(self.len[b]) + t] = (i[:, t], o[:, t], r[:, t])
            self.len[b] += c

    def check(self, rows=None, heads=None):
        """Every collected row (or the positions in rows, of the given heads) against the
        plain form."""
        w = self.w
        half_w, half_out = (2.0 ** -8, 2.0 ** -8) if w.v_dtype == "bf16" else (0.0, EPS)

        def one(bi):
            b, i = bi
            idx, out, rs = self.got[b][i]
            for h in range(w.H) if heads is None else heads:
                win, o, s, bo, bs = self.seqs[b].row(h, i, half_w, half_out)
                want = win if len(win) else np.full(w.k, -1)
                assert np.array_equal(idx[h], want), (b, h, i)
                assert (np.abs(out[h] - o) <= bo).all(), (b, h, i, np.abs(out[h] - o).max())
                assert abs(rs[h] - s) <= bs, (b, h, i, rs[h], s)

        todo = [(b, i) for b in range(w.B) for i in self.got[b] if rows is None or i in rows]
        assert todo
        in_threads(one, todo)

    def check_order(self):
        """The latest prefixes in the order pools, entry by entry; both planes where
        two chunks are complete."""
        w = self.w
        codes = self.cache.order_codes.cpu().numpy()
        codes = codes.view(np.uint32 if codes.dtype == np.int32 else np.uint64).astype(np.uint64)
        idx = self.cache.order_idx.cpu().numpy()
        for b in range(w.B):
            top = int(self.len[b]) // w.C
            for c in {top, top - 1} - {0, -1}:
                e = np.arange(c * w.C)
                at = self.otable_np[b][e // self.page], e % self.page
                for h in range(w.H):
                    z, tok = self.seqs[b].prefix(h, c)
                    assert np.array_equal(codes[c & 1, at[0], h, at[1]], z), (b, h, c)
                    assert np.array_equal(idx[c & 1, at[0], h, at[1]], tok), (b, h, c)

    def check_pages(self):
        """Every token in its row; rows of no token still zero."""
        w = self.w
        kp = torch.zeros_like(self.cache.k_pages)
        vp = torch.zeros_like(self.cache.v_pages)
        for b in range(w.B):
            m = int(self.len[b])
            e = torch.arange(m, device="cuda")
            ids, off = self.table[b].long()[e // self.page], e % self.page
            kp[ids, :, off] = self.k[b, :, :m].transpose(0, 1)
            vp[ids, :, off] = self.v[b, :, :m].transpose(0, 1)
        assert torch.equal(kp, self.cache.k_pages) and torch.equal(vp, self.cache.v_pages)


def _work(**kw):
    base = dict(name="cache", B=2, H=2, N=512, d_K=3, d_V=64, k=16, C=64, bits=10, v_dtype="bf16",
                gamma=(0.5, 1.0), dist="uniform", v_dist="normal", seed=91)
    base.update(kw)
    return W.Workload(**base)


SHAPES = [
    (dict(), 16), (dict(v_dtype="f32"), 16),
    (dict(C=40, N=400, k=7), 16),                          # chunks that end inside pages
    (dict(C=100, N=500, k=33, d_V=40), 32),
    (dict(C=128, k=128, d_V=32, v_dtype="f32"), 8),        # window as long as a chunk
    (dict(d_K=1, bits=21, d_V=128), 64),
    (dict(d_K=2, bits=21, v_dtype="f32", d_V=128), 1),     # one token per page
    (dict(d_K=4, bits=8, d_V=96), 256),                    # 32-bit codes to the top bit
    (dict(d_K=8, bits=8, d_V=256, H=1), 512),              # 64-bit codes to the top bit
    (dict(d_K=5, bits=12, d_V=256, v_dtype="f32", H=1), 16),
    (dict(d_V=1), 16), (dict(d_V=33, v_dtype="f32"), 16), (dict(d_V=250, H=1), 16),
    (dict(bits=1), 16),                                    # eight codes, all ties
    (dict(dist="clusters", bits=12, H=5), 32),
    (dict(C=1, N=96, k=1, H=1), 16), (dict(C=8, N=96, k=3), 16),
    (dict(C=512, N=512), 64),                              # a single chunk: no window at all
]


@pytest.mark.parametrize("kw,page", SHAPES, ids=lambda x: str(x) if isinstance(x, int) else
                         "-".join(f"{a}{b}" for a, b in x.items()) or "base")
def test_pieces_then_tokens(kw, page):
    """Ragged pieces of up to C tokens across chunk ends, then single tokens."""
    w = _work(**kw)
    sv = Serving(w, page)
    rng = np.random.default_rng(3)
    left = np.full(w.B, w.N - 4)
    while left.any():
        c = [int(min(m, rng.choice([0, w.C, rng.integers(0, w.C + 1)]))) for m in left]
        left -= np.array(c)
        sv.step(c, n=w.C if rng.random() < 0.3 else None)
    sv.check_order()
    for _ in range(4):
        sv.step([1] * w.B)
    sv.check_order()
    sv.check_pages()
    sv.check()


# Pieces large enough for the tile kernel, 32 rows a block (5 sequences of 2 heads) and 64
# (of 8 heads); blocks of 16 are in test_gpu_cache_blocks.py.
TILES = [
    dict(), dict(H=8), dict(d_V=40), dict(d_V=96, k=65), dict(d_V=128, H=8, k=100),
    dict(d_K=1, bits=21, d_V=32), dict(d_K=2, bits=21, H=8), dict(d_K=4, bits=8, d_V=128),
    dict(bits=1, H=8), dict(dist="clusters", bits=12, H=8), dict(C=500, N=2000, H=8, k=33),
    dict(C=500, N=2000, k=7), dict(k=130, H=8), dict(N=20480, H=8, B=5, k=16),
]


@pytest.mark.parametrize("weight", ["cauchy", "softmax", "inv_euclid"])
@pytest.mark.parametrize("kw", TILES, ids=lambda x: "-".join(f"{a}{b}" for a, b in x.items())
                         or "base")
def test_large_pieces(kw, weight):
    """The first pieces (no window), pieces across chunk ends of unequal length with an
    idle sequence, whole pieces; rows of every kind against the plain form."""
    w = _work(**{**dict(B=5, N=2048, C=512, k=24, gamma=(0.3, 1.0)), **kw})
    sv = Serving(w, 64, weight)
    stop = w.N - 3 * w.C
    while sv.len[0] < stop:                              # up to the last four chunks
        sv.got = [dict() for _ in range(w.B)]
        sv.step([w.C] * w.B)
    c = w.C
    sv.step([c, c - 100, 17, 0, c - 1], n=c)
    sv.step([c, c, c - 60, 90, 1], n=c)
    sv.step([c] * 4 + [c - 3], n=c)
    sv.check_order()
    rng = np.random.default_rng(11)
    first = stop - c
    rows = set(rng.integers(first, w.N, 60).tolist()) | {first, stop, stop + c - 1, stop + c}
    sv.check(rows, heads=(0, w.H - 1))


@pytest.mark.parametrize("H", [2, 8])
def test_large_pieces_with_values_that_are_not_finite(H):
    """Infinities and NaN in later tokens of the own chunk and in keys of other rows'
    windows reach only the rows that attend to them."""
    w = _work(B=5, H=H, N=1536, C=512, k=24)
    sv = Serving(w, 64)
    bad = {0: 700, 1: 1200, 2: 100}                       # sequence: token
    for b, t in bad.items():
        sv.v[b, :, t] = float("inf") if b else float("nan")
    plain = sv.v.clone()
    for _ in range(3):
        sv.step([512] * 5, n=512)
    for b, t in bad.items():
        for i in range(0, w.N, 7):
            win, o, r = (x[0] for x in sv.got[b][i])
            sees = t in win.tolist() or (t // 512 == i // 512 and t <= i)
            assert np.isfinite(o).all() != sees, (b, i)
            assert np.isfinite(r)
    # finite rows are what they would be with any other value there
    sv.seqs = [Sequence(s.q, s.k, np.nan_to_num(s.v, nan=0.0, posinf=0.0), s.C, s.ksel, w.bits,
                        s.gamma, "cauchy") for s in sv.seqs]
    for b, t in bad.items():
        sv.got[b] = {i: x for i, x in sv.got[b].items() if np.isfinite(x[1]).all()}
    sv.check(set(range(0, w.N, 11)), heads=(0, H - 1))
    assert torch.equal(plain.nan_to_num(), sv.v.nan_to_num())


@pytest.mark.parametrize("weight", ["softmax", "inv_euclid"])
@pytest.mark.parametrize("v_dtype,d_V", [("bf16", 64), ("f32", 64), ("bf16", 24)])
def test_weight_kernels(weight, v_dtype, d_V):
    w = _work(v_dtype=v_dtype, d_V=d_V, C=96, N=480, k=20, dist="clusters")
    sv = Serving(w, 32, weight)
    while sv.len.min() < w.N - 2:
        sv.step([min(w.C, w.N - 2 - int(m)) for m in sv.len])
    sv.step([1, 1])
    sv.step([1, 0])
    sv.check()


@pytest.mark.parametrize("B", [1, 3, 160])
@pytest.mark.parametrize("v_dtype", ["bf16", "f32"])
def test_single_tokens_from_the_first(B, v_dtype):
    """Decoding from an empty cache, one token per call, for batches that split a
    token over a cluster and batches that do not; the sequences drift apart."""
    w = _work(B=B, N=96, C=32, k=9, v_dtype=v_dtype, d_V=64 if v_dtype == "bf16" else 24)
    sv = Serving(w, 16)
    for t in range(70):
        sv.step([1 if (b + t) % 7 else 0 for b in range(B)], n=1)
    sv.check_order()
    sv.check_pages()
    sv.check(rows=None if B < 10 else {0, 31, 32, 33, 50, 58})


@pytest.mark.parametrize("n,H", [(1, 2), (5, 2), (64, 2), (200, 2), (1024, 2), (1024, 5)])
def test_long_context(n, H):
    """The efficiency workload's shape, chunks of 1024 and windows of 64, the call's
    last rows against the plain form."""
    w = W.EFFICIENCY.replace(name="cache_long", B=1, H=H, N=16384, seed=17)
    sv = Serving(w, 64)
    stop = w.N - n
    while sv.len[0] < stop:
        sv.step([min(w.C, stop - int(sv.len[0]))])
    sv.got = [dict()]
    sv.step([n])
    sv.check_order()
    rows = {w.N - 1, w.N - n} | set(range(w.N - n, w.N, max(1, n // 16)))
    sv.check(rows)


def test_equals_the_training_forward():
    """A prompt read in pieces against the framework's attention of the whole."""
    w = W.CLUSTERED.replace(name="cache_train", B=1, H=4, N=2048)
    sv = Serving(w, 128)
    whole = zeta_attention(sv.q, sv.k, sv.v, sv.gamma, w.C, w.k, w.bits).double().cpu().numpy()
    while sv.len[0] < w.N:
        sv.step([min(200, w.N - int(sv.len[0]))])
    got = np.stack([sv.got[0][i][1] for i in range(w.N)], 1)
    # both round the weights and the result to bf16, each within 2^-8 of sizes <= max |v|
    size = np.abs(sv.seqs[0].v).max()
    assert np.abs(got - whole[0]).max() <= 4 * 2.0 ** -8 * size
    sv.check(set(range(0, w.N, 37)))


@pytest.mark.parametrize("kw", [dict(), dict(v_dtype="f32", d_V=24), dict(d_K=8, bits=8)],
                         ids=["bf16", "f32", "dk8"])
def test_longest_chunks_and_long_prefixes(kw):
    """Chunks of 8192, the longest that are sorted in shared memory, under a prefix of
    more than 65,536 entries; pieces of a chunk, a short piece, a token."""
    w = _work(**{**dict(B=1, H=1, N=81920, C=8192, k=40, seed=5), **kw})
    sv = Serving(w, 256)
    for _ in range(9):
        sv.got = [dict()]
        sv.step([8192])
    sv.step([8000])
    sv.step([100])
    sv.step([1])
    sv.check_order()
    sv.check({73728 - 8192, 73727, 73728, 73728 + 4000, 81727, 81728, 81800, 81828})


@pytest.mark.parametrize("H", [2, 8])
def test_bad_pages_of_large_pieces(H):
    """The tile kernel's share of bad tables: keys on pages out of range are left out of
    the own chunk and of the windows, everything else stays."""
    w = _work(B=5, H=H, N=1536, C=512, k=24)
    sv = Serving(w, 64)
    sv.step([512] * 5)
    start, count, q, k, v = sv.batch([512] * 5, 512)
    sv.cache.append(k, v, start, count, sv.table)
    bad = sv.table.clone()
    bad[0, 3] = -1                             # tokens 192..255: in the prefix
    bad[1, 8] = 10 ** 6                        # tokens 512..575: in the own chunk
    out = torch.full((5, H, 512, 64), PAD, dtype=torch.bfloat16, device="cuda")
    rs = torch.full((5, H, 512), PAD, device="cuda")
    sv.cache.attend(q, sv.gamma, start, count, bad, out, rs, sv.table)
    assert int(sv.cache.status.item()) == 6
    out, rs = out.double().cpu().numpy(), rs.cpu().numpy()
    for b in (0, 1, 2):
        s = sv.seqs[b]
        gone = {0: range(192, 256), 1: range(512, 576), 2: ()}[b]
        for t in (0, 63, 64, 300, 511):
            i = 512 + t
            win = window(s.qc[0, i], s.kc[0], i, w.C, w.k)
            j = np.array([x for x in [*win, *range(512, i + 1)] if x not in gone])
            if len(j) == 0:
                continue
            d2 = ((s.q[0, i].astype(np.float64) - s.k[0][j]) ** 2).sum(1)
            wt = 1 / (1 + d2 / float(s.gamma[0]) ** 2)
            size = (wt @ np.abs(s.v[0][j])) / wt.sum()
            assert abs(rs[b, 0, t] - wt.sum()) <= 1e-5 * wt.sum()
            # weight and result rounded to bf16 once each
            assert (np.abs(out[b, 0, t] - (wt @ s.v[0][j]) / wt.sum()) <= 2.1 * 2.0 ** -8 * size).all()


def test_order_tables_of_their_own_and_shared_prompt_pages():
    """Two sequences share the K/V pages of a common prompt; their prefixes live in
    pages of their own."""
    w = _work(N=256, C=64, k=11, H=3)
    sv = Serving(w, 16, split_tables=True)
    common = 128
    for x in (sv.q, sv.k, sv.v):
        x[1, :, :common] = x[0, :, :common]
    g = {n: getattr(sv, n).float().cpu().numpy() for n in ("q", "k", "v")}
    sv.seqs = [Sequence(g["q"][b], g["k"][b], g["v"][b].astype(np.float64), w.C, w.k, w.bits,
                        sv.gamma.cpu().numpy(), "cauchy") for b in range(2)]
    sv.table_np[1, :common // 16] = sv.table_np[0, :common // 16]
    sv.table = torch.from_numpy(sv.table_np).cuda()
    sv.step([64, 64])
    sv.step([64, 64])
    while sv.len[0] < 250:
        sv.step([13, 1] if sv.len[0] < 235 else [1, 5])
    sv.check_order()
    sv.check()


def test_masked_places_may_hold_anything():
    """NaN and infinities in rows that no query sees: unused pages, rows behind the
    last token, own-chunk keys after the query."""
    w = _work(N=128, C=64, k=8)
    sv = Serving(w, 32)
    sv.cache.k_pages.fill_(float("nan"))
    sv.cache.v_pages.fill_(float("inf"))
    sv.step([60, 3])
    sv.step([11, 40])
    sv.step([20, 0])
    sv.check()


def _small(n=4, B=2):
    w = _work(B=B, N=128, C=32, k=4)
    sv = Serving(w, 16)
    sv.step([32] * B)
    return w, sv, n


def _fresh(w, n):
    return (torch.full((w.B, w.H, n, w.d_V), PAD, dtype=torch.bfloat16, device="cuda"),
            torch.full((w.B, w.H, n), PAD, device="cuda"))


@pytest.mark.parametrize("start,count", [(-1, 1), (128, 1), (126, 3), (40, -1), (40, 5),
                                         (2 ** 31 - 1, 1)])
def test_bad_lengths_skip_the_sequence(start, count):
    w, sv, n = _small()
    before = [x.clone() for x in (sv.cache.k_pages, sv.cache.v_pages, sv.cache.order_codes,
                                  sv.cache.order_idx)]
    st = torch.tensor([start, 32], dtype=torch.int32).cuda()
    ct = torch.tensor([count, 0], dtype=torch.int32).cuda()
    q, k = (torch.zeros(2, w.H, n, 3, device="cuda") for _ in range(2))
    v = torch.ones(2, w.H, n, 64, dtype=torch.bfloat16, device="cuda")
    out, rs = _fresh(w, n)
    for call in (lambda: sv.cache.append(k, v, st, ct, sv.table),
                 lambda: sv.cache.attend(q, sv.gamma, st, ct, sv.table, out, rs)):
        sv.cache.status.zero_()
        call()
        assert int(sv.cache.status.item()) == 6
    if (start, count) != (40, 5):              # order takes any count up to C
        sv.cache.status.zero_()
        sv.cache.order(st, ct, sv.table)
        assert int(sv.cache.status.item()) == 6
    assert (out == PAD).all() and (rs == PAD).all()
    for a, b in zip(before, (sv.cache.k_pages, sv.cache.v_pages, sv.cache.order_codes,
                             sv.cache.order_idx)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("page_id", [-1, 10 ** 6, -2 ** 31])
def test_bad_pages_are_skipped(page_id):
    """A table entry out of range drops its tokens and is reported; everything else
    is as it should be."""
    w, sv, n = _small()
    kp, vp = sv.cache.k_pages.clone(), sv.cache.v_pages.clone()
    bad = sv.table.clone()
    bad[0, 2] = page_id                        # tokens 32..47 of sequence 0
    st = torch.tensor([32, 32], dtype=torch.int32).cuda()
    ct = torch.tensor([n, n], dtype=torch.int32).cuda()
    k = torch.zeros(2, w.H, n, 3, device="cuda")
    v = torch.ones(2, w.H, n, 64, dtype=torch.bfloat16, device="cuda")
    sv.cache.append(k, v, st, ct, bad)
    assert int(sv.cache.status.item()) == 6
    ids = sv.table[1, 2].long()
    kp[ids, :, :n] = 0
    vp[ids, :, :n] = 1
    assert torch.equal(kp, sv.cache.k_pages) and torch.equal(vp, sv.cache.v_pages)
    sv.cache.status.zero_()
    out, rs = _fresh(w, n)
    sv.cache.attend(k, sv.gamma, st, ct, bad, out, rs)     # sequence 0 sees its window only
    assert int(sv.cache.status.item()) == 6
    assert (rs[0] > 0).all() and (rs[0] < w.k + 1e-3).all() and torch.isfinite(out).all()
    sv.cache.status.zero_()
    old = sv.cache.order_idx.clone()
    ct.fill_(32)
    sv.cache.order(st, ct, bad)
    assert int(sv.cache.status.item()) == 6
    own = sv.table[0].long()[:8]
    own = own[own >= 0]
    assert torch.equal(old[:, own], sv.cache.order_idx[:, own])


def test_bad_order_entries_are_dropped():
    """Tokens outside the prefix in the order pool: the key is left out and reported."""
    w, sv, n = _small(n=1)
    sv.cache.order_idx[1] = 10 ** 6
    st = torch.tensor([32, 32], dtype=torch.int32).cuda()
    ct = torch.ones(2, dtype=torch.int32).cuda()
    q = torch.zeros(2, w.H, 1, 3, device="cuda")
    v = torch.ones(2, w.H, 1, 64, dtype=torch.bfloat16, device="cuda")
    sv.cache.append(q, v, st, ct, sv.table)
    out, rs = _fresh(w, 1)
    idx = torch.zeros(2, w.H, 1, w.k, dtype=torch.int32, device="cuda")
    sv.cache.attend(q, sv.gamma, st, ct, sv.table, out, rs, idx=idx)
    assert int(sv.cache.status.item()) == 6
    assert (idx == -1).all() and (rs == 1).all() and (out == 1).all()   # itself alone, at d2 = 0


def test_refused_arguments():
    w, sv, n = _small()
    c = sv.cache
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    q = torch.zeros(2, w.H, n, 3, device="cuda")
    v = torch.zeros(2, w.H, n, 64, dtype=torch.bfloat16, device="cuda")
    out, rs = _fresh(w, n)
    with pytest.raises(TypeError):
        c.append(q.half(), v, st, st, sv.table)
    with pytest.raises(TypeError):
        c.append(q, v.float(), st, st, sv.table)
    with pytest.raises(TypeError):
        c.append(q, v, st.long(), st, sv.table)
    with pytest.raises(ValueError):
        c.append(q, v[:, :, :2], st, st, sv.table)
    with pytest.raises(ValueError):
        c.append(q.transpose(1, 2).contiguous().transpose(1, 2), v, st, st, sv.table)
    with pytest.raises(ValueError):
        c.append(q, v, st.cpu(), st, sv.table)
    with pytest.raises(ValueError):
        c.attend(q.clone().requires_grad_(), sv.gamma, st, st, sv.table, out, rs)
    with pytest.raises(ValueError):
        c.attend(q, sv.gamma[:1], st, st, sv.table, out, rs)
    with pytest.raises(ZetaError) as e:                     # a table too short for N
        c.append(q, v, st, st, sv.table[:, :4].contiguous())
    assert e.value.code == 1
    big = torch.zeros(2, w.H, w.C + 1, 3, device="cuda")
    with pytest.raises(ZetaError) as e:                     # more than C tokens per sequence
        c.append(big, torch.zeros(2, w.H, w.C + 1, 64, dtype=torch.bfloat16, device="cuda"), st,
                 st, sv.table)
    assert e.value.code == 2
    with pytest.raises(ZetaError):                          # a page that is no power of two
        ZetaCache.empty(4, 24, 2, 3, 64, 128, 32, 4).order(st, st, sv.table)
    with pytest.raises(ZetaError):                          # C does not divide N
        ZetaCache.empty(4, 16, 2, 3, 64, 100, 32, 4)
    with torch.no_grad():
        c.attend(q.clone().requires_grad_(), sv.gamma, st, st, sv.table, out, rs)
    assert int(c.status.item()) == 0 and (out == PAD).all()


def test_the_binding_runs_the_same_calls():
    """zeta_cache_* of the binding on the handle's pools: the same outputs, bit for bit."""
    w, sv, n = _small()
    c = sv.cache
    p = c._problem(w.B)
    cc = zb.zeta_cache_t(n, c.page, c.pages, c.order_pages, sv.table.shape[1])
    start, count, q, k, v = sv.batch([n, n - 1], n)
    twin = ZetaCache(c.k_pages.clone(), c.v_pages.clone(), c.order_codes.clone(),
                     c.order_idx.clone(), w.N, w.C, w.k, w.bits)
    out, rs = _fresh(w, n)
    out2, rs2 = _fresh(w, n)
    c.append(k, v, start, count, sv.table)
    c.order(start, count, sv.table)
    c.attend(q, sv.gamma, start, count, sv.table, out, rs)
    zb.zeta_cache_append(p, cc, k, v, start, count, sv.table, twin.k_pages, twin.v_pages)
    zb.zeta_cache_order(p, cc, start, count, sv.table, twin.k_pages, sv.table, twin.order_codes,
                        twin.order_idx)
    zb.zeta_cache_attend(p, cc, q, sv.gamma, start, count, sv.table, twin.k_pages, twin.v_pages,
                         sv.table, twin.order_codes, twin.order_idx, out2, rs2)
    assert torch.equal(c.k_pages, twin.k_pages) and torch.equal(c.v_pages, twin.v_pages)
    assert torch.equal(c.order_codes, twin.order_codes)
    assert torch.equal(out, out2) and torch.equal(rs, rs2)


@pytest.mark.parametrize("B,n,C", [(2, 1, 32), (160, 1, 32), (2, 24, 32), (5, 500, 512)])
def test_captured_steps_equal_eager_ones(B, n, C):
    """One graph of the three calls replayed over many steps, start advanced on the
    device, against eager calls on a second cache; on a stream of its own."""
    w = _work(B=B, N=5 * C, C=C, k=5, H=2)
    one, two = Serving(w, 16), Serving(w, 16)
    st = torch.zeros(B, dtype=torch.int32, device="cuda")
    ct = torch.full((B,), n, dtype=torch.int32, device="cuda")
    bufs = [torch.zeros(B, w.H, n, d, dtype=dt, device="cuda")
            for d, dt in ((3, torch.float32), (3, torch.float32), (64, torch.bfloat16))]
    out, rs = _fresh(w, n)

    def step():
        one.cache.append(bufs[1], bufs[2], st, ct, one.table)
        one.cache.order(st, ct, one.table)
        one.cache.attend(bufs[0], one.gamma, st, ct, one.table, out, rs)
        st.add_(n)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()                                             # warm up; the tokens come again
        st.zero_()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.synchronize()
    st.zero_()
    one.cache.order_idx.zero_()
    for t in range(w.N // n):
        for buf, x in zip(bufs, (one.q, one.k, one.v)):
            buf.copy_(x[:, :, t * n:(t + 1) * n])
        graph.replay()
        two.step([n] * B)
        torch.cuda.synchronize()
        want = np.stack([np.stack([two.got[b][t * n + x][1] for x in range(n)], 1)
                         for b in range(B)])
        assert np.array_equal(out.double().cpu().numpy(), want), t
    assert torch.equal(one.cache.order_idx, two.cache.order_idx)


def test_two_streams_at_once():
    """Calls on different sequences of one cache overlap on two streams."""
    w = _work(B=2, N=256, C=64, k=9)
    sv, ref = Serving(w, 16), Serving(w, 16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        ref.step([50, 50])
    torch.cuda.synchronize()
    outs = []
    for b, s in enumerate(streams):
        with torch.cuda.stream(s):
            got = []
            for t in range(5):
                st = torch.tensor([50 * t], dtype=torch.int32, device="cuda")
                ct = torch.tensor([50], dtype=torch.int32, device="cuda")
                x = [y[b:b + 1, :, 50 * t:50 * t + 50].contiguous() for y in (sv.q, sv.k, sv.v)]
                o = torch.empty(1, w.H, 50, 64, dtype=torch.bfloat16, device="cuda")
                r = torch.empty(1, w.H, 50, device="cuda")
                tb = sv.table[b:b + 1].contiguous()
                sv.cache.append(x[1], x[2], st, ct, tb)
                sv.cache.order(st, ct, tb)
                sv.cache.attend(x[0], sv.gamma, st, ct, tb, o, r)
                got.append(o)
            outs.append(got)
    torch.cuda.synchronize()
    for b in range(2):
        got = torch.cat(outs[b], 2)[0].double().cpu().numpy()
        want = np.stack([ref.got[b][i][1] for i in range(250)], 1)
        assert np.array_equal(got, want)


def test_pools_past_32_bit_offsets():
    """Value rows more than 2^31 elements (and 2^32 bytes) into the pool."""
    w = _work(N=256, C=64, k=9, H=8)
    page = 64
    pages = (2 ** 31 + 2 ** 27) // (64 * w.H * page)
    sv = Serving(w, page)
    per = w.N // page
    sv.table_np[:, :per] = pages - 1 - np.arange(2 * per).reshape(2, per)
    sv.otable_np = np.full_like(sv.table_np, -1)
    sv.otable_np[:, :per] = np.arange(2 * per).reshape(2, per)
    sv.table, sv.otable = (torch.from_numpy(x).cuda() for x in (sv.table_np, sv.otable_np))
    sv.cache = ZetaCache.empty(pages, page, w.H, 3, 64, w.N, w.C, w.k, w.bits,
                               order_pages=2 * per)
    assert sv.cache.v_pages.numel() > 2 ** 31
    for c in ([64, 30], [64, 64], [40, 64], [1, 1]):
        sv.step(c)
    sv.check_order()
    sv.check()
    sv.cache = None


def test_empty_calls():
    c = ZetaCache.empty(4, 16, 2, 3, 64, 64, 32, 4)
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    tb = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    x = torch.zeros(0, 2, 1, 3, device="cuda")
    v = torch.zeros(0, 2, 1, 64, dtype=torch.bfloat16, device="cuda")
    c.append(x, v, z, z, tb)
    c.order(z, z, tb)
    c.attend(x, torch.ones(2, device="cuda"), z, z, tb, v, torch.zeros(0, 2, 1, device="cuda"))
    torch.cuda.synchronize()
    assert int(c.status.item()) == 0


@pytest.mark.parametrize("d_K,bits,page", [(3, 10, 64), (3, 10, 2), (3, 12, 4), (2, 21, 1),
                                           (8, 8, 16)])
@pytest.mark.parametrize("B", [3, 40])
def test_order_of_many_short_chunks(d_K, bits, page, B):
    """Runs of 64 keys into prefixes of up to 8128 entries, many steps a warp: keys all
    over the box (a few among 128 old entries), in one corner of it (many) and equal."""
    H, C, N = 8, 64, 8192
    width = N // page
    cache = ZetaCache.empty(B * width, page, H, d_K, 8, N, C, 8, bits)
    gen = torch.Generator(device="cuda").manual_seed(page)
    table = torch.randperm(B * width, device="cuda", generator=gen).int().view(B, width)
    k = torch.rand(B, H, N // C, C, d_K, device="cuda", generator=gen) * 2 - 1
    k[:, :, 1::3] = k[:, :, 1::3] * 0.02 + 0.5
    k[:, :, 5::9] = k[:, :, 5::9, :1].clone()
    k = k.view(B, H, N, d_K).contiguous()
    v = torch.zeros(B, H, N, 8, dtype=torch.bfloat16, device="cuda")
    p = zb.zeta_problem_t(B, H, N, d_K, 8, 8, C, bits, zb.ZETA_BF16, 0)
    codes = torch.empty(B, H, N, dtype=zb.code_dtype(p), device="cuda")
    zb.zeta_encode(p, k, codes)
    key = codes.cpu().numpy().view(np.uint64 if codes.dtype == torch.int64 else np.uint32)
    count = torch.full((B,), C, dtype=torch.int32, device="cuda")
    rows = table.long().repeat_interleave(page, 1), torch.arange(N, device="cuda") % page
    for c in range(N // C):
        start = torch.full((B,), c * C, dtype=torch.int32, device="cuda")
        at = slice(c * C, c * C + C)
        cache.append(k[:, :, at].contiguous(), v[:, :, at].contiguous(), start, count, table)
        cache.order(start, count, table)
        if c % 25 != 2 and c < N // C - 2:
            continue
        M = c * C + C
        for got, want in ((cache.order_idx, None), (cache.order_codes, key)):
            got = got[(c + 1) & 1][rows[0][:, :M], :, rows[1][:M]]      # [B, M, H]
            got = got.permute(0, 2, 1).contiguous().cpu().numpy()
            order = np.argsort(key[:, :, :M], axis=2, kind="stable")
            want = order if want is None else np.take_along_axis(want[:, :, :M], order, 2)
            assert np.array_equal(got.view(want.dtype) if want is not order else got, want), c
    assert int(cache.status.item()) == 0
