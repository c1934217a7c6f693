"""Trees of drafted tokens on the host and the plain forms of the drafting calls."""
import numpy as np
import torch

import oracle
from order_retrieval_gb300 import ZetaCache
from order_retrieval_gb300 import workloads as W

from cache_util import EPS, attend_row, window
from gpu_util import in_threads

PAD = 7.0          # what rows without a result hold before and after


def line(parent, t):
    """Nodes from the top down to t."""
    got = []
    while t >= 0:
        got.append(int(t))
        t = parent[t]
    return got[::-1]


def tree(rng, n, kind):
    """Parents of n nodes."""
    if kind == "chain":
        return np.arange(n) - 1
    if kind == "star":
        return np.full(n, -1)
    low = max(0, 3 if kind == "bushy" else 1)
    return np.array([rng.integers(-1, t) if t >= low else t - 1 for t in range(n)])


def reserve_plain(table, held, free, F, start, count, n, page, pages, N):
    """What reserve makes of lists and numpy tables (changed in place): (granted, slots, F)."""
    B, tlen = table.shape
    fit = [0 <= c <= n and 0 <= s <= N - c and 0 <= h <= tlen
           for s, c, h in zip(start, count, held)]
    want = [-(-(int(s) + int(c)) // page) if ok else int(h)
            for s, c, ok, h in zip(start, count, fit, held)]
    back = sum(max(int(h) - w, 0) for h, w in zip(held, want))
    slots = np.full((B, n), -1, np.int64)
    if F < 0 or F + back > pages:
        return np.zeros(B, np.int64), slots, F
    gone = []
    for b, w in enumerate(want):
        gone += table[b, w:held[b]].tolist() if w < held[b] else []
        table[b, w:max(w, held[b])] = -1
        held[b] = min(held[b], w)
    for x in reversed(gone):
        free[F] = x
        F += 1
    granted, short = [], False
    for b, w in enumerate(want):
        more = w - int(held[b])
        short = short or more > F
        if not fit[b] or (more and short):
            granted.append(0)
            continue
        for e in range(held[b], w):
            F -= 1
            table[b, e] = free[F]
        held[b] = w
        granted.append(int(count[b]))
        for t in range(granted[b]):
            i = int(start[b]) + t
            slots[b, t] = table[b, i // page] * page + i % page
    return np.array(granted), slots, F


class Drafting:
    """Sequences of one workload, their first `start` tokens in a cache, and one draft."""

    def __init__(self, w, page, starts, counts, n, weight="cauchy", kind="tree", seed=0,
                 split_tables=False):
        self.w, self.page, self.weight, self.n = w, page, weight, n
        self.starts, self.counts = list(starts), list(counts)
        rng = np.random.default_rng(seed)
        g = W.generate(w)
        self.g, bf = g, w.v_dtype == "bf16"
        self.vdt = torch.bfloat16 if bf else torch.float32
        vt = torch.from_numpy(np.ascontiguousarray(g["v"]))
        k = torch.from_numpy(g["k"]).cuda()
        v = (vt.view(torch.bfloat16) if bf else vt).cuda()
        self.values = [W.values_f64(w, g["v"][b]) for b in range(w.B)]
        self.gamma = torch.from_numpy(g["gamma"]).cuda()
        self.codes = [np.stack([oracle.encode(x, w.bits) for x in g["k"][b]]) for b in range(w.B)]
        per = -(-w.N // page)
        self.pages = w.B * per + 2

        def tables():
            t = np.full((w.B, per + 1), -1, np.int32)          # one entry nobody reads
            t[:, :per] = rng.permutation(self.pages)[:w.B * per].reshape(w.B, per)
            return t

        self.table_np = tables()
        self.table = torch.from_numpy(self.table_np).cuda()
        self.otable = torch.from_numpy(tables()).cuda() if split_tables else None
        self.cache = ZetaCache.empty(self.pages, page, w.H, w.d_K, w.d_V, w.N, w.C, w.k, w.bits,
                                     self.vdt, weight)
        at = np.zeros(w.B, np.int64)
        while (at < self.starts).any():
            cnt = np.minimum(np.array(self.starts) - at, w.C)
            st, ct = self.ints(at), self.ints(cnt)
            rows = [torch.zeros(w.B, w.H, w.C, x.shape[-1], dtype=x.dtype, device="cuda")
                    for x in (k, v)]
            for b in range(w.B):
                for r, x in zip(rows, (k, v)):
                    r[b, :, :cnt[b]] = x[b, :, at[b]:at[b] + cnt[b]]
            self.cache.append(*rows, st, ct, self.table)
            self.cache.order(st, ct, self.table, self.otable)
            at += cnt
        self.start, self.count = self.ints(self.starts), self.ints(self.counts)
        # the draft; padding is NaN and has wild parents
        self.parents = [tree(rng, c, kind) for c in self.counts]
        par = rng.integers(-2 ** 31, 2 ** 31, (w.B, n))
        f32 = rng.uniform(-1, 1, (2, w.B, w.H, n, w.d_K)).astype(np.float32)
        if w.dist == "clusters":
            f32 = np.clip(f32 * 0.1 + 0.3, -1, 1 - 2.0 ** -24).astype(np.float32)
        vv = torch.from_numpy(rng.standard_normal((w.B, w.H, n, w.d_V)).astype(np.float32))
        vv = vv.to(self.vdt)
        for b, c in enumerate(self.counts):
            par[b, :c] = self.parents[b]
            f32[:, b, :, c:] = np.nan
            vv[b, :, c:] = float("nan")
        self.parent = self.ints(par)
        self.qn, self.kn, self.vn = f32[0], f32[1], vv.double().numpy()
        self.q, self.k, self.v = (x.cuda() for x in (torch.from_numpy(f32[0]).contiguous(),
                                                     torch.from_numpy(f32[1]).contiguous(), vv))

    @staticmethod
    def ints(x):
        return torch.from_numpy(np.asarray(x).astype(np.int32)).cuda()

    def outputs(self):
        w, n = self.w, self.n
        return (torch.full((w.B, w.H, n, w.d_V), PAD, dtype=self.vdt, device="cuda"),
                torch.full((w.B, w.H, n), PAD, device="cuda"),
                torch.full((w.B, w.H, n, w.k), 77, dtype=torch.int32, device="cuda"))

    def attend(self, status=0, idx=True):
        out, rs, ix = self.outputs()
        self.cache.attend_tree(self.q, self.k, self.v, self.gamma, self.start, self.count,
                               self.parent, self.table, out, rs, self.otable, ix if idx else None)
        assert int(self.cache.status.item()) == status
        self.out, self.rs, self.idx = out, rs, ix
        return out, rs, ix

    def has_result(self, b, t):
        """Node t's line ends before the chunk does."""
        s, C = self.starts[b], self.w.C
        return t < self.counts[b] and s + len(line(self.parents[b], t)) <= (s // C + 1) * C

    def plain(self, b, t, h, gone=()):
        """(window, out, rowsum, bounds) of node t; gone: tokens and ~nodes without a key."""
        w, s = self.w, self.starts[b]
        nodes = line(self.parents[b], t)
        i = s + len(nodes) - 1
        keys = np.concatenate([self.g["k"][b, h, :s], self.kn[b, h, nodes]])
        vals = np.concatenate([self.values[b][h][:s], self.vn[b, h, nodes]])
        q = self.qn[b, h, t]
        half_w, half_out = (2.0 ** -16, 2.0 ** -8) if w.v_dtype == "bf16" else (0.0, EPS)
        win = window(oracle.encode(q[None], w.bits)[0], self.codes[b][h], i, w.C, w.k)
        gm = float(self.g["gamma"][h])
        if not gone:
            return (win, *attend_row(q, keys, vals, gm, win, i, w.C, self.weight, half_w, half_out))
        own = [j for j in range(i // w.C * w.C, i + 1) if j not in gone]
        left = np.concatenate([[j for j in win if j not in gone], own]).astype(np.int64)
        # the same row over the keys that are left, as one chunk's
        return (win, *attend_row(q, keys[left], vals[left], gm, np.empty(0, np.int64),
                                 len(left) - 1, len(left), self.weight, half_w, half_out))

    def check(self, rows=None, heads=None, gone=None, skip=()):
        """Every node's result (or of nodes `rows` (b, t)) against the plain form; nodes without
        one are left as they were."""
        w = self.w
        out, rs = self.out.double().cpu().numpy(), self.rs.cpu().numpy()
        idx = self.idx.cpu().numpy()

        def one(bt):
            b, t = bt
            if not self.has_result(b, t) or (b, t) in skip:
                assert (out[b, :, t] == PAD).all() and (rs[b, :, t] == PAD).all(), bt
                assert (idx[b, :, t] == 77).all(), bt
                return
            for h in range(w.H) if heads is None else heads:
                win, o, s, bo, bs = self.plain(b, t, h, gone(b) if gone else ())
                want = win if len(win) else np.full(w.k, -1)
                assert np.array_equal(idx[b, h, t], want), (b, h, t)
                err = np.abs(out[b, h, t] - o)
                assert (err <= bo).all(), (b, h, t, err.max(), (err / bo).max())
                assert abs(rs[b, h, t] - s) <= bs, (b, h, t, rs[b, h, t], s)

        todo = rows or [(b, t) for b in range(w.B) for t in range(self.n)]
        in_threads(one, todo)
