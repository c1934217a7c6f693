"""GPU tests of drafting when pages run out and at the end of a text: the step as it is documented
(reserve the longest line up to the chunk's end, attend the whole tree, accept what was granted); calls
that only give pages back."""
import numpy as np
import pytest
import torch

from order_retrieval_gb300 import ZetaCache
from order_retrieval_gb300 import binding as zb
from order_retrieval_gb300 import workloads as W

from draft_util import Drafting, line, reserve_plain, tree

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU"),
]


def _work(**kw):
    base = dict(name="draft", B=5, H=2, N=128, d_K=3, d_V=64, k=12, C=32, bits=10, v_dtype="bf16",
                gamma=(0.5, 1.0), dist="uniform", v_dist="normal", seed=31)
    base.update(kw)
    return W.Workload(**base)


@pytest.mark.parametrize("v_dtype,page", [("bf16", 16), ("f32", 4), ("bf16", 64)])
def test_steps_under_a_short_list(v_dtype, page):
    """Texts are written up to their last place, N - 1 among the starts; the list is too short for
    all.  Who is refused accepts nothing, no page is read that was never written, and nothing is
    recorded.  Where nobody gets a page the longest text ends and its place begins again."""
    w = _work(v_dtype=v_dtype)
    n, B, N, C = 11, w.B, w.N, w.C
    d = Drafting(w, page, [0] * B, [0] * B, n)
    c, rng = d.cache, np.random.default_rng(page)
    full = [torch.from_numpy(d.g[x]).cuda() for x in "qk"]
    full.append(torch.from_numpy(np.stack(d.values).astype(np.float32)).cuda().to(d.vdt))
    pages = 7 if page == 64 else 3 * N // page       # of 5 N / page
    table, held = d.ints(np.full((B, N // page), -1)), d.ints([0] * B)
    free = d.ints(np.concatenate([rng.permutation(d.pages)[:pages], np.full(d.pages - pages, -7)]))
    fc = d.ints([pages])
    ours = set(free[:pages].tolist())
    at, ended, refused, last, checked = np.zeros(B, np.int64), 0, 0, 0, 0
    for step in range(400):
        if ended >= 5 and last and refused > 20:
            break
        ended += int((at == N).sum())
        at[at == N] = 0                              # a text is whole: another one begins
        count = rng.integers(0, n + 1, B)
        par, true, longest = np.full((B, n), 99), [[] for _ in range(B)], np.zeros(B, np.int64)
        for b in range(B):
            p = tree(rng, count[b], "tree")
            par[b, :count[b]] = p
            if count[b]:
                true[b] = line(p, int(rng.integers(0, count[b])))
                longest[b] = max(len(line(p, t)) for t in range(count[b]))
        q, k = (torch.rand(B, w.H, n, w.d_K, device="cuda") * 2 - 1 for _ in range(2))
        v = torch.randn(B, w.H, n, w.d_V, device="cuda").to(d.vdt)
        for b in range(B):
            for j, t in enumerate(true[b][:N - at[b]]):
                for x, y in zip((q, k, v), full):
                    x[b, :, t] = y[b, :, at[b] + j]
        start, cnt, parent = d.ints(at), d.ints(count), d.ints(par)
        leaf = d.ints([x[-1] if x else -1 for x in true])
        want = torch.minimum(d.ints(longest), C - start % C)
        out, rs, idx = d.outputs()
        acc, granted = d.ints([9] * B), d.ints([9] * B)
        c.reserve(start, want, table, held, free, fc, granted, n=n)
        c.attend_tree(q, k, v, d.gamma, start, cnt, parent, table, out, rs, idx=idx)
        c.accept(k, v, start, cnt, parent, leaf, table, acc, granted=granted)
        c.order(start, acc, table, n=n)
        assert int(c.status.item()) == 0
        got, g = acc.cpu().numpy(), granted.cpu().numpy()
        for b in range(B):
            line_of = min(len(true[b]), C - at[b] % C)
            assert g[b] in (0, int(want[b])) and got[b] == (line_of if g[b] else 0)
            assert held[b] * page >= at[b] + got[b]
            refused += int(want[b]) > 0 and g[b] == 0
            last += at[b] == N - 1 and got[b] == 1
            for j in range(got[b])[:2]:
                i, t, h = int(at[b]) + j, true[b][j], j % w.H
                d.parents[b], d.starts[b] = [-1], i
                d.qn[b, h, 0], d.kn[b, h, 0] = d.g["q"][b, h, i], d.g["k"][b, h, i]
                d.vn[b, h, 0] = d.values[b][h][i]
                win, o, s, bo, bs = d.plain(b, 0, h)
                assert np.array_equal(idx[b, h, t].cpu().numpy(), win if len(win) else [-1] * w.k)
                assert (np.abs(out[b, h, t].double().cpu().numpy() - o) <= bo).all()
                assert abs(float(rs[b, h, t]) - s) <= bs
                checked += 1
            e = torch.arange(int(at[b] + got[b]), device="cuda")
            ids = table[b].long()[e // page]
            for x, y in zip((c.k_pages, c.v_pages), full[1:]):
                assert torch.equal(x[ids, :, e % page], y[b, :, e].transpose(0, 1))
        at += got
        if (count > 0).any() and not got.any():      # nobody moves: the longest one leaves
            at[at.argmax()] = 0
        c.reserve(d.ints(at), d.ints([0] * B), table, held, free, fc, granted, n=n)
        used = sum((table[b, :int(held[b])].tolist() for b in range(B)), [])
        left = used + free[:int(fc)].tolist()
        assert len(left) == pages and set(left) == ours
    assert ended >= 5 and refused > 20 and last and checked > 300, (ended, refused, last)


@pytest.mark.parametrize("kw", [dict(), dict(v_dtype="f32", d_V=33), dict(d_V=250)])
def test_granted_ends_the_line(kw):
    w = _work(B=6, **kw)
    d = Drafting(w, 16, [40, 40, 40, 40, 60, 0], [20, 20, 20, 20, 20, 0], 20, kind="chain")
    kp, vp = d.cache.k_pages.clone(), d.cache.v_pages.clone()
    granted = [3, 0, -5, 2 ** 31 - 1, 2, 7]
    m = [3, 0, 0, 20, 2, 0]
    for b in range(6):
        for j in range(m[b]):
            i = d.starts[b] + j
            kp[d.table_np[b][i // 16], :, i % 16] = d.k[b, :, j]
            vp[d.table_np[b][i // 16], :, i % 16] = d.v[b, :, j]
    table = d.table.clone()
    table[1, 2:], table[0, 3:] = -1, -1              # pages that nothing was granted for
    acc, path = d.ints([9] * 6), d.ints(np.full((6, 20), 9))
    d.cache.accept(d.k, d.v, d.start, d.count, d.parent, d.ints([19] * 6), table, acc, path,
                   granted=d.ints(granted))
    assert int(d.cache.status.item()) == 0 and acc.tolist() == m
    for b in range(6):
        assert path[b].tolist() == list(range(m[b])) + [-1] * (20 - m[b])
    assert torch.equal(kp, d.cache.k_pages) and torch.equal(vp, d.cache.v_pages)
    # the binding's call, and what it refuses
    p = zb.problem(w.B, w.H, w.N, w.d_K, w.d_V, w.k, w.C, w.bits, w.v_dtype)
    cc = zb.zeta_cache_t(20, 16, d.cache.pages, d.cache.order_pages, table.shape[1])
    acc2 = d.ints([9] * 6)
    args = (p, cc, d.k, d.v, d.start, d.count, d.parent, d.ints([19] * 6))
    pools = (table, d.cache.k_pages, d.cache.v_pages)
    zb.zeta_cache_accept_granted(*args, d.ints(granted), *pools, acc2)
    assert torch.equal(acc, acc2)
    for bad in (d.ints(granted).long(), d.ints(granted[:5])):
        with pytest.raises((TypeError, ValueError)):
            d.cache.accept(*args[2:], table, acc, granted=bad)
        with pytest.raises((TypeError, ValueError)):
            zb.zeta_cache_accept_granted(*args, bad, *pools, acc2)


@pytest.mark.parametrize("how", ["n", "slots", "heads", "binding"])
def test_reserve_without_rows_gives_back(how):
    """Requests that end or were cut short, and no row of a new token in the call."""
    B, page, pages, N = 9, 8, 80, 128
    up, rng = Drafting.ints, np.random.default_rng(3)
    cache = ZetaCache.empty(pages, page, 1, 1, 8, N, 32, 1, 8, order_pages=1)
    table, held = np.full((B, N // page), -1), np.zeros(B, np.int64)
    free, F = rng.permutation(pages), pages
    _, _, F = reserve_plain(table, held, free, F, 10 * np.arange(B), [10] * B, 10, page, pages, N)
    start = np.array([0, 3, 30, 0, 41, 8, 70, 16, 0])
    x = [up(table), up(held), up(free), up([F])]
    want, _, F2 = reserve_plain(table, held, free, F, start, [0] * B, 0, page, pages, N)
    assert F2 > F
    got, none = up([9] * B), up([0] * B)
    if how == "n":
        cache.reserve(up(start), none, *x, got, n=0)
    elif how == "slots":
        cache.reserve(up(start), none, *x, got, up(np.zeros((B, 0))))
    else:
        p = zb.problem(B, 0 if how == "heads" else 1, N, 1, 8, 1, 32, 8, "bf16")
        cc = zb.zeta_cache_t(4 if how == "heads" else 0, page, pages, 1, N // page)
        zb.zeta_cache_reserve(p, cc, up(start), none, *x, got)
    assert int(cache.status.item()) == 0 and got.tolist() == want.tolist()
    for a, b in zip(x, (table, held, free, [F2])):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("v_dtype", ["bf16", "f32"])
def test_arrays_side_by_side(v_dtype):
    """All arrays of one node a sequence, end to end in one buffer: none meets another."""
    w = _work(B=6, H=1, k=1, d_K=1, d_V=8, v_dtype=v_dtype)
    d = Drafting(w, 16, [40, 33, 0, 100, 127, 64], [1] * 6, 1)
    want = [x.clone() for x in d.attend()]
    buf = torch.zeros(4096, dtype=torch.int32, device="cuda")
    at = 0

    def put(x):
        """The tensor's copy behind the last one (values on 16 bytes)."""
        nonlocal at
        words = x.numel() * x.element_size() // 4
        at = -(-at // 4) * 4 if x.dim() == 4 and x.shape[-1] == 8 else at
        y = buf[at:at + words].view(x.dtype).view(x.shape)
        at += words
        y.copy_(x)
        return y

    out, rs, idx = d.outputs()
    v, out = put(d.v), put(out)
    q, k, rs, idx = put(d.q), put(d.k), put(rs), put(idx)
    start, count, parent, table, gamma = (put(x) for x in (d.start, d.count, d.parent, d.table,
                                                           d.gamma))
    d.cache.attend_tree(q, k, v, gamma, start, count, parent, table, out, rs, idx=idx)
    for a, b in zip((out, rs, idx), want):
        assert torch.equal(a, b)
    leaf, acc, granted, path = (put(d.ints(x)) for x in ([0] * 6, [9] * 6, [1] * 6, [[9]] * 6))
    d.cache.accept(k, v, start, count, parent, leaf, table, acc, path, granted=granted)
    assert acc.tolist() == [1] * 6 and path.tolist() == [[0]] * 6
    tab, held = put(d.ints(np.full((6, w.N // 16), -1))), put(d.ints([0] * 6))
    free, fc = put(d.ints(np.arange(d.pages))), put(d.ints([d.pages]))
    got, slots = put(d.ints([0] * 6)), put(d.ints([[0]] * 6))
    d.cache.reserve(start, count, tab, held, free, fc, got, slots)
    assert int(d.cache.status.item()) == 0 and got.tolist() == [1] * 6 and at < 4096
    want = [-(-(s + 1) // 16) for s in d.starts]
    assert held.tolist() == want and fc.tolist() == [d.pages - sum(want)]
    for b, s in enumerate(d.starts):
        assert slots[b, 0] == int(tab[b, s // 16]) * 16 + s % 16


def test_row_numbers_of_other_dimensions():
    """Refused as every other wrong shape is."""
    up, cache = Drafting.ints, ZetaCache.empty(10, 8, 1, 1, 8, 64, 32, 1, 8, order_pages=1)
    x = [up(np.full((1, 8), -1)), up([0]), up(np.arange(10)), up([10])]
    for slots in (up(7), up([7]), up([[[7]]])):
        for n in (None, 1):
            with pytest.raises(ValueError):
                cache.reserve(up([0]), up([1]), *x, up([0]), slots, n=n)
    assert x[3].tolist() == [10]


def test_a_captured_step_under_a_short_list():
    """reserve, attend_tree, accept and order captured once; replayed with lists of other lengths they
    give what eager calls do."""
    w = _work(B=6, H=2)
    starts, n = [46, 33, 95, 110, 127, 64], 7        # pages for the first, fourth and last
    d = Drafting(w, 16, starts, [n] * 6, n, kind="chain")
    c, leaf = d.cache, d.ints([6, 3, 5, 6, 6, 2])
    longest = torch.minimum(d.count, w.C - d.start % w.C)
    spare = d.ints(np.arange(d.pages))
    pools = (c.k_pages, c.v_pages, c.order_codes, c.order_idx)
    kept = [x.clone() for x in pools]
    state = [d.table.clone(), d.ints([-(-s // 16) for s in starts]), spare, d.ints([0])]
    state[0][:, w.N // 16:] = -1
    for b, s in enumerate(starts):                   # pages of the text alone; the others are free
        state[0][b, -(-s // 16):] = -1
    used = {int(x) for x in state[0].flatten() if x >= 0}
    rest = [x for x in range(d.pages) if x not in used]
    state[2][:len(rest)] = d.ints(rest)
    outs = [*d.outputs(), d.ints([9] * 6), d.ints([9] * 6), d.ints(np.full((6, n), 9))]
    work = [x.clone() for x in state + outs]

    def reset(places):
        for a, b in zip([*work, *pools], [*state, *outs, *kept]):
            a.copy_(b)
        work[3].fill_(places)

    def step():
        table, held, free, fc, out, rs, idx, acc, granted, path = work
        c.reserve(d.start, longest, table, held, free, fc, granted, n=n)
        c.attend_tree(d.q, d.k, d.v, d.gamma, d.start, d.count, d.parent, table, out, rs, idx=idx)
        c.accept(d.k, d.v, d.start, d.count, d.parent, leaf, table, acc, path, granted=granted)
        c.order(d.start, acc, table, n=n)

    want = {}
    for places in (0, 1, 2, len(rest)):
        reset(places)
        step()
        want[places] = [x.clone() for x in [*work, *pools]]
    assert len({tuple(x[7].tolist()) for x in want.values()}) == 4
    reset(0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for places in (2, 0, len(rest), 1):
        reset(places)
        graph.replay()
        for a, b in zip([*work, *pools], want[places]):
            assert torch.equal(a, b), places
    assert int(c.status.item()) == 0
