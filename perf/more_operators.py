"""Cases and plain forms of drafting over the paged cache (serving).

A server that guesses tokens ahead brings, per step and sequence, a tree of up to n
drafted tokens: node t hangs below node parent[t] < t, or below the sequence's last
token (parent -1).  Three operators carry such a step over a cache whose sequences
hold ``start`` tokens in pages, beside the framework's append, order and attend:

  reserve  page tables and row numbers of new tokens from the requests' lengths:
           pages are taken from a list of free ones and given back to it
  tree     each node attends as the token at position start + depth of the text made
           of its sequence and its branch: to the k keys around its rank in the sorted
           prefix, to the sequence's tokens of its own chunk, to the nodes above it
           and to itself.  Nodes behind the end of the chunk that start lies in get
           nothing (the prefix they would need depends on their branch)
  accept   the branch that ends in a given node becomes the sequence's next tokens:
           its keys and values go to their pages, up to the chunk's end

Rows from count[b] on are padding and are left as they were.

Pages: token t of sequence b is row t % page of page table[b, t // page]; entry e of
prefix c likewise, in plane c & 1 of the order pools.  The pools' last page belongs to
no sequence.

Where ``own`` is false the plain forms below run (elementary torch operations in
float32, integers in 64 bits); where it is true, the framework's calls.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
FAR = 1 << 62          # sorts behind every code (codes have at most 42 bits here)


def _case(name, op, B, n, ctx, H=8, C=1024, k=64, dK=3, bits=10, dV=64, page=64, dtype="bf16",
          weight="cauchy", gamma=0.5, shape="tree", depth=8, clusters=False, turnover=0.0,
          spare=1.0, lengths=1):
    """op on B sequences of up to ctx tokens with up to n drafted (reserve: new) ones.  H heads,
    chunks of C, windows of k, dK coordinates on a grid of 2^bits cells, values dV wide; shape
    and depth of the trees; turnover: share of the requests that end or begin with the step,
    spare: free pages per page that the step wants; lengths seeds lengths and trees."""
    c = dict(op=op, B=B, n=n, ctx=ctx, H=H, C=C, k=k, dK=dK, bits=bits, dV=dV, page=page,
             dtype=dtype, weight=weight, gamma=gamma, shape=shape, depth=depth,
             clusters=clusters, turnover=turnover, spare=spare, lengths=lengths)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # One user, a few guesses in a short text: nothing but latency.
        _case("tree_one_user", "tree", 1, 8, 1000, H=1, C=128, k=32, dV=32, dtype="f32", page=16,
              depth=4, lengths=1),
        # A small server: small trees under long texts.
        _case("tree_8_users", "tree", 8, 16, 32768, depth=6, lengths=2),
        # A full server: trees of the usual size.
        _case("tree_64_users", "tree", 64, 32, 16384, k=48, page=128, lengths=3),
        # Large trees under long texts.
        _case("tree_32_large", "tree", 32, 64, 65536, depth=10, lengths=4),
        # Long single guesses (text copied from the prompt), values wider, 64-bit codes, softmax.
        _case("tree_chains", "tree", 6, 200, 20000, C=512, k=40, bits=12, dV=96, page=32,
              weight="softmax", shape="chain", clusters=True, lengths=5),
        # Float32 values, odd sizes, chunks that end inside a page.
        _case("tree_f32_odd", "tree", 24, 23, 5000, H=2, C=200, k=37, dV=40, dtype="f32", page=16,
              weight="inv_euclid", lengths=6),
        # A branch per user into the pages.
        _case("accept_64_users", "accept", 64, 32, 4096, lengths=7),
        # Long accepted texts, float32 rows that are no multiple of 16 bytes.
        _case("accept_chains_f32", "accept", 48, 128, 2048, H=4, C=512, dV=33, dtype="f32",
              page=16, shape="chain", lengths=8),
        # One token for each of many requests.
        _case("reserve_512_tokens", "reserve", 512, 1, 16384, lengths=9),
        # Prompt pieces while requests end and begin, and not enough pages for all.
        _case("reserve_turnover", "reserve", 256, 1024, 65536, turnover=0.5, spare=0.7,
              lengths=10),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm uniform."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99))) - 0.5)))


def draw(rng):
    H = rng.choice([1, 2, 5, 8, 8])
    C = rng.choice([128, 200, 256, 512, 1000, 1024, 1024, 2048])
    k = _log(rng, 7, min(C, 100))
    dK, bits = rng.choice([(3, 10), (3, 10), (3, 12), (2, 21), (1, 21), (4, 8)])
    dV = rng.choice([64, 64, 64, 32, 40, 96, 128])
    op = rng.choice(["tree", "tree", "tree", "accept", "reserve"])
    n = _log(rng, 1, min(C, 256 if op != "reserve" else 1024))
    B = _log(rng, 1, max(1, min(256, (4096 if op != "reserve" else 1 << 18) // n)))
    ctx = _log(rng, max(n, C // 2), 65536)
    ctx = max(n, C // 2, min(ctx, (1 << 20 if op != "accept" else 1 << 18) // B))
    c = _case(None, op, B, n, ctx, H=H, C=C, k=k, dK=dK, bits=bits, dV=dV,
              page=rng.choice([16, 32, 64, 128, 256]),
              dtype=rng.choice(["bf16", "bf16", "f32"]),
              weight=rng.choice(["cauchy", "cauchy", "softmax", "inv_euclid"]),
              gamma=round(rng.uniform(0.3, 1.0), 3),
              shape=rng.choice(["tree", "tree", "star", "chain"]), depth=rng.randint(2, 16),
              clusters=rng.random() < 0.3, turnover=round(rng.uniform(0.0, 0.8), 2),
              spare=round(rng.uniform(0.3, 1.5), 2), lengths=rng.randrange(1 << 20))
    while c["B"] > 1 and work(c)["bytes"] > 350e6:          # no more than the largest listed case
        c["B"] //= 2
    return c


def _drafts(case):
    """Per sequence (start, count, parents, leaf): tokens it has, drafted ones, their tree (padding
    nodes have wild parents) and the accepted branch's last node (-1: none)."""
    r = random.Random(case["lengths"])
    B, n, ctx = case["B"], case["n"], case["ctx"]
    got = []
    for b in range(B):
        cnt = n if B == 1 or r.random() < 0.5 else r.randint(1, n)
        start = r.randint(ctx // 8, ctx - 1)
        if B >= 8 and b % 13 == 5:
            cnt = 0                                            # an idle slot of the batch
        par, dep = [], []
        for t in range(cnt):
            if case["shape"] == "chain" or (case["shape"] == "tree" and t < min(3, case["depth"])):
                p = t - 1                                      # the likeliest guesses, one by one
            elif case["shape"] == "star":
                p = -1
            else:
                p = r.choice([-1] + [u for u in range(t) if dep[u] + 1 < case["depth"]])
            par.append(p)
            dep.append(0 if p < 0 else dep[p] + 1)
        leaf = r.randint(-1, cnt - 1) if cnt and r.random() < 0.9 else -1
        if case["shape"] == "chain" and cnt:
            leaf = r.randint(cnt // 2, cnt - 1)
        got.append((start, cnt, par + [r.randint(-9, 3 * n) for _ in range(n - cnt)], leaf))
    return got


def _requests(case):
    """Per request (start, count) of a step and the tokens it had before (a request that begins
    had none, one that ends has nothing any more)."""
    r = random.Random(case["lengths"])
    n, ctx = case["n"], case["ctx"]
    got = []
    for _ in range(case["B"]):
        cnt = n if r.random() < 0.5 else r.randint(1, n)
        before = r.randint(0, max(0, ctx - cnt))
        kind = r.random()
        if kind < case["turnover"] / 2:
            got.append((0, 0, before))
        elif kind < case["turnover"]:
            got.append((0, cnt, 0))
        else:
            got.append((before, 0 if r.random() < 0.1 else cnt, before))
    return got


def _depths(par, cnt):
    dep = []
    for t in range(cnt):
        dep.append(0 if par[t] < 0 else dep[par[t]] + 1)
    return dep


def work(case):
    H, C, k, dK, dV, page = (case[x] for x in ("H", "C", "k", "dK", "dV", "page"))
    e = 2 if case["dtype"] == "bf16" else 4
    row = 4 * dK + e * dV
    if case["op"] == "reserve":                     # both calls of a pass, see run
        moved = sum(abs(-(-(s + c) // page) - -(-t // page)) for s, c, t in _requests(case))
        return {"bytes": 2 * (case["B"] * 20 + 8 * moved) + 4 * case["B"] * case["n"],
                "flops": 2 * (case["B"] + moved)}
    nb = nf = 0
    for s, cnt, par, leaf in _drafts(case):
        if case["op"] == "accept":
            m = min(_depths(par, cnt)[leaf] + 1, C - s % C) if leaf >= 0 else 0
            nb += 2 * m * row * H + 4 * cnt + 4 * (case["n"] + 4)
            nf += m
            continue
        rows = [d for d in _depths(par, cnt) if d < C - s % C]
        if rows:
            m = s // C * C
            seen = min(len(rows) * k, m)            # window rows, each once
            nb += H * ((s % C + len(rows) + seen) * row + 4 * seen
                       + len(rows) * (4 * dK + e * dV + 4))
            pairs = sum(s % C + d + 1 + (k if m else 0) for d in rows)
            nf += H * pairs * (3 * dK + 4 + 2 * dV)
    return {"bytes": max(1, nb), "flops": max(1, nf)}


# ------------------------------------------------------------------- inputs ---

def _points(shape, dK, mid, g):
    """Points of the box: uniform, or around the centres mid (one mixture for queries and keys)."""
    if mid is None:
        x = torch.rand(*shape, dK, device="cuda", generator=g) * 2 - 1
    else:
        at = torch.randint(0, 64, shape, device="cuda", generator=g)
        x = mid[at] + 0.05 * torch.randn(*shape, dK, device="cuda", generator=g)
    return x.clamp(-1.0, 1.0 - 2.0 ** -24).contiguous()


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _tables(need, width, spare, g):
    """(table, unused pages, pages): need[b] pages a sequence in random order, -1 behind them."""
    pages = sum(need) + spare
    perm = torch.randperm(pages, device="cuda", generator=g).int()
    table = torch.full((len(need), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    return table, perm[at:], pages


def _prepare_reserve(case, g):
    B, n, C, page = (case[x] for x in ("B", "n", "C", "page"))
    req = _requests(case)
    width = -(-(case["ctx"] + n) // page)
    N = -(-width * page // C) * C
    width = -(-N // page)
    held = [-(-t // page) for _, _, t in req]
    want = [-(-(s + c) // page) for s, c, _ in req]
    grow = sum(max(0, w - h) for w, h in zip(want, held))
    spare = max(1, int(case["spare"] * grow) - sum(max(0, h - w) for w, h in zip(want, held)))
    table, rest, pages = _tables(held, width, spare, g)
    free = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    free[:spare] = rest
    return dict(case=case, N=N, pages=pages, table=table, held=_ints(held), free=free,
                free_count=_ints([spare]), start=_ints([s for s, _, _ in req]),
                count=_ints([c for _, c, _ in req]), before=_ints([t for _, _, t in req]),
                none=torch.zeros(B, dtype=torch.int32, device="cuda"),
                granted=torch.zeros(B, dtype=torch.int32, device="cuda"),
                back=torch.zeros(B, dtype=torch.int32, device="cuda"),
                slots=torch.zeros(B, n, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "reserve":
        return _prepare_reserve(case, g)
    B, H, n, C, page = (case[x] for x in ("B", "H", "n", "C", "page"))
    dK, dV, bits, op = case["dK"], case["dV"], case["bits"], case["op"]
    drafts = _drafts(case)
    longest = max(s + n for s, *_ in drafts)
    N = -(-(-(-longest // page) * page) // C) * C
    width = -(-N // page)
    need = [-(-(s + (cnt if op == "accept" else 0)) // page) for s, cnt, *_ in drafts]
    table, _, pages = _tables(need, width, 1, g)
    dt = DTYPES[case["dtype"]]
    mid = torch.rand(64, dK, device="cuda", generator=g) * 1.8 - 0.9 if case["clusters"] else None
    k_pages = _points((pages, H, page), dK, mid, g)
    v_pages = torch.randn(pages, H, page, dV, device="cuda", generator=g, dtype=dt)
    k_pages[-1] = 0
    v_pages[-1] = 0
    zt = torch.int64 if dK * bits > 32 else torch.int32
    hold = pages if op == "tree" else 1             # accept does not read the order
    codes = torch.zeros(2, hold, H, page, dtype=zt, device="cuda")
    idx = torch.zeros(2, hold, H, page, dtype=torch.int32, device="cuda")
    if op == "tree":
        for b, (s, cnt, *_) in enumerate(drafts):
            c = s // C
            if c == 0:
                continue
            ids = table[b, :need[b]].long()
            keys = k_pages[ids].transpose(0, 1).reshape(H, -1, dK)[:, :c * C]
            zs, order = torch.sort(_codes(keys, bits), dim=1, stable=True)
            e = torch.arange(c * C, device="cuda")
            codes[c & 1, ids[e // page], :, e % page] = zs.t().to(zt)
            idx[c & 1, ids[e // page], :, e % page] = order.t().int()
    st = dict(case=case, N=N, k_pages=k_pages, v_pages=v_pages, codes=codes, idx=idx, table=table,
              start=_ints([s for s, *_ in drafts]), count=_ints([c for _, c, *_ in drafts]),
              parent=_ints([p for _, _, p, _ in drafts]), k=_points((B, H, n), dK, mid, g),
              v=torch.randn(B, H, n, dV, device="cuda", generator=g, dtype=dt))
    if op == "tree":
        st["q"] = _points((B, H, n), dK, mid, g)
        st["gamma"] = case["gamma"] * (1 + 0.2 * torch.rand(H, device="cuda", generator=g))
        st["out"] = torch.zeros(B, H, n, dV, device="cuda", dtype=dt)
        st["rowsum"] = torch.zeros(B, H, n, device="cuda")
    else:
        st["leaf"] = _ints([f for *_, f in drafts])
        st["accepted"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        st["path"] = torch.zeros(B, n, dtype=torch.int32, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms ---

def _codes(x, bits):
    """Z-order codes (int64) of points [..., dK]: cells in float32, coordinate 0 the most
    significant bit of each level."""
    dK = x.shape[-1]
    u = torch.floor((x + 1.0) * 2.0 ** (bits - 1)).nan_to_num(0.0).clamp(0, 2 ** bits - 1).long()
    j = torch.arange(bits, device=x.device)
    d = torch.arange(dK, device=x.device)[:, None]
    return (((u[..., None] >> j) & 1) << (j * dK + dK - 1 - d)).sum((-1, -2))


def _above(parent, count):
    """[B, n, n]: node u is t or above it; padding nodes are alone."""
    B, n = parent.shape
    t = torch.arange(n, device="cuda")
    a = (t[:, None] == t) | (parent.long()[..., None] == t) & (t < count[:, None])[..., None]
    a = a.float()
    for _ in range(max(1, (n - 1).bit_length())):              # paths of twice the length each time
        a = (a @ a > 0).float()
    return a > 0


def _rows(table, page, pos):
    """(page, row in page) of the tokens pos [B, ...] (any value where there is none)."""
    flat = pos.reshape(pos.shape[0], -1)
    ids = torch.gather(table.long(), 1, (flat // page).clamp(0, table.shape[1] - 1))
    return ids.clamp(min=0).reshape(pos.shape), pos % page


def _distance(q, k):
    return (q - k).square().sum(-1)


def _plain_tree(s):
    case = s["case"]
    B, H, n = s["q"].shape[:3]
    C, k, page = case["C"], case["k"], case["page"]
    q, start = s["q"], s["start"].long()
    t = torch.arange(n, device="cuda")
    above = _above(s["parent"], s["count"])
    depth = above.sum(2) - 1
    live = (t < s["count"][:, None]) & (depth < (C - start % C)[:, None])
    first = start // C * C                                     # of the chunk; the prefix's length
    # the sequence's tokens of the chunk
    pos = first[:, None] + torch.arange(C, device="cuda")
    ids, off = _rows(s["table"], page, pos)
    own_k = s["k_pages"][ids, :, off].transpose(1, 2)                     # [B, H, C, dK]
    own_v = s["v_pages"][ids, :, off].transpose(1, 2).float()
    seen = (pos < start[:, None])[:, None, None]
    d_own = torch.where(seen, _distance(q[:, :, :, None], own_k[:, :, None]), math.inf)
    # the nodes above, and the node
    d_new = torch.where(above[:, None], _distance(q[:, :, :, None], s["k"][:, :, None]), math.inf)
    # the window in prefix first / C
    last = s["N"]
    e = torch.arange(last, device="cuda")
    ids, off = _rows(s["table"], page, e.expand(B, last))
    plane = (first // C & 1)[:, None]
    z = s["codes"][plane, ids, :, off].transpose(1, 2).long()
    z = z & 0xFFFFFFFF if s["codes"].dtype == torch.int32 else z
    z = torch.where(e < first[:, None, None], z, FAR).contiguous()
    tok = s["idx"][plane, ids, :, off].transpose(1, 2).long()
    rank = torch.searchsorted(z, _codes(q, case["bits"]).contiguous(), right=True)
    m = first[:, None, None]
    lo = torch.minimum((rank - (k + 1) // 2).clamp(min=0), (m - k).clamp(min=0))
    at = (lo[..., None] + torch.arange(k, device="cuda")).clamp(max=last - 1)
    there = (m > 0)[..., None]
    w_pos = torch.where(there, torch.gather(tok, 2, at.flatten(2)).view(at.shape), 0)
    ids, off = _rows(s["table"], page, w_pos)
    h = torch.arange(H, device="cuda")[None, :, None, None]
    win_k, win_v = s["k_pages"][ids, h, off], s["v_pages"][ids, h, off].float()
    d_win = torch.where(there, _distance(q[:, :, :, None], win_k), math.inf)
    # weights
    d = torch.cat([d_win, d_own, d_new], 3)
    g2 = s["gamma"].float().square()[None, :, None, None]
    if case["weight"] == "cauchy":
        w = 1 / (1 + d / g2)
    elif case["weight"] == "softmax":
        w = torch.exp((d.amin(3, keepdim=True) - d) / g2)
    else:
        w = (d + 1e-12).rsqrt()
    total = w.sum(3)
    o = (w[..., :k, None] * win_v).sum(3) + w[..., k:k + C] @ own_v
    o = (o + w[..., k + C:] @ s["v"].float()) / total[..., None]
    ok = live[:, None, :]
    s["out"] = torch.where(ok[..., None], o.to(s["out"].dtype), s["out"])
    s["rowsum"] = torch.where(ok, total, s["rowsum"])
    return {"out": s["out"], "rowsum": s["rowsum"]}


def _plain_accept(s):
    case = s["case"]
    B, H, n = s["k"].shape[:3]
    C, page = case["C"], case["page"]
    t = torch.arange(n, device="cuda")
    start, leaf = s["start"].long(), s["leaf"].long()
    above = _above(s["parent"], s["count"])
    line = torch.gather(above, 1, leaf.clamp(min=0)[:, None, None].expand(B, 1, n))[:, 0]
    line = line & (leaf >= 0)[:, None]
    got = torch.minimum(line.sum(1), C - start % C)
    path = torch.where(line, t, n).sort(1).values              # parents come before their children
    live = t < got[:, None]
    path = torch.where(live, path, -1)
    spare = s["k_pages"].shape[0] - 1
    ids, off = _rows(s["table"], page, start[:, None] + t)
    ids = torch.where(live, ids, spare)[:, None, :]
    off = torch.where(live, off, 0)[:, None, :]
    h = torch.arange(H, device="cuda")[None, :, None]
    b = torch.arange(B, device="cuda")[:, None, None]
    src = path.clamp(min=0)[:, None, :]
    ok = live[:, None, :, None]
    s["k_pages"][ids, h, off] = torch.where(ok, s["k"][b, h, src], 0)
    s["v_pages"][ids, h, off] = torch.where(ok, s["v"][b, h, src], 0)
    s["accepted"].copy_(got)
    s["path"].copy_(path)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "accepted": s["accepted"],
            "path": s["path"]}


def _plain_reserve(s, start, count, granted, slots):
    page, table, held, free = s["case"]["page"], s["table"], s["held"].long(), s["free"]
    want = (start.long() + count + page - 1) // page
    e = torch.arange(table.shape[1], device="cuda")
    # back: the sequences' pages in order, the first of them on top
    less = (held - want).clamp(min=0)
    f = s["free_count"].long() + less.sum()
    i = (less.cumsum(0) - less)[:, None] + e - want[:, None]
    drop = (e >= want[:, None]) & (e < held[:, None])
    stack = torch.cat([free, free.new_zeros(1)])               # the last place takes the others
    stack[torch.where(drop, f - 1 - i, free.shape[0]).flatten()] = table.flatten()
    free.copy_(stack[:-1])
    # out: from the top, as long as there are enough
    more = (want - held).clamp(min=0)
    through = more.cumsum(0)
    ok = (more == 0) | (through <= f)
    take = (e >= held[:, None]) & (e < want[:, None]) & ok[:, None]
    i = (through - more)[:, None] + e - held[:, None]
    pages = free[torch.where(take, f - 1 - i, 0).clamp(min=0)]
    table.copy_(torch.where(drop, -1, torch.where(take, pages, table)))
    s["held"].copy_(torch.where(ok, want, held))
    s["free_count"].copy_(f - torch.where(ok, more, 0).sum())
    granted.copy_(torch.where(ok, count, 0))
    if slots is not None:
        t = torch.arange(slots.shape[1], device="cuda")
        ids, off = _rows(table, page, start[:, None].long() + t)
        slots.copy_(torch.where(t < granted[:, None], ids * page + off, -1))


# ------------------------------------------------------------------- one pass ---

def _cache(s):
    """The framework's handle on the pools; a program makes it once, with the pools."""
    if "cache" not in s:
        from order_retrieval_gb300 import ZetaCache
        case = s["case"]
        if case["op"] == "reserve":                 # only tables and lists are looked at
            s["cache"] = ZetaCache.empty(s["pages"], case["page"], 1, 1, 8, s["N"], case["C"],
                                         case["k"], bits=8, order_pages=1)
        else:
            s["cache"] = ZetaCache(s["k_pages"], s["v_pages"], s["codes"], s["idx"], N=s["N"],
                                   C=case["C"], k=case["k"], bits=case["bits"],
                                   weight=case["weight"])
    return s["cache"]


def run(s):
    op = s["case"]["op"]
    if op == "reserve":
        # A step's pages, and the step taken back, as after a draft of which nothing was
        # accepted: what was taken returns, and who had ended is resumed.
        both = ((s["start"], s["count"], s["granted"], s["slots"]),
                (s["before"], s["none"], s["back"], None))
        for start, count, granted, slots in both:
            if own:
                _cache(s).reserve(start, count, s["table"], s["held"], s["free"],
                                  s["free_count"], granted, slots, n=s["case"]["n"])
            else:
                _plain_reserve(s, start, count, granted, slots)
        return {x: s[x] for x in ("granted", "slots", "table", "held", "free", "free_count")}
    if not own:
        return _plain_tree(s) if op == "tree" else _plain_accept(s)
    cache = _cache(s)
    if op == "tree":
        cache.attend_tree(s["q"], s["k"], s["v"], s["gamma"], s["start"], s["count"], s["parent"],
                          s["table"], s["out"], s["rowsum"])
        return {"out": s["out"], "rowsum": s["rowsum"]}
    cache.accept(s["k"], s["v"], s["start"], s["count"], s["parent"], s["leaf"], s["table"],
                 s["accepted"], s["path"])
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "accepted": s["accepted"],
            "path": s["path"]}


# ------------------------------------------------------------- the definition ---

def _curve(x, bits):
    """Codes by the definition, bit by bit (the cells are defined in float32)."""
    cell = ((x + torch.ones((), device=x.device)) * float(1 << (bits - 1))).floor()
    cell = torch.minimum(torch.maximum(cell, torch.zeros_like(cell)),
                         torch.full_like(cell, (1 << bits) - 1)).to(torch.int64)
    z = torch.zeros(x.shape[:-1], dtype=torch.int64, device=x.device)
    for level in reversed(range(bits)):
        for d in range(x.shape[-1]):
            z = z * 2 + ((cell[..., d] >> level) & 1)
    return z


def _line(par, t):
    """Nodes from the first one down to t."""
    got = []
    while t >= 0:
        got.append(t)
        t = par[t]
    return got[::-1]


def _exact_reserve(s, case):
    page = case["page"]
    table, held = s["table"].tolist(), s["held"].tolist()
    free = s["free"].tolist()
    F = s["free_count"].item()
    before = s["before"].tolist()
    got, slots = [], []
    for start, count in ((s["start"].tolist(), s["count"].tolist()), (before, [0] * len(before))):
        want = [-(-(a + c) // page) for a, c in zip(start, count)]
        gone = []
        for b, w in enumerate(want):
            for e in range(w, held[b]):
                gone.append(table[b][e])
                table[b][e] = -1
            held[b] = min(held[b], w)
        for x in reversed(gone):
            free[F] = x
            F += 1
        short, granted = False, []
        for b, w in enumerate(want):
            more = w - held[b]
            short = short or more > F
            if more and short:
                granted.append(0)
                continue
            for e in range(held[b], w):
                F -= 1
                table[b][e] = free[F]
            held[b] = w
            granted.append(count[b])
        if not got:
            got = granted
            slots = [[table[b][(a + t) // page] * page + (a + t) % page if t < granted[b] else -1
                      for t in range(case["n"])] for b, a in enumerate(start)]
    return {"granted": _ints(got), "slots": _ints(slots), "table": _ints(table),
            "held": _ints(held), "free": _ints(free), "free_count": _ints([F])}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "reserve":
        return _exact_reserve(s, case)
    C, k, page = case["C"], case["k"], case["page"]
    if case["op"] == "accept":
        for b, (start, cnt, par, leaf) in enumerate(_drafts(case)):
            path = _line(par, leaf)[:C - start % C] if leaf >= 0 else []
            for d, t in enumerate(path):
                p = int(s["table"][b, (start + d) // page])
                s["k_pages"][p, :, (start + d) % page] = s["k"][b, :, t]
                s["v_pages"][p, :, (start + d) % page] = s["v"][b, :, t]
            s["accepted"][b] = len(path)
            s["path"][b] = _ints(path + [-1] * (case["n"] - len(path)))
        return {x: s[x] for x in ("k_pages", "v_pages", "accepted", "path")}
    out, rowsum = s["out"].double(), s["rowsum"].double()
    for b, (start, cnt, par, _) in enumerate(_drafts(case)):
        lines = [_line(par, t) for t in range(cnt)]
        rows = [t for t in range(cnt) if len(lines[t]) <= C - start % C]
        if not rows:
            continue
        ids = s["table"][b, :-(-start // page)].long()
        keys = s["k_pages"][ids].transpose(0, 1).flatten(1, 2)[:, :start]
        vals = s["v_pages"][ids].transpose(0, 1).flatten(1, 2)[:, :start].double()
        m = start // C * C
        near = torch.zeros(cnt, cnt, dtype=torch.bool)
        for t in rows:
            near[t, lines[t]] = True
        near = near[rows].cuda()
        qd = s["q"][b][:, rows].double()
        all_k = torch.cat([keys[:, m:], s["k"][b][:, :cnt]], 1).double()
        all_v = torch.cat([vals[:, m:], s["v"][b][:, :cnt].double()], 1)
        mask = torch.cat([torch.ones(len(rows), start - m, dtype=torch.bool, device="cuda"), near], 1)
        dist = sum((qd[:, :, None, x] - all_k[:, None, :, x]) ** 2 for x in range(case["dK"]))
        dist = dist.masked_fill(~mask, math.inf)
        if m:
            zs, by = _curve(keys[:, :m], case["bits"]).sort(dim=1, stable=True)
            zq = _curve(s["q"][b][:, rows], case["bits"])
            r = torch.searchsorted(zs, zq.contiguous(), side="right")
            lo = (r - (k + 1) // 2).clamp(0, m - k)
            win = torch.gather(by, 1, (lo[..., None] + torch.arange(k, device="cuda")).flatten(1))
            pick = torch.gather(keys.double(), 1, win[..., None].expand(-1, -1, keys.shape[2]))
            pick = pick.view(*lo.shape, k, -1)
            dw = ((qd[:, :, None] - pick) ** 2).sum(-1)
            pv = torch.gather(vals, 1, win[..., None].expand(-1, -1, vals.shape[2]))
            pv = pv.view(*lo.shape, k, -1)
            both = torch.cat([dist, dw], 2)
        else:
            both, pv = dist, None
        g2 = s["gamma"].double()[:, None, None] ** 2
        if case["weight"] == "cauchy":
            w = torch.where(torch.isinf(both), 0.0, g2 / (g2 + both))
        elif case["weight"] == "softmax":
            w = torch.exp(-(both - both.min(2, keepdim=True).values) / g2)
        else:
            w = 1 / torch.sqrt(both + 1e-12)
        total = w.sum(2)
        o = torch.einsum("hqj,hjd->hqd", w[:, :, :all_k.shape[1]], all_v)
        if pv is not None:
            o = o + torch.einsum("hqk,hqkd->hqd", w[:, :, all_k.shape[1]:], pv)
        out[b][:, rows] = o / total[..., None]
        rowsum[b][:, rows] = total
    return {"out": out, "rowsum": rowsum}
