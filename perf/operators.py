"""Cases and plain forms of the paged-cache operators (serving).

A cache holds the keys and values of several sequences in pages, and for every
sequence the order of its completed chunks' keys along the Z-order curve.  Per
call a batch of sequences brings up to n new tokens each (n <= C, ragged):

  append   keys and values of the new tokens go to their pages
  order    a sequence that completes chunk c gets prefix c + 1: the keys of
           chunks 0..c by (code, token), merged from prefix c and the chunk
  attend   each new token attends to the k keys around its rank in its prefix
           and to its own chunk's keys up to itself

Pages: token t of sequence b is row t % page of page table[b, t // page]; entry e
of prefix c likewise, in plane c & 1 of the order pools.  The pools' last page
belongs to no sequence.

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
          weight="cauchy", gamma=0.5, ragged=True, clusters=False, lengths=1):
    """op on B sequences of up to ctx tokens, up to n of them new; H heads, chunks of C, windows
    of k, dK coordinates on a grid of 2^bits cells, values dV wide; lengths seeds the sequences'
    lengths."""
    c = dict(op=op, B=B, n=n, ctx=ctx, H=H, C=C, k=k, dK=dK, bits=bits, dV=dV, page=page,
             dtype=dtype, weight=weight, gamma=gamma, ragged=ragged, clusters=clusters,
             lengths=lengths)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # One user, one token of a short text: nothing but latency.
        _case("attend_one_token", "attend", 1, 1, 1000, H=1, C=128, k=32, dV=32, dtype="f32",
              page=16, ragged=False, lengths=1),
        # A batch of users answering, one token each, at any depth of long texts.
        _case("attend_64_tokens", "attend", 64, 1, 65536, lengths=2),
        # A full server: many users, shorter texts.
        _case("attend_512_tokens", "attend", 512, 1, 16384, k=48, page=128, lengths=3),
        # A few guessed tokens per user checked at once; the finer grid has 64-bit codes.
        _case("attend_5_guesses", "attend", 8, 5, 4096, C=256, k=32, bits=12, page=16,
              weight="softmax", clusters=True, lengths=4),
        # One long prompt read in pieces of a chunk, the last piece.
        _case("attend_one_piece", "attend", 1, 1024, 65536, ragged=False, lengths=5),
        # Prompts of several users read together, pieces of unequal length across chunk ends.
        _case("attend_16_pieces", "attend", 16, 1024, 32768, lengths=6),
        # Float32 values, odd widths and chunks that end inside a page.
        _case("attend_f32_pieces", "attend", 4, 173, 5000, H=2, C=200, k=37, dV=40, dtype="f32",
              page=16, weight="inv_euclid", lengths=7),
        # One token per user into the pages.
        _case("append_64_tokens", "append", 64, 1, 16384, lengths=8),
        # Prompt pieces into the pages.
        _case("append_16_pieces", "append", 16, 1024, 32768, lengths=9),
        # One long text completes a chunk while it is answered.
        _case("order_one", "order", 1, 1, 65536, ragged=False, lengths=10),
        # Prompt pieces complete chunks in most sequences of a batch.
        _case("order_32_pieces", "order", 32, 1024, 65536, page=128, lengths=11),
        # Short chunks, 64-bit codes, clustered keys with many equal codes.
        _case("order_short_chunks", "order", 12, 40, 6000, H=4, C=128, dK=2, bits=21, page=16,
              clusters=True, lengths=12),
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
    n = 1 if rng.random() < 0.4 else _log(rng, 2, min(C, 1024))
    op = rng.choice(["attend", "attend", "attend", "append", "order"])
    B = _log(rng, 1, max(1, min(256, 8192 // n)))
    ctx = _log(rng, max(n, C // 2), 65536)
    ctx = max(n, C // 2, min(ctx, (1 << 21) // B))
    if op == "order":
        ctx = max(ctx, C)
    c = _case(None, op, B, n, ctx, H=H, C=C, k=k, dK=dK, bits=bits, dV=dV,
              page=rng.choice([16, 32, 64, 128, 256]),
              dtype=rng.choice(["bf16", "bf16", "f32"]),
              weight=rng.choice(["cauchy", "cauchy", "softmax", "inv_euclid"]),
              gamma=round(rng.uniform(0.3, 1.0), 3), ragged=rng.random() < 0.8,
              clusters=rng.random() < 0.3, lengths=rng.randrange(1 << 20))
    while c["B"] > 1 and work(c)["bytes"] > 400e6:          # no more than the largest listed case
        c["B"] //= 2
    return c


def _lengths(case):
    """(start, count) of every sequence: tokens it had before, tokens it brings."""
    r = random.Random(case["lengths"])
    B, n, ctx, C = case["B"], case["n"], case["ctx"], case["C"]
    got = []
    for b in range(B):
        if not case["ragged"]:
            cnt, end = n, ctx
        else:
            cnt = n if n == 1 or r.random() < 0.5 else r.randint(1, n)
            end = r.randint(max(cnt, ctx // 8), ctx)
        if case["op"] == "order" and (b == 0 or r.random() < 0.8):
            end = max(C, end // C * C) + r.randint(0, cnt - 1)     # completes a chunk
            end = max(end, cnt)
        if case["ragged"] and B >= 8 and b % 13 == 5:
            end, cnt = end - cnt, 0                                # an idle slot of the batch
        got.append((end - cnt, cnt))
    return got


def work(case):
    H, C, k, dK, dV, n = (case[x] for x in ("H", "C", "k", "dK", "dV", "n"))
    e = 2 if case["dtype"] == "bf16" else 4
    z = 8 if case["dK"] * case["bits"] > 32 else 4
    row = 4 * dK + e * dV
    nb = nf = 0
    for s, cnt in _lengths(case):
        end = s + cnt
        if case["op"] == "append":
            nb += 2 * cnt * row
        elif case["op"] == "order":
            c = end // C
            if c > s // C:
                nb += 4 * dK * C + (z + 4) * (2 * (c - 1) * C + C)
                nf += (c * C) + C * max(1, int(math.log2(C)))
        elif cnt:
            for c in range(s // C, (end - 1) // C + 1):
                i0, i1 = max(s, c * C) - c * C, min(end, (c + 1) * C) - c * C
                q = i1 - i0                       # queries of chunk c; they see i0 + 1 .. i1 keys
                seen = min(q * k, c * C)          # window rows, each once
                nb += (i1 + seen) * row + 4 * seen + q * (4 * dK + e * dV + 4)
                pairs = q * (i0 + i1 + 1) // 2 + (q * k if c else 0)
                nf += pairs * (3 * dK + 4 + 2 * dV)
    return {"bytes": max(1, H * nb), "flops": H * nf}


# ------------------------------------------------------------------- inputs ---

def _points(shape, dK, mid, g):
    """Points of the box: uniform, or around the centres mid (one mixture for queries and keys)."""
    if mid is None:
        x = torch.rand(*shape, dK, device="cuda", generator=g) * 2 - 1
    else:
        at = torch.randint(0, 64, shape, device="cuda", generator=g)
        x = mid[at] + 0.05 * torch.randn(*shape, dK, device="cuda", generator=g)
    return x.clamp(-1.0, 1.0 - 2.0 ** -24).contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, n, C, page = (case[x] for x in ("B", "H", "n", "C", "page"))
    dK, dV, bits, op = case["dK"], case["dV"], case["bits"], case["op"]
    lens = _lengths(case)
    longest = max(s + c for s, c in lens)
    width = -(-max(longest, 1) // page)
    N = -(-width * page // C) * C
    width = -(-N // page)
    need = [-(-(s + c) // page) for s, c in lens]
    pages = sum(need) + 1
    perm = torch.randperm(pages - 1, device="cuda", generator=g).int()
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
    dt = DTYPES[case["dtype"]]
    mid = torch.rand(64, dK, device="cuda", generator=g) * 1.8 - 0.9 if case["clusters"] else None
    k_pages = _points((pages, H, page), dK, mid, g)
    k_pages[-1] = 0
    v_pages = torch.randn(pages, H, page, dV, device="cuda", generator=g, dtype=dt)
    v_pages[-1] = 0
    zt = torch.int64 if dK * bits > 32 else torch.int32
    hold = pages if op != "append" else 1          # append does not read the order
    codes = torch.zeros(2, hold, H, page, dtype=zt, device="cuda")
    idx = torch.zeros(2, hold, H, page, dtype=torch.int32, device="cuda")
    if op != "append":
        for b, (s, cnt) in enumerate(lens):
            first = s // C
            last = (s + cnt - 1) // C if op == "attend" and cnt else first
            if last == 0:
                continue
            ids = table[b, :need[b]].long()
            keys = k_pages[ids].transpose(0, 1).reshape(H, -1, dK)[:, :last * C]
            z = _codes(keys, bits)
            for c in range(max(first, 1), last + 1):
                zs, order = torch.sort(z[:, :c * C], dim=1, stable=True)
                e = torch.arange(c * C, device="cuda")
                codes[c & 1, ids[e // page], :, e % page] = zs.t().to(zt)
                idx[c & 1, ids[e // page], :, e % page] = order.t().int()
    st = dict(case=case, N=N, k_pages=k_pages, v_pages=v_pages, codes=codes, idx=idx, table=table,
              start=torch.tensor([s for s, _ in lens], dtype=torch.int32, device="cuda"),
              count=torch.tensor([c for _, c in lens], dtype=torch.int32, device="cuda"))
    if op == "append":
        st["k"] = _points((B, H, n), dK, mid, g)
        st["v"] = torch.randn(B, H, n, dV, device="cuda", generator=g, dtype=dt)
    if op == "attend":
        st["q"] = _points((B, H, n), dK, mid, g)
        st["gamma"] = case["gamma"] * (1 + 0.2 * torch.rand(H, device="cuda", generator=g))
        st["out"] = torch.zeros(B, H, n, dV, device="cuda", dtype=dt)
        st["rowsum"] = torch.zeros(B, H, n, device="cuda")
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


def _unsigned(z):
    return z.long() & 0xFFFFFFFF if z.dtype == torch.int32 else z


def _plain_append(s):
    B, H, n = s["k"].shape[:3]
    page = s["k_pages"].shape[2]
    t = torch.arange(n, device="cuda")
    pos = s["start"][:, None].long() + t
    live = t < s["count"][:, None]
    spare = s["k_pages"].shape[0] - 1
    ids = torch.gather(s["table"].long(), 1, torch.where(live, pos // page, 0))
    ids = torch.where(live, ids, spare)[:, None, :]
    h = torch.arange(H, device="cuda")[None, :, None]
    off = torch.where(live, pos % page, 0)[:, None, :]
    ok = live[:, None, :, None]
    s["k_pages"][ids, h, off] = torch.where(ok, s["k"], 0)
    s["v_pages"][ids, h, off] = torch.where(ok, s["v"], 0)
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _rows(s, pos):
    """(page, row in page) of the tokens pos [B, ...] (any value where there is none)."""
    page = s["k_pages"].shape[2]
    flat = pos.reshape(pos.shape[0], -1)
    ids = torch.gather(s["table"].long(), 1, (flat // page).clamp(0, s["table"].shape[1] - 1))
    return ids.clamp(min=0).reshape(pos.shape), pos % page


def _prefix(s, c, length):
    """Codes and tokens [B, H, length] of prefix c [B]."""
    B = c.shape[0]
    e = torch.arange(length, device="cuda").expand(B, length)
    ids, off = _rows(s, e)
    plane = (c & 1)[:, None]
    return (_unsigned(s["codes"][plane, ids, :, off]).transpose(1, 2),
            s["idx"][plane, ids, :, off].long().transpose(1, 2))


def _plain_order(s):
    case = s["case"]
    B, H, C, page = case["B"], case["H"], case["C"], case["page"]
    spare = s["k_pages"].shape[0] - 1
    M = s["N"] - C
    end = s["start"].long() + s["count"]
    c = end // C - 1                                   # the chunk that may be complete
    done = (end // C > s["start"].long() // C)[:, None, None]
    old_z, old_i = _prefix(s, c.clamp(min=0), M)
    e = torch.arange(M, device="cuda")
    old = done & (e < (c * C)[:, None, None])
    pos = c.clamp(min=0)[:, None] * C + torch.arange(C, device="cuda")
    ids, off = _rows(s, pos)
    new_z = _codes(s["k_pages"][ids, :, off].transpose(1, 2), case["bits"])
    z = torch.cat([torch.where(old, old_z, FAR), new_z], 2)
    i = torch.cat([old_i, pos[:, None, :].expand(B, H, C)], 2)
    z, by = torch.sort(z, dim=2, stable=True)          # equal codes: earlier tokens first
    i = torch.gather(i, 2, by)
    e = torch.arange(M + C, device="cuda").expand(B, M + C)
    live = done & (e < ((c + 1) * C)[:, None])[:, None, :]
    ids, off = _rows(s, e)
    at = ((c.clamp(min=0) + 1 & 1)[:, None, None].expand(B, 1, M + C) * live,
          torch.where(live, ids[:, None], spare), torch.arange(H, device="cuda")[None, :, None],
          torch.where(live, off[:, None], 0))
    s["codes"][at] = torch.where(live, z, 0).to(s["codes"].dtype)
    s["idx"][at] = torch.where(live, i, 0).int()
    return {"codes": s["codes"], "idx": s["idx"]}


def _distance(q, k):
    return (q - k).square().sum(-1)


def _plain_attend(s):
    case = s["case"]
    B, H, n = s["q"].shape[:3]
    C, k = case["C"], case["k"]
    q = s["q"]
    t = torch.arange(n, device="cuda")
    pos = s["start"][:, None].long() + t               # [B, n]
    live = t < s["count"][:, None]
    c0 = s["start"].long() // C
    # own chunk: the new tokens lie in chunk c0 or the next one
    span = C if n == 1 else 2 * C
    own_pos = c0[:, None] * C + torch.arange(span, device="cuda")
    ids, off = _rows(s, own_pos)
    own_k = s["k_pages"][ids, :, off].transpose(1, 2)                     # [B, H, span, dK]
    own_v = s["v_pages"][ids, :, off].transpose(1, 2).float()
    seen = (own_pos[:, None] // C == pos[..., None] // C) & (own_pos[:, None] <= pos[..., None])
    d_own = torch.where(seen[:, None], _distance(q[:, :, :, None], own_k[:, :, None]), math.inf)
    # window: k entries around the rank in prefix c
    last = s["N"]
    z = _codes(q, case["bits"])
    parts = [_prefix(s, c0, last)] + ([_prefix(s, c0 + 1, last)] if n > 1 else [])
    e = torch.arange(last, device="cuda")
    second = (pos // C > c0[:, None])[:, None]                            # [B, 1, n]
    r = [torch.searchsorted(torch.where(e < ((c0 + j) * C)[:, None, None], pz, FAR).contiguous(),
                            z.contiguous(), right=True) for j, (pz, _) in enumerate(parts)]
    rank = r[0] if n == 1 else torch.where(second, r[1], r[0])
    m = (pos // C * C)[:, None]
    first = torch.minimum((rank - (k + 1) // 2).clamp(min=0), (m - k).clamp(min=0))
    at = (first[..., None] + torch.arange(k, device="cuda")).clamp(max=last - 1)
    w_pos = torch.gather(parts[0][1], 2, at.flatten(2)).view(at.shape)
    if n > 1:
        w_pos = torch.where(second[..., None],
                            torch.gather(parts[1][1], 2, at.flatten(2)).view(at.shape), w_pos)
    there = (m > 0)[..., None]
    w_pos = torch.where(there, w_pos, 0)
    ids, off = _rows(s, w_pos)
    h = torch.arange(H, device="cuda")[None, :, None, None]
    win_k, win_v = s["k_pages"][ids, h, off], s["v_pages"][ids, h, off].float()
    d_win = torch.where(there, _distance(q[:, :, :, None], win_k), math.inf)
    # weights
    d = torch.cat([d_win, d_own], 3)
    g2 = s["gamma"].float().square()[None, :, None, None]
    if case["weight"] == "cauchy":
        w = 1 / (1 + d / g2)
    elif case["weight"] == "softmax":
        w = torch.exp((d.amin(3, keepdim=True).nan_to_num(posinf=0.0) - d) / g2)
    else:
        w = (d + 1e-12).rsqrt()
    total = w.sum(3)
    o = (w[..., :k, None] * win_v).sum(3) + w[..., k:] @ own_v
    o = o / total[..., None]
    ok = live[:, None, :]
    s["out"] = torch.where(ok[..., None], o.to(s["out"].dtype), s["out"])
    s["rowsum"] = torch.where(ok, total, s["rowsum"])
    return {"out": s["out"], "rowsum": s["rowsum"]}


# ------------------------------------------------------------------- one pass ---

def _cache(s):
    """The framework's handle on the pools; a program makes it once, with the pools."""
    if "cache" not in s:
        from order_retrieval_gb300 import ZetaCache
        case = s["case"]
        s["cache"] = ZetaCache(s["k_pages"], s["v_pages"], s["codes"], s["idx"], N=s["N"],
                               C=case["C"], k=case["k"], bits=case["bits"], weight=case["weight"])
    return s["cache"]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _plain_append, "order": _plain_order, "attend": _plain_attend}[op](s)
    cache = _cache(s)
    if op == "append":
        cache.append(s["k"], s["v"], s["start"], s["count"], s["table"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "order":
        cache.order(s["start"], s["count"], s["table"])
        return {"codes": s["codes"], "idx": s["idx"]}
    cache.attend(s["q"], s["gamma"], s["start"], s["count"], s["table"], s["out"], s["rowsum"])
    return {"out": s["out"], "rowsum": s["rowsum"]}


# ------------------------------------------------------------- the definition ---

def _sequence(pool, table, length):
    """[H, length, ...] of one sequence, page by page."""
    page = pool.shape[2]
    parts = [pool[int(i)] for i in table[:-(-length // page)].tolist()]
    return torch.cat(parts, 1)[:, :length] if parts else pool[0][:, :0]


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


def exact(case, seed):
    s = prepare(case, seed)
    C, k, op = case["C"], case["k"], case["op"]
    if op == "append":
        for b, (start, cnt) in enumerate(_lengths(case)):
            table = s["table"][b].tolist()
            for p in range(start // case["page"], -(-(start + cnt) // case["page"]) if cnt else 0):
                lo, hi = max(start, p * case["page"]), min(start + cnt, (p + 1) * case["page"])
                rows = slice(lo - p * case["page"], hi - p * case["page"])
                s["k_pages"][table[p], :, rows] = s["k"][b, :, lo - start:hi - start]
                s["v_pages"][table[p], :, rows] = s["v"][b, :, lo - start:hi - start]
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if op == "order":
        return None                       # whole numbers: equal to the plain form's or wrong
    out, rowsum = s["out"].double(), s["rowsum"].double()
    for b, (start, cnt) in enumerate(_lengths(case)):
        end = start + cnt
        if cnt == 0:
            continue
        keys = _sequence(s["k_pages"], s["table"][b], end)
        vals = _sequence(s["v_pages"], s["table"][b], end).double()
        z = _curve(keys, case["bits"])
        zq = _curve(s["q"][b], case["bits"])
        kd, qd = keys.double(), s["q"][b].double()
        g2 = s["gamma"].double()[:, None, None] ** 2
        for c in range(start // C, (end - 1) // C + 1):
            i = torch.arange(max(start, c * C), min(end, (c + 1) * C), device="cuda")
            row = i - start
            j = torch.arange(c * C, int(i[-1]) + 1, device="cuda")
            dist = sum((qd[:, row, None, x] - kd[:, None, j, x]) ** 2 for x in range(case["dK"]))
            dist = dist.masked_fill((j > i[:, None])[None], math.inf)
            if c:
                zs, by = z[:, :c * C].sort(dim=1, stable=True)
                r = torch.searchsorted(zs, zq[:, row].contiguous(), side="right")
                lo = (r - (k + 1) // 2).clamp(0, c * C - k)
                win = torch.stack([by[x][lo[x][:, None] + torch.arange(k, device="cuda")]
                                   for x in range(by.shape[0])])            # [H, rows, k]
                near = torch.stack([kd[x][win[x]] for x in range(by.shape[0])])
                dw = ((qd[:, row][:, :, None] - near) ** 2).sum(-1)
                near_v = torch.stack([vals[x][win[x]] for x in range(by.shape[0])])
            else:
                dw, near_v = dist[:, :, :0], vals[:, None, :0].expand(-1, len(row), -1, -1)
            both = torch.cat([dist, dw], 2)
            if case["weight"] == "cauchy":
                w = g2 / (g2 + both)
                w = torch.where(torch.isinf(both), 0.0, w)
            elif case["weight"] == "softmax":
                w = torch.exp(-(both - both.min(2, keepdim=True).values) / g2)
            else:
                w = 1 / torch.sqrt(both + 1e-12)
            total = w.sum(2)
            o = torch.einsum("hqj,hjd->hqd", w[:, :, :len(j)], vals[:, j])
            o = o + torch.einsum("hqk,hqkd->hqd", w[:, :, len(j):], near_v)
            out[b][:, row] = o / total[..., None]
            rowsum[b][:, row] = total
    return {"out": out, "rowsum": rowsum}
