"""User-facing API: run the whole ZETA hot path through the C ABI.

``ZetaPlan`` owns the device buffers of one problem size (codes, prefix table,
workspaces, outputs) so that repeated steps allocate nothing.  ``forward`` and
``backward`` enqueue the five library calls on the current stream;
``ZetaAttention`` wraps them as a torch.autograd.Function (selection is not
differentiated).  All arithmetic runs in the library's CUDA kernels.

With ``curves`` = 3 or 6 the plan follows the multi-curve variant (the keys
are indexed along the cyclic shifts, or all orderings, of the three
coordinates and every curve contributes k // curves keys): the codes and
prefix tables gain a leading curve dimension, one sort call covers every
curve, and the union of the windows feeds the same attend kernels.

``ZetaCache`` serves a trained model: keys and values of many sequences in
pages, new tokens appended and attended in batches of up to C per sequence.
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as zb

_C, _F32, _I32 = torch._C, torch.float32, torch.int32


class ZetaPlan:
    def __init__(self, p: zb.zeta_problem_t, device="cuda", backward: bool = True,
                 curves: int = 1, fused: bool = False):
        """fused: select and attend in one call (zeta_select_attend_fwd); one
        curve only."""
        if fused and curves != 1:
            raise ValueError("the fused select + attend call takes one curve")
        self.p = p
        self.curves = curves
        self.fused = fused
        self.axes = zb.curve_axes(p.d_K, curves)
        # Every curve's slices sort as one problem with curves*B batches.
        self.p_sort = zb.problem(p.B * curves, p.H, p.N, p.d_K, p.d_V, p.k, p.C, p.bits,
                                 p.v_dtype, flags=p.flags) if curves > 1 else p
        dev = torch.device(device)
        S = p.B * p.H
        N = p.N
        cdt = zb.code_dtype(p)
        vdt = zb.v_torch_dtype(p)
        T = zb.zeta_prefix_entries(p)
        if T < 0:
            raise zb.ZetaError("zeta_prefix_entries", 1)
        self.T = T
        G = curves * S
        self.q_codes = torch.empty(G * N, dtype=cdt, device=dev)
        self.k_codes = torch.empty(G * N, dtype=cdt, device=dev)
        self.prefix_codes = torch.empty(max(G * T, 1), dtype=cdt, device=dev)[: G * T]
        self.prefix_idx = torch.empty(max(G * T, 1), dtype=torch.int32, device=dev)[: G * T]
        self.sort_ws = torch.empty(max(zb.zeta_sort_workspace_bytes(self.p_sort), 256),
                                   dtype=torch.uint8, device=dev)
        self.idx = torch.empty(S * N * p.k, dtype=torch.int32, device=dev)
        self.out = torch.empty(S * N * p.d_V, dtype=vdt, device=dev)
        self.rowsum = torch.empty(S * N, dtype=torch.float32, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.has_bwd = backward
        if backward:
            self.bwd_ws = torch.empty(max(zb.zeta_bwd_workspace_bytes(p), 256),
                                      dtype=torch.uint8, device=dev)
            self.dq = torch.empty(S * N * p.d_K, dtype=torch.float32, device=dev)
            self.dk = torch.empty(S * N * p.d_K, dtype=torch.float32, device=dev)
            self.dv = torch.empty(S * N * p.d_V, dtype=vdt, device=dev)
            self.dgamma = torch.empty(p.H, dtype=torch.float32, device=dev)

    def forward(self, q, k, v, gamma, stream=None):
        """Encode, sort, select, attend.  Returns (out, rowsum, idx) views."""
        p = self.p
        if self.curves == 1:
            zb.zeta_encode(p, q, self.q_codes, stream)
            zb.zeta_encode(p, k, self.k_codes, stream)
        else:
            zb.zeta_encode_curves(p, q, self.axes, self.q_codes, stream)
            zb.zeta_encode_curves(p, k, self.axes, self.k_codes, stream)
        zb.zeta_sort_chunks(self.p_sort, self.k_codes, self.prefix_codes, self.prefix_idx,
                            self.sort_ws, stream)
        if self.fused:
            zb.zeta_select_attend_fwd(p, q, k, v, gamma, self.q_codes, self.prefix_codes,
                                      self.prefix_idx, self.idx, self.out, self.rowsum,
                                      self.status, stream)
            return self.out, self.rowsum, self.idx
        if self.curves == 1:
            zb.zeta_select_topk(p, self.q_codes, self.prefix_codes, self.prefix_idx, self.idx,
                                stream)
        else:
            zb.zeta_select_topk_curves(p, self.curves, self.q_codes, self.prefix_codes,
                                       self.prefix_idx, self.idx, stream)
        zb.zeta_attend_fwd(p, q, k, v, gamma, self.idx, self.out, self.rowsum, self.status,
                           stream)
        return self.out, self.rowsum, self.idx

    def backward(self, q, k, v, gamma, dout, stream=None):
        """Gradients for the last forward.  Returns (dq, dk, dv, dgamma) views."""
        p = self.p
        zb.zeta_attend_bwd(p, q, k, v, gamma, self.idx, dout, self.dq, self.dk, self.dv,
                           self.dgamma, self.bwd_ws, self.status, stream)
        return self.dq, self.dk, self.dv, self.dgamma


class ZetaAttention(torch.autograd.Function):
    """out = ZETA attention(q, k, v, gamma); q, k [B,H,N,d_K] f32, v [B,H,N,d_V]."""

    @staticmethod
    def forward(ctx, q, k, v, gamma, C: int, k_sel: int, bits: int, curves: int = 1,
                weight: str = "cauchy"):
        B, H, N, d_K = q.shape
        d_V = v.shape[-1]
        vd = "bf16" if v.dtype == torch.bfloat16 else "f32"
        p = zb.problem(B, H, N, d_K, d_V, k_sel, C, bits, vd, weight=weight)
        plan = ZetaPlan(p, q.device, curves=curves)
        q, k, v, gamma = (t.contiguous() for t in (q, k, v, gamma))
        out, _, _ = plan.forward(q, k, v, gamma)
        ctx.plan = plan
        ctx.save_for_backward(q, k, v, gamma)
        return out.view(B, H, N, d_V).clone()

    @staticmethod
    def backward(ctx, dout):
        q, k, v, gamma = ctx.saved_tensors
        dq, dk, dv, dg = ctx.plan.backward(q, k, v, gamma, dout.contiguous().to(v.dtype))
        return (dq.view_as(q).clone(), dk.view_as(k).clone(), dv.view_as(v).clone(),
                dg.clone(), None, None, None, None, None)


def zeta_attention(q, k, v, gamma, C: int, k_sel: int, bits: int = 10, curves: int = 1,
                   weight: str = "cauchy"):
    """weight: 'cauchy' (the method), 'softmax' (of -|q-k|^2/gamma^2) or
    'inv_euclid' (1/|q-k|); see zeta_weight_t in include/zeta.h."""
    return ZetaAttention.apply(q, k, v, gamma, C, k_sel, bits, curves, weight)


class ZetaCache:
    """Paged key/value cache: the three serving calls on one set of pools.

    k_pages f32 [pages, H, page, d_K], v_pages [pages, H, page, d_V],
    order_codes (the problem's code type) and order_idx (int32)
    [2, order_pages, H, page]; ``empty`` allocates them.  N: the longest
    sequence (a multiple of C); C, k, bits, weight as for ``zeta_attention`` with one
    curve (selections over several curves have no cached form).

    Tables are int32 [B, table_len]: token t of sequence b is row t % page of page
    table[b, t // page]; which pages a sequence gets is the caller's business.
    Per step and batch, with the same start and count (int32 [B], tokens before
    the step and tokens brought, count <= n <= C; n is the rows of k, v and q)::

        cache.append(k, v, start, count, table)
        cache.order(start, count, table, n=n)     # when a sequence completes a chunk
        cache.attend(q, gamma, start, count, table, out, rowsum)

    Drafted tokens, a tree of up to n nodes per sequence (parent int32 [B, n], -1 at the
    top), whose keys and values stay in k and v until a line of them is accepted::

        longest = torch.minimum(longest, C - start % C)      # a line ends with its chunk
        cache.reserve(start, longest, table, held, free, free_count, granted)
        cache.attend_tree(q, k, v, gamma, start, count, parent, table, out, rowsum)
        cache.accept(k, v, start, count, parent, leaf, table, accepted, granted=granted)
        cache.order(start, accepted, table, n=n)

    longest (int32 [B], 0 where count is 0): tokens of the longest line that may be accepted.
    Where the free list was too short for a sequence, granted is 0 and so is accepted: nothing
    counts as a token that has no page.

    The prefixes of completed chunks are kept in the order pools through
    order_table (default: table; pass another one when sequences share K/V pages).
    Everything is enqueued on the given or current stream and allocates nothing,
    so a step can be captured into a CUDA graph.  Weights and sums are float32; for bf16
    values large calls of attend take the weights of a row's own chunk as two bf16 parts (within
    2^-16), so that a token's outputs in calls of different sizes agree to one step of bf16;
    attend_tree keeps all of a weight's bits.  Findings of the kernels (a length or page out of
    range) go to ``status``, one int32 word, unless dev_status is given.  There is no backward.
    Pools and sizes are those the cache was made with: they cannot be assigned, and a pool whose
    memory changes in place is taken as it then lies, or refused where it no longer fits.
    """

    _lib = None                          # set last; from then on these stay as they are
    _FIXED = frozenset(("k_pages", "v_pages", "order_codes", "order_idx", "status", "pages",
                        "order_pages", "page", "H", "d_K", "d_V", "N", "C", "k", "bits", "flags",
                        "v_dtype", "device"))

    def __init__(self, k_pages, v_pages, order_codes, order_idx, N: int, C: int, k: int,
                 bits: int = 10, weight: str = "cauchy"):
        if k_pages.dim() != 4 or v_pages.dim() != 4 or k_pages.shape[:3] != v_pages.shape[:3]:
            raise ValueError("k_pages and v_pages must be [pages, H, page, d] of the same pages")
        if order_codes.dim() != 4:
            raise ValueError("order_codes must be [2, order_pages, H, page]")
        self.pages, self.H, self.page, self.d_K = k_pages.shape
        self.d_V = v_pages.shape[3]
        if v_pages.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError(f"v_pages: dtype {v_pages.dtype}, expected bfloat16 or float32")
        self.v_dtype = zb.ZETA_BF16 if v_pages.dtype == torch.bfloat16 else zb.ZETA_F32
        self.N, self.C, self.k, self.bits = N, C, k, bits
        self.flags = zb.WEIGHTS[weight]
        p = self._problem(1)
        if zb.zeta_code_bytes(p) == 0:
            raise zb.ZetaError("zeta_code_bytes", 1)
        shape = (2, order_codes.shape[1], self.H, self.page)
        self.order_pages = order_codes.shape[1]
        self.device = k_pages.device
        if self.device.type != "cuda":
            raise ValueError("ZETA tensors must be CUDA tensors")
        self._index = self.device.index
        self._vt = v_pages.dtype
        self.k_pages, self.v_pages = k_pages, v_pages
        self.order_codes, self.order_idx = order_codes, order_idx
        self.status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._pools = ((k_pages, "k_pages", torch.float32, tuple(k_pages.shape)),
                       (v_pages, "v_pages", self._vt, tuple(v_pages.shape)),
                       (order_codes, "order_codes", zb.code_dtype(p), shape),
                       (order_idx, "order_idx", torch.int32, shape),
                       (self.status, "status", torch.int32, (1,)))
        self._where = tuple(t.data_ptr for t, *_ in self._pools)
        self._ptrs = tuple(self._take(*x) for x in self._pools)
        self._heads = (self.H,)
        self._structs = {}
        self._lib = zb.lib()

    def __setattr__(self, name, value):
        # The structs of earlier calls and captured graphs hold the pools and sizes.
        if name in self._FIXED and self._lib is not None:
            raise AttributeError(f"{name}: a ZetaCache keeps the pools and sizes it was made "
                                 "with; make another one")
        super().__setattr__(name, value)

    def _memory(self):
        """Pointers of the four pools and the status word as they lie now; checked anew where
        one has moved."""
        a, b, c, d, e = self._where
        now = a(), b(), c(), d(), e()
        return now if now == self._ptrs else tuple(self._take(*x) for x in self._pools)

    @classmethod
    def empty(cls, pages: int, page: int, H: int, d_K: int, d_V: int, N: int, C: int, k: int,
              bits: int = 10, v_dtype=torch.bfloat16, weight: str = "cauchy", device="cuda",
              order_pages: int | None = None):
        """A cache with pools of its own (order_pages defaults to pages)."""
        op = pages if order_pages is None else order_pages
        ct = torch.int64 if d_K * bits > 32 else torch.int32
        return cls(torch.zeros(pages, H, page, d_K, device=device),
                   torch.zeros(pages, H, page, d_V, dtype=v_dtype, device=device),
                   torch.zeros(2, op, H, page, dtype=ct, device=device),
                   torch.zeros(2, op, H, page, dtype=torch.int32, device=device),
                   N, C, k, bits, weight)

    def _problem(self, B: int) -> zb.zeta_problem_t:
        return zb.zeta_problem_t(B, self.H, self.N, self.d_K, self.d_V, self.k, self.C, self.bits,
                                 self.v_dtype, self.flags)

    def _sizes(self, B: int, n: int, width: int):
        """References to the C structs of a batch size and the shapes its tensors have
        ([B], [B,H,n], [B,H,n,d_K], [B,H,n,d_V], [B,H,n,k]), made once per (B, n, width) and
        never changed (a step costs the host a few microseconds, of which building them
        would be a good part)."""
        got = self._structs.get((B, n, width))
        if got is None:
            if len(self._structs) >= 1024:
                self._structs.clear()
            rows = (B, self.H, n)
            got = (ctypes.byref(self._problem(B)),
                   ctypes.byref(zb.zeta_cache_t(n, self.page, self.pages, self.order_pages,
                                                width)),
                   (B,), rows, (*rows, self.d_K), (*rows, self.d_V), (*rows, self.k))
            self._structs[B, n, width] = got
        return got

    def _take(self, t, name, dtype, shape):
        """Pointer of a tensor of the given type, shape and the cache's device."""
        if (t.dtype is dtype and t.shape == shape and t.get_device() == self._index
                and t.is_contiguous() and not t.requires_grad):
            return t.data_ptr()
        if t.dtype is not dtype:
            raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
        if t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
        if t.device != self.device:
            raise ValueError(f"{name}: on {t.device}, the cache is on {self.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name}: ZETA tensors must be contiguous")
        if torch.is_grad_enabled():
            raise ValueError(f"{name}: the cache calls have no backward (use torch.no_grad)")
        return t.data_ptr()

    def _table(self, t):
        """Pointer and both sizes of a page table."""
        shape = t.shape
        if len(shape) != 2:
            raise ValueError(f"page_table: {t.dim()} dimensions, expected 2")
        if (t.dtype is _I32 and t.get_device() == self._index and t.is_contiguous()
                and not t.requires_grad):
            return t.data_ptr(), *shape
        return self._take(t, "page_table", _I32, shape), *shape

    @staticmethod
    def _rows(t, name):
        try:
            return t.shape[2]
        except IndexError:
            raise ValueError(f"{name}: {t.dim()} dimensions, expected 4") from None

    def _call(self, f, args, status, dev_status, stream):
        st = status if dev_status is None else self._take(dev_status, "dev_status", _I32, (1,))
        if stream is None:
            stream = _C._cuda_getCurrentRawStream(self._index)
        elif not isinstance(stream, int):
            stream = stream.cuda_stream
        if _C._cuda_getDevice() == self._index:
            code = f(*args, st, stream)
        else:
            with torch.cuda.device(self._index):
                code = f(*args, st, stream)
        if code != 0:
            raise zb.ZetaError(f.__name__, code)

    def append(self, k, v, start, count, page_table, dev_status=None, stream=None):
        """k f32 [B,H,n,d_K], v [B,H,n,d_V]: rows 0 .. count[b]-1 of sequence b become its
        tokens start[b] .. start[b]+count[b]-1."""
        tp, B, width = self._table(page_table)
        p, c, per_seq, _, k_shape, v_shape, _ = self._sizes(B, self._rows(k, "k"), width)
        take = self._take
        kp, vp, _, _, st = self._memory()
        self._call(self._lib.zeta_cache_append,
                   (p, c, take(k, "k", _F32, k_shape), take(v, "v", self._vt, v_shape),
                    take(start, "start", _I32, per_seq), take(count, "count", _I32, per_seq),
                    tp, kp, vp), st, dev_status, stream)

    def order(self, start, count, page_table, order_table=None, dev_status=None, stream=None,
              n=None):
        """The sorted prefix of every sequence that completes a chunk with these tokens.  n: the
        step's rows per sequence (default C, the most there can be); a sequence that brings
        more of them than that is skipped, as append and attend skip it."""
        tp, B, width = self._table(page_table)
        p, c, per_seq, *_ = self._sizes(B, self.C if n is None else n, width)
        take = self._take
        op = tp if order_table is None else take(order_table, "order_table", _I32, (B, width))
        kp, _, ocp, oip, st = self._memory()
        self._call(self._lib.zeta_cache_order,
                   (p, c, take(start, "start", _I32, per_seq), take(count, "count", _I32, per_seq),
                    tp, kp, op, ocp, oip), st, dev_status, stream)

    def attend(self, q, gamma, start, count, page_table, out, rowsum, order_table=None, idx=None,
               dev_status=None, stream=None):
        """q f32 [B,H,n,d_K], gamma f32 [H] -> out [B,H,n,d_V], rowsum f32 [B,H,n] and, where
        given, idx int32 [B,H,n,k]; rows count[b] .. n-1 stay as they were."""
        tp, B, width = self._table(page_table)
        p, c, per_seq, rows, q_shape, v_shape, i_shape = self._sizes(B, self._rows(q, "q"), width)
        take = self._take
        op = tp if order_table is None else take(order_table, "order_table", _I32, (B, width))
        kp, vp, ocp, oip, st = self._memory()
        self._call(self._lib.zeta_cache_attend,
                   (p, c, take(q, "q", _F32, q_shape), take(gamma, "gamma", _F32, self._heads),
                    take(start, "start", _I32, per_seq), take(count, "count", _I32, per_seq),
                    tp, kp, vp, op, ocp, oip, take(out, "out", self._vt, v_shape),
                    take(rowsum, "rowsum", _F32, rows),
                    None if idx is None else take(idx, "idx", _I32, i_shape)),
                   st, dev_status, stream)

    def attend_tree(self, q, k, v, gamma, start, count, parent, page_table, out, rowsum,
                    order_table=None, idx=None, dev_status=None, stream=None):
        """Drafted nodes over the cache and their lines: q, k f32 [B,H,n,d_K], v [B,H,n,d_V],
        parent int32 [B,n] (parent[b,t] < t, -1: below the sequence's last token) -> out
        [B,H,n,d_V], rowsum f32 [B,H,n] and, where given, idx int32 [B,H,n,k].  Rows from
        count[b] on and of nodes behind the end of the chunk that start[b] lies in stay as they
        were.  n <= 1024."""
        tp, B, width = self._table(page_table)
        n = self._rows(q, "q")
        p, c, per_seq, rows, q_shape, v_shape, i_shape = self._sizes(B, n, width)
        take = self._take
        op = tp if order_table is None else take(order_table, "order_table", _I32, (B, width))
        kp, vp, ocp, oip, st = self._memory()
        self._call(self._lib.zeta_cache_attend_tree,
                   (p, c, take(q, "q", _F32, q_shape), take(k, "k", _F32, q_shape),
                    take(v, "v", self._vt, v_shape), take(gamma, "gamma", _F32, self._heads),
                    take(start, "start", _I32, per_seq), take(count, "count", _I32, per_seq),
                    take(parent, "parent", _I32, (B, n)), tp, kp, vp, op, ocp, oip,
                    take(out, "out", self._vt, v_shape), take(rowsum, "rowsum", _F32, rows),
                    None if idx is None else take(idx, "idx", _I32, i_shape)),
                   st, dev_status, stream)

    def accept(self, k, v, start, count, parent, leaf, page_table, accepted, path=None,
               dev_status=None, stream=None, granted=None):
        """The line of nodes that ends in leaf int32 [B] (-1: none) becomes the sequence's next
        tokens, up to the end of the chunk that start[b] lies in and, where granted int32 [B] (of
        ``reserve``) is given, at most granted[b] of them; accepted int32 [B] gets how many, path
        int32 [B,n], where given, their nodes (-1 behind them).  Without granted the line's tokens
        must have their pages: one that has none is counted, but stored nowhere (``status``)."""
        tp, B, width = self._table(page_table)
        n = self._rows(k, "k")
        p, c, per_seq, _, k_shape, v_shape, _ = self._sizes(B, n, width)
        take = self._take
        kp, vp, _, _, st = self._memory()
        f, cap = self._lib.zeta_cache_accept, ()
        if granted is not None:
            f, cap = self._lib.zeta_cache_accept_granted, (take(granted, "granted", _I32, per_seq),)
        self._call(f, (p, c, take(k, "k", _F32, k_shape), take(v, "v", self._vt, v_shape),
                       take(start, "start", _I32, per_seq), take(count, "count", _I32, per_seq),
                       take(parent, "parent", _I32, (B, n)), take(leaf, "leaf", _I32, per_seq),
                       *cap, tp, kp, vp, take(accepted, "accepted", _I32, per_seq),
                       None if path is None else take(path, "path", _I32, (B, n))),
                   st, dev_status, stream)

    def reserve(self, start, count, page_table, held, free, free_count, granted, slots=None,
                dev_status=None, stream=None, n=None):
        """Sequence b is given or gives back pages until it holds those of its start[b] + count[b]
        tokens: page_table, held int32 [B] (pages it holds), free int32 [pages] (places
        [0, free_count) are the free pages) and free_count int32 [1] change in place.  granted
        int32 [B] gets count[b], or 0 where the list was too short; slots int32 [B,n], where
        given, the row number of every new token.  n: the step's rows (default: those of slots,
        or C).  start[b] + count[b] <= N: of a draft, the tokens of its longest line up to the
        chunk's end (``accept`` takes granted)."""
        tp, B, width = self._table(page_table)
        if slots is not None and slots.dim() != 2:
            raise ValueError(f"slots: {slots.dim()} dimensions, expected 2")
        if n is None:
            n = self.C if slots is None else slots.shape[1]
        p, c, per_seq, *_ = self._sizes(B, n, width)
        take = self._take
        st = self._memory()[4]
        self._call(self._lib.zeta_cache_reserve,
                   (p, c, take(start, "start", _I32, per_seq), take(count, "count", _I32, per_seq),
                    tp, take(held, "held", _I32, per_seq), take(free, "free", _I32, (self.pages,)),
                    take(free_count, "free_count", _I32, (1,)),
                    take(granted, "granted", _I32, per_seq),
                    None if slots is None else take(slots, "slots", _I32, (B, n))),
                   st, dev_status, stream)
