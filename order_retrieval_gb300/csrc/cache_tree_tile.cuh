// cache_tree_tile.cuh -- attention of trees of drafted tokens: bf16 values with d_V a
// multiple of 8, float32 with a multiple of 4, up to 128 wide, d_K <= 4.
//
// Same definition as the row kernel (cache_tree.cu).  A block of four warps takes 16
// nodes of one sequence and head, or a cluster of 2 or 4 blocks does where there are few:
// every block of it has some of the nodes' windows and some of the keys that all 16 share,
// and the sums are joined through distributed shared memory.
//  * Lines: a bit per node above, found by climbing in shared memory.  A run of nodes
//    that hang below one another by number (a chain) is one step of the climb.
//  * Window: a warp takes two nodes at a time.  The first code of every block of 2^fsh
//    prefix entries lies in shared memory; a warp counts there and among the block's
//    entries, looks up and weighs the entries a lane each and streams their value rows.
//  * The sequence's tokens of the chunk and the nodes are one list of keys, staged by
//    cp.async in tiles; a warp takes a quarter of each.  bf16: weights are built in mma A
//    fragments, as a bf16 half and the bf16 of what that leaves (within 2^-16 together).
//    float32: weights through shared memory, then a thread sums 4 nodes x 8 (16) columns.
//  * A masked weight of zero times a value that is not finite is NaN: a node whose result
//    is not finite is taken again, key by key, without the others.
#pragma once

#include <cooperative_groups.h>

#include "cache_tile.cuh"
#include "cache_tree.cuh"

namespace zeta {

// cs: blocks a group of 16 nodes (1, 2 or 4).
cudaError_t launch_tree_tile_bf16(const Prob &p, const TreeArgs &g, int cs, cudaStream_t st);
cudaError_t launch_tree_tile_f32(const Prob &p, const TreeArgs &g, int cs, cudaStream_t st);

namespace {

namespace cg = cooperative_groups;

constexpr int kTreeWarps = 4, kTreeThreads = 32 * kTreeWarps, kTreeRows = 16;
constexpr int kTreeFences = 256;
constexpr int kNoRow = INT32_MIN;

template <typename V, int DVP>
struct TreeSmem {
    static constexpr bool MMA = sizeof(V) == 2;
    static constexpr int TK = MMA ? 64 : 32;         // keys a tile
    union {
        struct {
            V v[3][TK * DVP];                        // bf16: 16-byte piece c of row r at c ^ (r & 7)
            float k[3][4][TK];                       // coordinates apart
        } own;
        float part[kTreeWarps][kTreeRows][DVP + 4];  // the warps' sums
    };
    uint64_t fence[kTreeFences];
    struct {                                         // a warp's two nodes
        float w[kTreeWarps][2][64];
        int row[kTreeWarps][2][64];
    } gather;
    float w[MMA ? 1 : kTreeWarps][8][20];            // float32: weights [key][node]
    union {
        int parent[kMaxDraft];
        float win[kTreeRows][DVP + 4];               // window sums
    };
    uint32_t run[kMaxDraft / 32];                    // bit u: parent[u] == u - 1
    uint32_t above[kTreeRows][kMaxDraft / 32];       // nodes of a line
    int rows[4][TK];                                 // pool rows of the tile's keys, ~node, kNoRow
    float q[kTreeRows][4];
    int depth[kTreeRows], wst[kTreeRows];
    float swin[kTreeRows], mwin[kTreeRows];
    float psum[kTreeWarps][kTreeRows], pmin[kTreeWarps][kTreeRows];
};

// The line of node t as bits of `above` (words of `run` read from the top one down);
// its depth, -1 where a parent is no earlier node.
__device__ __forceinline__ int climb_bits(const int *parent, const uint32_t *run, int t,
                                          uint32_t *above) {
    int depth = -1;
    while (t >= 0) {
        const int w = t >> 5;
        const uint32_t upto = 0xffffffffu >> (31 - (t & 31));
        const uint32_t ends = ~run[w] & upto;        // nodes whose parent is not the one before
        const int s = ends ? 31 - __clz(ends) : 0;
        const uint32_t part = upto & (0xffffffffu << s);
        above[w] |= part;
        depth += __popc(part);
        const int top = w * 32 + s, p = ends ? parent[top] : top - 1;
        if (p < -1 || p >= top) return -1;
        t = p;
    }
    return depth;
}

// Values of a 16-byte piece as pairs, times f, onto acc.
template <typename V>
__device__ __forceinline__ void add_piece(float2 (&acc)[8 / sizeof(V)], const uint4 &x, float f) {
    const float2 ff = dup2(f);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    if constexpr (sizeof(V) == 2) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
            acc[c] = fma2(ff, make_float2(__uint_as_float(w[c] << 16), __uint_as_float(w[c] & 0xffff0000u)), acc[c]);
    } else {
#pragma unroll
        for (int c = 0; c < 2; ++c)
            acc[c] = fma2(ff, make_float2(__uint_as_float(w[2 * c]), __uint_as_float(w[2 * c + 1])), acc[c]);
    }
}

// One node key by key (a warp, lanes over the value columns).
template <typename V, int DVP, int DK, int WK>
__device__ __noinline__ void slow_node(const TreeArgs &g, int64_t rid, int b, int h, int start,
                                       int first, const uint32_t *above, float inv_g2) {
    const int lane = threadIdx.x & 31, cC = start / g.C * g.C;
    const int32_t *ptab = g.c.ptab + (int64_t)b * g.c.tlen, *otab = g.c.otab + (int64_t)b * g.c.tlen;
    const int64_t plane = ((int64_t)g.c.opages * g.H << g.c.psh) * (start / g.C & 1);
    const int64_t node0 = ((int64_t)b * g.H + h) * g.c.n;
    const int t = (int)(rid - node0);
    const float4 q4 = ld_key(g.q + rid * g.dK, g.dK);
    const float q[4] = {q4.x, q4.y, q4.z, q4.w};
    const int nw = cC > 0 ? g.kw : 0, own = start - cC;
    float acc[DVP / 32], s = 0.f, m = INFINITY;
#pragma unroll
    for (int e = 0; e < DVP / 32; ++e) acc[e] = 0.f;
    for (int pass = WK == kWSoftmax ? 0 : 1; pass < 2; ++pass) {
        for (int x = 0; x < nw + own + t + 1; ++x) {
            const float *kp;
            const V *vp;
            if (x >= nw + own) {
                const int u = x - nw - own;
                if (!(above[u >> 5] >> (u & 31) & 1u)) continue;
                kp = g.k + (node0 + u) * g.dK;
                vp = static_cast<const V *>(g.v) + (node0 + u) * g.dV;
            } else {
                int j = cC + x - nw;
                if (x < nw) {
                    const int row = page_row(otab, first + x, h, g.H, g.c.psh, g.c.pmask, g.c.opages);
                    j = row >= 0 ? g.order_idx[plane + row] : -1;
                    if ((unsigned)j >= (unsigned)cC) continue;
                }
                const int row = page_row(ptab, j, h, g.H, g.c.psh, g.c.pmask, g.c.pages);
                if (row < 0) continue;
                kp = g.k_pages + (int64_t)row * g.dK;
                vp = static_cast<const V *>(g.v_pages) + (int64_t)row * g.dV;
            }
            const float4 k4 = ld_key(kp, g.dK);
            const float kc[4] = {k4.x, k4.y, k4.z, k4.w};
            float d2 = 0.f;
#pragma unroll
            for (int d = 0; d < DK; ++d) {
                const float e = q[d] - kc[d];
                d2 = __fmaf_rn(e, e, d2);
            }
            if (pass == 0) {
                m = fminf(m, d2);
                continue;
            }
            const float w = weight_fast<WK>(d2, m, inv_g2);
            s += w;
#pragma unroll
            for (int e = 0; e < DVP / 32; ++e)
                if (lane + 32 * e < g.dV) acc[e] = __fmaf_rn(w, VT<V>::ld(vp + lane + 32 * e), acc[e]);
        }
    }
    V *o = static_cast<V *>(g.out) + rid * g.dV;
#pragma unroll
    for (int e = 0; e < DVP / 32; ++e)
        if (lane + 32 * e < g.dV) VT<V>::st(o + lane + 32 * e, __fdiv_rn(acc[e], s));
}

template <typename V, int DVP, int DK, int WK>
__global__ void __launch_bounds__(kTreeThreads, 4)
tree_tile_kernel(const __grid_constant__ TreeArgs g, int cs) {
    using Sm = TreeSmem<V, DVP>;
    constexpr int TK = Sm::TK, NT = kTreeThreads, NW = kTreeWarps;
    constexpr int PPR = DVP * (int)sizeof(V) / 16;           // 16-byte pieces of a padded row
    constexpr int NP = 8 / (int)sizeof(V);                   // pairs of a piece
    extern __shared__ __align__(16) unsigned char raw[];
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cr = cs == 1 ? 0 : (int)(blockIdx.x % (unsigned)cs);   // block in the cluster
    const int f0 = (int)(blockIdx.x / (unsigned)cs) * kTreeRows;     // first node
    const int s = blockIdx.y, b = s / g.H, h = s - b * g.H;
    const Seq seq = drafts_of(g.c, b, g.N, g.status);
    if (f0 >= seq.count) return;                             // the whole cluster returns
    const int nn = min(f0 + kTreeRows, seq.count), nq = nn - f0;
    const int chunk = seq.start / g.C, cC = chunk * g.C, L = seq.start - cC;
    const int32_t *ptab = g.c.ptab + (int64_t)b * g.c.tlen, *otab = g.c.otab + (int64_t)b * g.c.tlen;
    const int64_t node0 = (int64_t)s * g.c.n;                // the slice's node 0
    const V *pool = static_cast<const V *>(g.v_pages);
    const V *fresh = static_cast<const V *>(g.v) + node0 * g.dV;
    const float gm = __ldg(g.gamma + h);
    const float inv_g2 = __frcp_rn(gm * gm);
    const int64_t plane = ((int64_t)g.c.opages * g.H << g.c.psh) * (chunk & 1);
    const int ppr = g.dV * (int)sizeof(V) / 16;
    auto order_row = [&](int id, int e) { return row_in(id, e, h, g.H, g.c.psh, g.c.pmask, g.c.opages); };
    auto pool_row = [&](int id, int t) { return row_in(id, t, h, g.H, g.c.psh, g.c.pmask, g.c.pages); };
    auto order_code = [&](int64_t at) -> uint64_t {
        return g.code64 ? __ldg(static_cast<const unsigned long long *>(g.order_codes) + at)
                        : (uint64_t)__ldg(static_cast<const uint32_t *>(g.order_codes) + at);
    };

    // ------------------------------------------------------------ set-up ---
    // Shared keys x: the chunk's L tokens, then the nodes up to the block's last one; the
    // block takes tiles cr, cr + cs, ...
    const int keys = L + nn, tiles = (keys + TK - 1) / TK;
    const int mine = cr < tiles ? (tiles - cr + cs - 1) / cs : 0;
    auto ask_row = [&](int i) {                              // page of the thread's key of its tile i
        const int x = (cr + i * cs) * TK + tid;
        return tid < TK && x < L ? page_id(ptab, cC + x, g.c.psh) : -1;
    };
    bool lost_key = false;                                   // this thread met a key without a page
    auto put_row = [&](int i, int id) {
        const int x = (cr + i * cs) * TK + tid;
        if (tid < TK && i < mine) {
            int row = kNoRow;
            if (x < L) {
                row = pool_row(id, cC + x);
                if (row < 0) {
                    set_status(g.status, ZETA_ERR_BOUNDS);
                    lost_key = true;
                    row = kNoRow;
                }
            } else if (x < keys) {
                row = ~(x - L);
            }
            sm.rows[i & 3][tid] = row;
        }
        __syncwarp();                                        // one branch again before the products
    };
    auto load_tile = [&](int i) {                            // into stage i % 3, asynchronously
        if (i < mine) {
            const int bf = i % 3;
            const int *rows = sm.rows[i & 3];
#pragma unroll
            for (int u = 0; u < TK * PPR / NT; ++u) {
                const int id = u * NT + tid;
                const int row = id / PPR, ch = id % PPR;
                if (ch < ppr) {
                    const int pr = rows[row];
                    const V *src = pr >= 0 ? pool + (int64_t)pr * g.dV : fresh + (int64_t)(pr == kNoRow ? 0 : ~pr) * g.dV;
                    const int at = Sm::MMA ? ch ^ (row & 7) : ch;
                    cp_async16(smem_u32(&sm.own.v[bf][row * DVP + at * (16 / (int)sizeof(V))]),
                               src + ch * (16 / (int)sizeof(V)), pr == kNoRow ? 0 : 16);
                }
            }
            for (int id = tid; id < TK * DK; id += NT) {
                const int d = id / TK, row = id % TK;
                const int pr = rows[row];
                const bool ok = pr != kNoRow && d < g.dK;
                const float *src = pr >= 0 ? g.k_pages + (int64_t)pr * g.dK : g.k + (node0 + ~pr) * g.dK;
                cp_async4(smem_u32(&sm.own.k[bf][d][row]), ok ? src + d : g.k_pages, ok ? 4 : 0);
            }
        }
        cp_async_commit();
    };
    {
        const int i0 = ask_row(0), i1 = ask_row(1), i2 = ask_row(2);
        for (int u = tid; u < nn; u += NT) sm.parent[u] = __ldg(g.parent + (int64_t)b * g.c.n + u);
        if (tid < kTreeRows * 4) {
            const int r = tid >> 2, d = tid & 3;
            sm.q[r][d] = r < nq && d < g.dK ? __ldg(g.q + (node0 + f0 + r) * g.dK + d) : 0.f;
        }
        for (int e = tid; e < kTreeRows * (kMaxDraft / 32); e += NT) (&sm.above[0][0])[e] = 0u;
        put_row(0, i0);
        put_row(1, i1);
        put_row(2, i2);
    }
    int kid = ask_row(3);
    __syncthreads();
    load_tile(0);
    load_tile(1);
    int fsh = 5;
    while ((cC >> fsh) >= kTreeFences) ++fsh;
    const int nf = (cC + (1 << fsh) - 1) >> fsh;
    if (chunk > 0) {
        constexpr int NF = kTreeFences / NT;
        int fr[NF];
        uint64_t fz[NF];
#pragma unroll
        for (int u = 0; u < NF; ++u) fr[u] = page_id(otab, min(u * NT + tid, nf - 1) << fsh, g.c.psh);
#pragma unroll
        for (int u = 0; u < NF; ++u) {
            fr[u] = order_row(fr[u], min(u * NT + tid, nf - 1) << fsh);
            fz[u] = order_code(plane + max(fr[u], 0));
        }
#pragma unroll
        for (int u = 0; u < NF; ++u) {
            if (fr[u] < 0) set_status(g.status, ZETA_ERR_BOUNDS);
            sm.fence[u * NT + tid] = u * NT + tid < nf && fr[u] >= 0 ? fz[u] : ~0ull;
        }
    }
    for (int w = warp; w * 32 < nn; w += NW) {
        const int u = w * 32 + lane;
        const uint32_t bits = __ballot_sync(kFull, u < nn && u > 0 && sm.parent[u] == u - 1);
        if (lane == 0) sm.run[w] = bits;
    }
    __syncthreads();
    if (tid < kTreeRows) {
        int depth = -1;
        if (tid < nq) {
            depth = climb_bits(sm.parent, sm.run, f0 + tid, sm.above[tid]);
            if (depth < 0) set_status(g.status, ZETA_ERR_BOUNDS);
            if (seq.start + depth >= cC + g.C) depth = -1;   // behind the chunk's end
        }
        sm.depth[tid] = depth;                               // -1: no result
    }
    __syncthreads();

    // ----------------------------------------------------------- windows ---
    const int CW = NW * cs, cw = cr * NW + warp;             // the cluster's warps, this one
    for (int r0 = cw; r0 < nq; r0 += 2 * CW) {
        int rr[2], st[2] = {0, 0};
        bool live[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            rr[u] = min(r0 + u * CW, kTreeRows - 1);
            live[u] = r0 + u * CW < nq && sm.depth[rr[u]] >= 0;
        }
        if (!live[0] && !live[1]) continue;
        float sw[2] = {0.f, 0.f}, mr[2] = {INFINITY, INFINITY};
        float2 o[2][NP];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < NP; ++c) o[u][c] = make_float2(0.f, 0.f);
        constexpr int LPR = PPR, RPI = 32 / LPR;             // lanes a value row, rows a load
        const int grp = lane / LPR, sub = lane % LPR;
        float q[2][DK];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int d = 0; d < DK; ++d) q[u][d] = sm.q[rr[u]][d];
        if (chunk > 0) {
            // Ranks: among the fences, then among a block's entries.
            uint64_t z[2];
            int a[2], e[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float p[kMaxDK];
#pragma unroll
                for (int d = 0; d < kMaxDK; ++d) p[d] = d < DK ? q[u][d < DK ? d : 0] : 0.f;
                z[u] = code_of(p, g.dK, g.bits);
                int le = 0;
#pragma unroll
                for (int f = 0; f < kTreeFences / 32; ++f) le += f * 32 + lane < nf && sm.fence[f * 32 + lane] <= z[u];
                const int fr = (int)__reduce_add_sync(kFull, (unsigned)le);
                a[u] = fr > 0 ? ((fr - 1) << fsh) + 1 : 0;   // entries before a are <= z
                e[u] = fr > 0 ? min(cC, fr << fsh) : 0;      // entries from e on are > z
            }
            for (int len = 1 << fsh; len > 0;) {             // most entries still open
                constexpr int PR = 2;                        // probes a lane and node
                const int step = (len + 32 * PR - 1) / (32 * PR);
                int row[2][PR];
                uint64_t zz[2][PR];
                auto at = [&](int u, int v) { return min(a[u] + (v * 32 + lane + 1) * step - 1, cC - 1); };
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int v = 0; v < PR; ++v) row[u][v] = page_id(otab, at(u, v), g.c.psh);
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int v = 0; v < PR; ++v) {
                        row[u][v] = order_row(row[u][v], at(u, v));
                        zz[u][v] = order_code(plane + max(row[u][v], 0));
                    }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    int le = 0;
#pragma unroll
                    for (int v = 0; v < PR; ++v) {
                        const bool open = a[u] + (v * 32 + lane + 1) * step - 1 < e[u];
                        if (open && row[u][v] < 0) set_status(g.status, ZETA_ERR_BOUNDS);
                        le += __popc(__ballot_sync(kFull, open && row[u][v] >= 0 && zz[u][v] <= z[u]));
                    }
                    a[u] = min(a[u] + le * step, e[u]);
                    e[u] = min(e[u], a[u] + step - 1);
                }
                len = step - 1;
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                st[u] = min(max(a[u] - (g.kw + 1) / 2, 0), cC - g.kw);
                if (lane == 0 && live[u]) sm.wst[rr[u]] = st[u];
            }
            // Up to 64 entries of both nodes at a time.
            for (int t0 = 0; t0 < g.kw; t0 += 64) {
                auto slot = [&](int v) { return t0 + (v & 1) * 32 + lane; };
                auto there = [&](int v) { return live[v >> 1] && slot(v) < g.kw; };
                int j[4], row[4];
                float x[4][DK];
#pragma unroll
                for (int v = 0; v < 4; ++v) j[v] = page_id(otab, min(st[v >> 1] + slot(v), cC - 1), g.c.psh);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int orow = order_row(j[v], st[v >> 1] + slot(v));
                    j[v] = ldi_if(g.order_idx + plane + orow, there(v) && orow >= 0);
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) row[v] = page_id(ptab, (unsigned)j[v] < (unsigned)cC ? j[v] : 0, g.c.psh);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    row[v] = (unsigned)j[v] < (unsigned)cC ? pool_row(row[v], j[v]) : -1;
                    const float *kp = g.k_pages + (int64_t)max(row[v], 0) * g.dK;
#pragma unroll
                    for (int d = 0; d < DK; ++d) x[v][d] = d < g.dK ? __ldg(kp + d) : 0.f;
                }
                float d2[4];
                bool lost = false;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    d2[v] = 0.f;
#pragma unroll
                    for (int d = 0; d < DK; ++d) {
                        const float f = q[v >> 1][d] - x[v][d];
                        d2[v] = __fmaf_rn(f, f, d2[v]);
                    }
                    if (row[v] < 0) d2[v] = INFINITY;
                    lost |= there(v) && row[v] < 0;
                    if (g.idx && there(v))
                        g.idx[(node0 + f0 + rr[v >> 1]) * g.kw + slot(v)] = (unsigned)j[v] < (unsigned)cC ? j[v] : -1;
                }
                if (lost) set_status(g.status, ZETA_ERR_BOUNDS);
                if constexpr (WK == kWSoftmax) {
                    __syncwarp();
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        float least = fminf(d2[2 * u], d2[2 * u + 1]);
#pragma unroll
                        for (int f = 16; f > 0; f >>= 1) least = fminf(least, __shfl_xor_sync(kFull, least, f));
                        if (least < mr[u]) {
                            const float f = mr[u] == INFINITY ? 0.f : __expf((least - mr[u]) * inv_g2);
#pragma unroll
                            for (int c = 0; c < NP; ++c) o[u][c] = mul2(o[u][c], dup2(f));
                            sw[u] *= f;
                            mr[u] = least;
                        }
                    }
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float w = row[v] >= 0 ? weight_fast<WK>(d2[v], mr[v >> 1], inv_g2) : 0.f;
                    sw[v >> 1] += w;
                    sm.gather.w[warp][v >> 1][(v & 1) * 32 + lane] = w;
                    sm.gather.row[warp][v >> 1][(v & 1) * 32 + lane] = row[v];
                }
                __syncwarp();
                // Value rows in batches of 4 RPI entries of both nodes, two batches in flight.
                constexpr int EB = 4 * RPI, NB = 64 / EB;
                const int last = min(64, g.kw - t0);
                uint4 bufs[2][2][4];
                auto load = [&](uint4 (&buf)[2][4], int e0) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const int pr = sm.gather.row[warp][u][e0 + grp + v * RPI];
                            buf[u][v] = ld16_if(pool + (int64_t)max(pr, 0) * g.dV + sub * (16 / (int)sizeof(V)),
                                                pr >= 0 && sub < ppr);
                        }
                };
                auto add = [&](const uint4 (&buf)[2][4], int e0) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            add_piece<V>(o[u], buf[u][v], sm.gather.w[warp][u][e0 + grp + v * RPI]);
                };
                load(bufs[0], 0);
                if (EB < last) load(bufs[1], EB);
#pragma unroll
                for (int e0 = 0; e0 < NB; ++e0) {
                    if (e0 * EB < last) add(bufs[e0 & 1], e0 * EB);
                    if (e0 + 2 < NB && (e0 + 2) * EB < last) load(bufs[e0 & 1], (e0 + 2) * EB);
                }
                __syncwarp();                                // the weights have been read
            }
        } else if (g.idx) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (live[u])
                    for (int f = lane; f < g.kw; f += 32) g.idx[(node0 + f0 + rr[u]) * g.kw + f] = -1;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            float ssum = sw[u];
#pragma unroll
            for (int f = 16; f > 0; f >>= 1) ssum += __shfl_xor_sync(kFull, ssum, f);
#pragma unroll
            for (int f = 16; f >= LPR; f >>= 1)
#pragma unroll
                for (int c = 0; c < NP; ++c) {
                    o[u][c].x += __shfl_xor_sync(kFull, o[u][c].x, f);
                    o[u][c].y += __shfl_xor_sync(kFull, o[u][c].y, f);
                }
            if (live[u]) {
                if (lane < LPR) {
#pragma unroll
                    for (int c = 0; c < NP; ++c)
                        *reinterpret_cast<float2 *>(&sm.win[rr[u]][sub * 2 * NP + 2 * c]) = o[u][c];
                }
                if (lane == 0) {
                    sm.swin[rr[u]] = ssum;
                    sm.mwin[rr[u]] = mr[u];
                }
            }
        }
    }

    // ------------------------------------------------------- shared keys ---
    // bf16: lane (g4, s4) has nodes g4 (a) and g4 + 8 (b) and the key pairs 2 s4, +1 and +8,
    // +9 of the warp's 16 keys.  float32: node lane % 16, keys 4 (lane / 16) .. + 3 of its 8.
    const int g4 = lane >> 2, s4 = lane & 3;
    const int na = Sm::MMA ? g4 : lane & 15, nb = g4 + 8;
    constexpr int ACC = Sm::MMA ? DVP / 8 * 4 : DVP / 2;
    float acc[ACC];                                          // MMA: [DVP / 8][4]; else [4 nodes][DVP / 8]
#pragma unroll
    for (int e = 0; e < ACC; ++e) acc[e] = 0.f;
    float2 sa = make_float2(0.f, 0.f), sb = sa;              // sums of weights, first and second keys
    float ma = INFINITY, mb = INFINITY;                      // softmax shifts
    float2 qa[DK], qb[DK];                                   // each coordinate twice
#pragma unroll
    for (int d = 0; d < DK; ++d) {
        qa[d] = dup2(sm.q[na][d]);
        qb[d] = dup2(sm.q[nb & 15][d]);
    }
    const float2 ig2 = dup2(inv_g2);
    const int nc = (g.dV + 15) >> 4;                         // 16-column pairs in use (bf16)
    auto dist = [&](const float (&k)[4][TK], int kl, const float2 (&q)[DK]) {
        float2 r = make_float2(0.f, 0.f);
#pragma unroll
        for (int d = 0; d < DK; ++d) {
            const float2 f = sub2(q[d], *reinterpret_cast<const float2 *>(&k[d][kl]));
            r = fma2(f, f, r);
        }
        return r;
    };
    for (int i = 0; i < mine; ++i) {
        cp_async_wait<1>();
        // Tile i is here, i - 1 used up; a key without a page up to tile i + 2 is known to all.
        const bool lost = __syncthreads_or(lost_key);
        load_tile(i + 2);
        put_row(i + 3, kid);
        kid = ask_row(i + 4);
        const int bf = i % 3, x0 = (cr + i * cs) * TK;
        const float(&ks)[4][TK] = sm.own.k[bf];
        const V *vs = sm.own.v[bf];
        const int *rows = sm.rows[i & 3];
        const bool masked = lost || x0 + TK > L;
        // Whether node r takes the tile's key kl.
        auto takes = [&](int r, int kl) {
            const int x = rows[kl];
            return x >= 0 || (x != kNoRow && (sm.above[r][~x >> 5] >> (~x & 31) & 1u));
        };
        auto mask = [&](int r, int kl, float2 x, float none) {
            return make_float2(takes(r, kl) ? x.x : none, takes(r, kl + 1) ? x.y : none);
        };
        if constexpr (Sm::MMA) {
            const int kb = warp * 16;
            if (x0 + kb >= keys) continue;
            float2 da[2], db[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int kl = kb + e * 8 + 2 * s4;
                da[e] = dist(ks, kl, qa);
                db[e] = dist(ks, kl, qb);
            }
            if constexpr (WK == kWSoftmax) {                 // move the shifts to the least d2
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int kl = kb + e * 8 + 2 * s4;
                        da[e] = mask(na, kl, da[e], INFINITY);
                        db[e] = mask(nb, kl, db[e], INFINITY);
                    }
                }
                float la = fminf(fminf(da[0].x, da[0].y), fminf(da[1].x, da[1].y));
                float lb = fminf(fminf(db[0].x, db[0].y), fminf(db[1].x, db[1].y));
#pragma unroll
                for (int f = 1; f <= 2; f <<= 1) {
                    la = fminf(la, __shfl_xor_sync(kFull, la, f));
                    lb = fminf(lb, __shfl_xor_sync(kFull, lb, f));
                }
                const float xa = fminf(ma, la), xb = fminf(mb, lb);
                const float fa = xa == ma ? 1.f : ma == INFINITY ? 0.f : __expf((xa - ma) * inv_g2);
                const float fb = xb == mb ? 1.f : mb == INFINITY ? 0.f : __expf((xb - mb) * inv_g2);
#pragma unroll
                for (int nt = 0; nt < DVP / 8; ++nt) {
                    acc[4 * nt] *= fa;
                    acc[4 * nt + 1] *= fa;
                    acc[4 * nt + 2] *= fb;
                    acc[4 * nt + 3] *= fb;
                }
                sa = mul2(sa, dup2(fa));
                sb = mul2(sb, dup2(fb));
                ma = xa;
                mb = xb;
            }
            // Finite even where no key is taken yet.
            const float xa = ma == INFINITY ? 0.f : ma, xb = mb == INFINITY ? 0.f : mb;
            uint32_t a[4], rest[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int kl = kb + e * 8 + 2 * s4;
                float2 wa = weight_pair<WK>(da[e], xa, ig2), wb = weight_pair<WK>(db[e], xb, ig2);
                if (masked) {
                    wa = mask(na, kl, wa, 0.f);
                    wb = mask(nb, kl, wb, 0.f);
                }
                sa = add2(sa, wa);
                sb = add2(sb, wb);
                a[2 * e] = pack_bf16(wa.x, wa.y);
                a[2 * e + 1] = pack_bf16(wb.x, wb.y);
                rest[2 * e] = pack_rest(wa, a[2 * e]);
                rest[2 * e + 1] = pack_rest(wb, a[2 * e + 1]);
            }
            __syncwarp();
            const uint32_t vbase = smem_u32(vs);
            const int m = lane >> 3, key = kb + (m & 1) * 8 + (lane & 7);
#pragma unroll
            for (int n2 = 0; n2 < DVP / 16; ++n2) {
                if (n2 < nc) {
                    uint32_t v[4];
                    ldsm_x4_trans(v, vbase + (uint32_t)(key * DVP + (((n2 * 2 + (m >> 1)) ^ (key & 7)) * 8)) * 2u);
                    float(&lo)[4] = *reinterpret_cast<float(*)[4]>(&acc[8 * n2]);
                    float(&hi)[4] = *reinterpret_cast<float(*)[4]>(&acc[8 * n2 + 4]);
                    mma16816(lo, a, v[0], v[1]);
                    mma16816(hi, a, v[2], v[3]);
                    mma16816(lo, rest, v[0], v[1]);
                    mma16816(hi, rest, v[2], v[3]);
                }
            }
        } else {
            const int kb = warp * 8;
            if (x0 + kb >= keys) continue;
            const int kl = kb + 4 * (lane >> 4);
            float2 d0 = dist(ks, kl, qa), d1 = dist(ks, kl + 2, qa);
            const int rg = lane >> 3, cg4 = lane & 7;        // 4 nodes, columns 4 cg4 + 32 j
            if constexpr (WK == kWSoftmax) {
                if (masked) {
                    d0 = mask(na, kl, d0, INFINITY);
                    d1 = mask(na, kl + 2, d1, INFINITY);
                }
                float la = fminf(fminf(d0.x, d0.y), fminf(d1.x, d1.y));
                la = fminf(la, __shfl_xor_sync(kFull, la, 16));
                const float xa = fminf(ma, la);
                const float fa = xa == ma ? 1.f : ma == INFINITY ? 0.f : __expf((xa - ma) * inv_g2);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float f = __shfl_sync(kFull, fa, rg * 4 + r);
#pragma unroll
                    for (int c = 0; c < DVP / 8; ++c) acc[r * (DVP / 8) + c] *= f;
                }
                sa = mul2(sa, dup2(fa));
                ma = xa;
            }
            const float xa = ma == INFINITY ? 0.f : ma;
            float2 w0 = weight_pair<WK>(d0, xa, ig2), w1 = weight_pair<WK>(d1, xa, ig2);
            if (masked) {
                w0 = mask(na, kl, w0, 0.f);
                w1 = mask(na, kl + 2, w1, 0.f);
            }
            sa = add2(sa, add2(w0, w1));
            float(&ws)[8][20] = sm.w[warp];
            ws[kl - kb][na] = w0.x;
            ws[kl - kb + 1][na] = w0.y;
            ws[kl - kb + 2][na] = w1.x;
            ws[kl - kb + 3][na] = w1.y;
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float4 w = *reinterpret_cast<const float4 *>(&ws[e][rg * 4]);
                const float wr[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int c = 0; c < DVP / 32; ++c) {
                    const float4 v = *reinterpret_cast<const float4 *>(vs + (kb + e) * DVP + cg4 * 4 + 32 * c);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        float *o = &acc[r * (DVP / 8) + 4 * c];
                        const float2 lo = fma2(dup2(wr[r]), make_float2(v.x, v.y), make_float2(o[0], o[1]));
                        const float2 hi = fma2(dup2(wr[r]), make_float2(v.z, v.w), make_float2(o[2], o[3]));
                        o[0] = lo.x;
                        o[1] = lo.y;
                        o[2] = hi.x;
                        o[3] = hi.y;
                    }
                }
            }
            __syncwarp();                                    // the weights have been read
        }
    }
    cp_async_wait<0>();
    __syncthreads();                                         // the tiles' memory is free

    // ---------------------------------------------------------- epilogue ---
    float suma = sa.x + sa.y, sumb = sb.x + sb.y;
    if constexpr (Sm::MMA) {
#pragma unroll
        for (int f = 1; f <= 2; f <<= 1) {
            suma += __shfl_xor_sync(kFull, suma, f);
            sumb += __shfl_xor_sync(kFull, sumb, f);
        }
#pragma unroll
        for (int nt = 0; nt < DVP / 8; ++nt) {
            const int col = nt * 8 + 2 * s4;
            *reinterpret_cast<float2 *>(&sm.part[warp][na][col]) = make_float2(acc[4 * nt], acc[4 * nt + 1]);
            *reinterpret_cast<float2 *>(&sm.part[warp][nb][col]) = make_float2(acc[4 * nt + 2], acc[4 * nt + 3]);
        }
        if (s4 == 0) {
            sm.psum[warp][na] = suma;
            sm.psum[warp][nb] = sumb;
            sm.pmin[warp][na] = ma;
            sm.pmin[warp][nb] = mb;
        }
    } else {
        suma += __shfl_xor_sync(kFull, suma, 16);
        const int rg = lane >> 3, cg4 = lane & 7;
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < DVP / 32; ++c) {
                const float *o = &acc[r * (DVP / 8) + 4 * c];
                *reinterpret_cast<float4 *>(&sm.part[warp][rg * 4 + r][cg4 * 4 + 32 * c]) = make_float4(o[0], o[1], o[2], o[3]);
            }
        if (lane < 16) {
            sm.psum[warp][na] = suma;
            sm.pmin[warp][na] = ma;
        }
    }
    cg::cluster_group cl = cg::this_cluster();
    if (cs > 1) cl.sync(); else __syncthreads();
    const int parts = NW * cs;
    V *out = static_cast<V *>(g.out);
    for (int r = cw; r < nq; r += CW) {                      // the nodes whose windows this warp has
        if (sm.depth[r] < 0) continue;
        float ps = 0.f, pm = INFINITY;
        if (lane < parts) {
            const Sm *o = cs > 1 ? cl.map_shared_rank(&sm, lane / NW) : &sm;
            ps = o->psum[lane % NW][r];
            pm = o->pmin[lane % NW][r];
        }
        float f = 1.f, fw = 1.f;
        if constexpr (WK == kWSoftmax) {
            float m = pm;
#pragma unroll
            for (int e = 16; e > 0; e >>= 1) m = fminf(m, __shfl_xor_sync(kFull, m, e));
            const float mw = sm.mwin[r];
            m = fminf(m, mw);
            f = pm == INFINITY ? 0.f : __expf((m - pm) * inv_g2);
            fw = mw == INFINITY ? 0.f : __expf((m - mw) * inv_g2);
        }
        float total = f * ps;
#pragma unroll
        for (int e = 16; e > 0; e >>= 1) total += __shfl_xor_sync(kFull, total, e);
        total = __fmaf_rn(fw, sm.swin[r], total);
        float o[DVP / 32];
#pragma unroll
        for (int e = 0; e < DVP / 32; ++e) o[e] = fw * sm.win[r][lane + 32 * e];
        for (int p = 0; p < parts; ++p) {
            const Sm *from = cs > 1 ? cl.map_shared_rank(&sm, p / NW) : &sm;
            const float fp = __shfl_sync(kFull, f, p);
#pragma unroll
            for (int e = 0; e < DVP / 32; ++e) o[e] = __fmaf_rn(fp, from->part[p % NW][r][lane + 32 * e], o[e]);
        }
        const int64_t rid = node0 + f0 + r;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < DVP / 32; ++e) {
            const int col = lane + 32 * e;
            if (col < g.dV) {
                const float x = __fdiv_rn(o[e], total);
                bad |= !isfinite(x);
                VT<V>::st(out + rid * g.dV + col, x);
            }
        }
        if (lane == 0) g.rowsum[rid] = total;
        if (__any_sync(kFull, bad)) {
            __syncwarp();                                    // the fast result is written first
            slow_node<V, DVP, DK, WK>(g, rid, b, h, seq.start, cC > 0 ? sm.wst[r] : 0, sm.above[r], inv_g2);
        }
    }
    if (cs > 1) cl.sync();                                   // read before any block ends
}

template <typename V, int DVP, int DK, int WK>
cudaError_t run_tree_tile(const Prob &p, const TreeArgs &g, int cs, cudaStream_t st) {
    static PerDeviceOnce once;
    constexpr size_t smem = sizeof(TreeSmem<V, DVP>);
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(tree_tile_kernel<V, DVP, DK, WK>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((g.c.n + kTreeRows - 1) / kTreeRows * cs), (unsigned)p.S);
    cfg.blockDim = dim3(kTreeThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, tree_tile_kernel<V, DVP, DK, WK>, g, cs);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename V, int DVP>
cudaError_t dispatch_tree_tile(const Prob &p, const TreeArgs &g, int cs, cudaStream_t st) {
#define ZETA_TREE(D)                                                                  \
    (p.wk == kWSoftmax     ? run_tree_tile<V, DVP, D, kWSoftmax>(p, g, cs, st)        \
     : p.wk == kWInvEuclid ? run_tree_tile<V, DVP, D, kWInvEuclid>(p, g, cs, st)      \
                           : run_tree_tile<V, DVP, D, kWCauchy>(p, g, cs, st))
    return p.dK == 3 ? ZETA_TREE(3) : ZETA_TREE(4);
#undef ZETA_TREE
}

}  // namespace
}  // namespace zeta
