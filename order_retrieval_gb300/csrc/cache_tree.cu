// cache_tree.cu -- attention of a tree of drafted tokens over the paged cache.
//
// Passages: as for the attention of new tokens over the cache (cache_attend.cu).
// A drafted token at depth d of its tree is the token at position start + d of the text
// that its branch continues: it takes the k keys around its code's rank in the prefix of
// the chunk that start lies in, the sequence's tokens of that chunk and its own line.
// Behind the chunk's end there is no result: the prefix there would hold the line's own
// keys, another one for each branch.
//
// Row kernel, for the types and sizes that the tile kernel (cache_tree_tile.cuh) does not
// take: a block of 128 threads per node and head.  The node's line is found by one thread in
// the parents in shared memory, its rank by 128 probes a step.  The keys (window, chunk,
// line) are one list, weighed a thread each 1024 at a time; then a thread per value column
// (and share of the keys) sums.  The chunk is read once per node, by which it is bound: 64 trees
// of up to 16 nodes, 8 heads, C 1024 take 1.30 ms with d_V 256 or 250 in bf16 (floor 49 us), 0.68 ms
// with d_K 8 and d_V 64, 0.66 ms with d_V 33 in float32; of d_V 64 in the tile kernel 38 us.
#include <algorithm>

#include "cache_tree_tile.cuh"

namespace zeta {
namespace {

constexpr int kNT = 128;
constexpr int kSeg = 1024;             // keys weighed at a time
constexpr int kNone = INT32_MIN;

__device__ __forceinline__ float weight_rt(int wk, float d2, float m, float inv_g2) {
    if (wk == kWSoftmax) return weight_of<kWSoftmax>(d2, m, inv_g2);
    if (wk == kWInvEuclid) return weight_of<kWInvEuclid>(d2, m, inv_g2);
    return weight_of<kWCauchy>(d2, m, inv_g2);
}

template <typename K, typename V>
__global__ void __launch_bounds__(kNT)
tree_rows_kernel(const __grid_constant__ TreeArgs g) {
    __shared__ int parent[kMaxDraft], line[kMaxDraft];
    __shared__ int from[kSeg];                       // pool row, ~node of the line, or none
    __shared__ float ws[kSeg];                       // weights (softmax: distances first)
    __shared__ float part[2][kNT];
    __shared__ float red[kNT / 32];
    __shared__ int depth_sh;
    const int tid = threadIdx.x;
    const int t = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const Seq seq = drafts_of(g.c, b, g.N, g.status);
    if (t >= seq.count) return;
    for (int u = tid; u <= t; u += kNT) parent[u] = __ldg(g.parent + (int64_t)b * g.c.n + u);
    __syncthreads();
    if (tid == 0) {
        int m = 0;
        depth_sh = climb(parent, t, [&](int u) { line[m++] = u; });
    }
    __syncthreads();
    const int depth = depth_sh, chunk = seq.start / g.C, cC = chunk * g.C;
    if (depth < 0 || seq.start + depth >= cC + g.C) {
        if (depth < 0 && tid == 0) set_status(g.status, ZETA_ERR_BOUNDS);
        return;
    }
    const int64_t slice = (int64_t)b * g.H + h, rid = slice * g.c.n + t;
    const int32_t *ptab = g.c.ptab + (int64_t)b * g.c.tlen, *otab = g.c.otab + (int64_t)b * g.c.tlen;
    const int64_t plane = ((int64_t)g.c.opages * g.H << g.c.psh) * (chunk & 1);
    const float gm = __ldg(g.gamma + h), inv_g2 = __frcp_rn(gm * gm);
    float q[kMaxDK];
    load_point(q, g.q + rid * g.dK, g.dK);

    const int nw = chunk > 0 ? g.kw : 0;             // window entries
    int first = 0;
    if (nw > 0) {
        const K *codes = static_cast<const K *>(g.order_codes) + plane;
        const K z = (K)code_of(q, g.dK, g.bits);
        int lo = 0, hi = cC;
        while (lo < hi) {                            // entries with a code <= z
            const int step = (hi - lo + kNT - 1) / kNT, at = lo + (tid + 1) * step - 1;
            bool le = false;
            if (at < hi) {
                const int row = page_row(otab, at, h, g.H, g.c.psh, g.c.pmask, g.c.opages);
                if (row < 0) set_status(g.status, ZETA_ERR_BOUNDS);
                else le = __ldg(codes + row) <= z;
            }
            lo = min(lo + __syncthreads_count(le) * step, hi);
            hi = min(hi, lo + step - 1);
        }
        first = min(max(lo - (g.kw + 1) / 2, 0), cC - g.kw);
    } else if (g.idx) {
        for (int e = tid; e < g.kw; e += kNT) g.idx[rid * g.kw + e] = -1;
    }

    const int own = seq.start - cC, total = nw + own + depth + 1;
    // Columns col and col + 128 of the share sub of the keys.
    const int lanes = g.dV <= 32 ? 32 : g.dV <= 64 ? 64 : 128;
    const int col = tid % lanes, sub = tid / lanes, subs = kNT / lanes;
    const V *pool = static_cast<const V *>(g.v_pages);
    const V *fresh = static_cast<const V *>(g.v) + slice * g.c.n * g.dV;
    float acc0 = 0.f, acc1 = 0.f, sum = 0.f, m = INFINITY;
    const bool soft = g.wk == kWSoftmax;
    for (int x0 = 0; x0 < total; x0 += kSeg) {
        const int n = min(kSeg, total - x0);
        float least = INFINITY;
        for (int e = tid; e < n; e += kNT) {
            const int x = x0 + e;
            int at = kNone;
            if (x >= nw + own) {
                at = ~line[x - nw - own];
            } else {
                int j = cC + x - nw;
                if (x < nw) {
                    const int row = page_row(otab, first + x, h, g.H, g.c.psh, g.c.pmask, g.c.opages);
                    j = row >= 0 ? __ldg(g.order_idx + plane + row) : -1;
                    if ((unsigned)j >= (unsigned)cC) j = -1;
                    if (g.idx) g.idx[rid * g.kw + x] = j;
                }
                if (j >= 0) {
                    const int row = page_row(ptab, j, h, g.H, g.c.psh, g.c.pmask, g.c.pages);
                    if (row >= 0) at = row;
                }
                if (at == kNone) set_status(g.status, ZETA_ERR_BOUNDS);
            }
            float d2 = INFINITY, w = 0.f;
            if (at != kNone) {
                const float *kp = at < 0 ? g.k + (slice * g.c.n + ~at) * g.dK
                                         : g.k_pages + (int64_t)at * g.dK;
                d2 = 0.f;
#pragma unroll
                for (int d = 0; d < kMaxDK; ++d)
                    if (d < g.dK) {
                        const float a = q[d] - __ldg(kp + d);
                        d2 = __fmaf_rn(a, a, d2);
                    }
                if (!soft) w = weight_rt(g.wk, d2, 0.f, inv_g2);
            }
            from[e] = at;
            ws[e] = soft ? d2 : w;
            sum += w;
            least = fminf(least, d2);
        }
        if (soft) {                                  // onto the least distance so far
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(kFull, least, o));
            if ((tid & 31) == 0) red[tid >> 5] = least;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kNT / 32; ++w) least = fminf(least, red[w]);
            if (least < m) {
                const float f = m == INFINITY ? 0.f : expf((least - m) * inv_g2);
                acc0 *= f;
                acc1 *= f;
                sum *= f;
                m = least;
            }
            for (int e = tid; e < n; e += kNT) {
                const float w = from[e] == kNone ? 0.f : weight_of<kWSoftmax>(ws[e], m, inv_g2);
                ws[e] = w;
                sum += w;
            }
        }
        __syncthreads();
        for (int e = sub; e < n; e += subs) {
            const int at = from[e];
            if (at == kNone) continue;
            const V *row = at < 0 ? fresh + (int64_t)~at * g.dV : pool + (int64_t)at * g.dV;
            const float w = ws[e];
            if (col < g.dV) acc0 = __fmaf_rn(w, VT<V>::ld(row + col), acc0);
            if (col + kNT < g.dV) acc1 = __fmaf_rn(w, VT<V>::ld(row + col + kNT), acc1);
        }
        __syncthreads();
    }
    part[0][tid] = acc0;
    part[1][tid] = acc1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kNT / 32; ++w) s += red[w];
    if (sub == 0) {
        for (int u = 1; u < subs; ++u) acc0 += part[0][u * lanes + col];
        V *o = static_cast<V *>(g.out) + rid * g.dV;
        if (col < g.dV) VT<V>::st(o + col, __fdiv_rn(acc0, s));
        if (col + kNT < g.dV) VT<V>::st(o + col + kNT, __fdiv_rn(acc1, s));
    }
    if (tid == 0) g.rowsum[rid] = s;
}

// How the tile kernel's blocks are laid out, measured in us with 8 heads, d_V 64, windows of
// 64, 8 K tokens a sequence (weights in two parts; with three all sides take about a twentieth more):
//  * Groups of 8 nodes to a block, and 4 warps to a group: one where a tree has no more, or
//    values are wider than 64 (whose sums fill the registers).  Trees of 4 nodes, 64 sequences:
//    one group (four blocks an SM) 25, two (two an SM) 30; of 12 nodes 41 : 39, of 32 62 : 58.  In
//    calls that do not fill the SMs two groups' warps help: 4 sequences of 8 nodes, C 256, 9.7 : 9.1.
//  * Blocks to the same nodes (a cluster), as many as run at once, where a warp has several
//    windows or many of the chunk's keys: 4 sequences of 16 nodes, 1 / 2 / 4 / 8 blocks: 16 / 12 /
//    10.5 / 9.9; C 4096 31 / 20 / 15 / 13; of 8 nodes, C 256, where neither holds, 9.0 / 9.7 / 9.8 /
//    9.9.  More than run at once: 16 sequences of 16 nodes 19 / 15 / 24 / 43.
struct Layout {
    int ng, cs;
};
Layout tile_layout(const Prob &p, int n) {
    Layout l{p.dV <= 64 && (n > 8 || p.S <= 64) ? 2 : 1, 1};
    const int rows = 8 * l.ng, warps = 4 * l.ng;
    const int64_t groups = p.S * ((n + rows - 1) / rows);
    while (l.cs < 8 && groups * l.cs * 2 <= 152 * (4 / l.ng) &&
           (std::min(n, rows) > warps * l.cs || p.C > 256 * l.cs))
        l.cs *= 2;
    return l;
}

}  // namespace

cudaError_t launch_cache_attend_tree(const Prob &p, const TreeArgs &g, cudaStream_t st) {
    const int piece = p.vdt == ZETA_BF16 ? 8 : 4;    // values of 16 bytes
    if (p.dK <= 4 && p.dV <= 128 && p.dV % piece == 0) {
        const Layout l = tile_layout(p, g.c.n);
        return p.vdt == ZETA_BF16 ? launch_tree_tile_bf16(p, g, l.ng, l.cs, st) : launch_tree_tile_f32(p, g, l.ng, l.cs, st);
    }
    const dim3 grid((unsigned)g.c.n, (unsigned)p.H, (unsigned)p.B);
    if (p.vdt == ZETA_BF16) {
        if (p.code64) tree_rows_kernel<uint64_t, __nv_bfloat16><<<grid, kNT, 0, st>>>(g);
        else tree_rows_kernel<uint32_t, __nv_bfloat16><<<grid, kNT, 0, st>>>(g);
    } else {
        if (p.code64) tree_rows_kernel<uint64_t, float><<<grid, kNT, 0, st>>>(g);
        else tree_rows_kernel<uint32_t, float><<<grid, kNT, 0, st>>>(g);
    }
    return cudaGetLastError();
}

}  // namespace zeta
