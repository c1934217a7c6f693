// cache_attend.cu -- attention of new tokens over the paged cache.
//
// Passages: as for the select and attend steps (OpenReview discussion of "ZETA:
// Leveraging Z-order Curves for Efficient Top-k Attention", reply A3 "Chunking
// ...": binary search of the insertion position and the window around it; reply
// A2 "Discussion on its robustness": the Cauchy softmax).
//
// Row kernel: one new token of one head per block, or per cluster of blocks when
// there are few tokens.  The work is a read of the token's own chunk (up to C keys
// and values, contiguous within pages) and of k scattered rows, bound by HBM when
// many tokens come at once and by the chain of dependent loads (rank search, window
// entry, page, row) when few do:
//  * Own chunk, in two phases per 1024 keys: a thread per key computes its weight into
//    shared memory; then warps stream the value rows, LPR lanes per row, two batches
//    of four 16-byte pieces in flight per lane.  A warp's rows follow one another in
//    their page, so a batch needs one address; its first batch is asked for before the
//    weights.
//  * Meanwhile one warp searches the rank (32 probes a step instead of one), looks up
//    the window's rows and weighs them; when it is done, all warps stream them.
//    In a cluster the last block takes the window and the others the own chunk.
//  * Blocks of four warps and at most 72 registers, seven to an SM, so that one
//    block's search and joins hide behind the others' loads.  Taken for the 3,784 rows
//    measured below: 69 us; six blocks to an SM 72, eight (64 registers) 73, nine 75;
//    batches of half or twice as many pieces 80 and 77; weights made 32 at a time by
//    the warp that streams those rows, without barriers, 88; eight warps a block 81; a
//    warp per row with its rows through shared memory onto the tensor cores 100.
//  * Sums of weights and of weighted values are held in float32 per thread and
//    joined in a fixed order, in shared memory and across the cluster through
//    distributed shared memory: no workspace, one launch, the same bits each run.
//
// 473 sequences with one new token, 8 heads, 9 K tokens before each and 522 in its
// chunk of 1024 on average, windows of 48, 128-byte value rows: 69 us for 300 MB, 4.4
// TB/s (64 % of the measured HBM rate; DRAM reads 343 MB, the rank probes and table
// sectors among them).  Half of the issue slots are used; the warps wait for loads and
// at the block's barriers.  59 sequences with 37 K tokens before each: 16 us, one row's
// chain (rank search, window lookups, join) beside the longest own chunk, all blocks at
// once.  One sequence, one head, a chunk of 128: 4.3 us.
#include <cmath>

#include <cooperative_groups.h>

#include "cache_tile.cuh"

namespace zeta {
namespace {

namespace cg = cooperative_groups;

constexpr int kPerSM = 7;              // blocks of four warps to an SM
constexpr int kSeg = 1024;             // keys weighed at a time
constexpr int kWin = 64;               // window entries that the searching warp prepares

struct Args {
    Cache c;
    const float *q, *gamma, *k_pages;
    const int32_t *order_idx;
    float *rowsum;
    int32_t *idx, *status;
    int N, H, dK, dV, k, C, bits, wk;
};

// A piece of a value row: 16 bytes (WIDE) or one value.
template <typename V, bool WIDE>
struct Piece {
    static constexpr int N = WIDE ? 16 / (int)sizeof(V) : 1;       // values
    uint32_t w[WIDE ? 4 : 1];
    __device__ __forceinline__ void load(const V *row, int piece, bool ok) {
        if constexpr (WIDE) {
            const uint4 x = ld16_if(reinterpret_cast<const uint4 *>(row) + piece, ok);
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
        } else if constexpr (sizeof(V) == 2) {
            w[0] = ld2_if(row + piece, ok);
        } else {
            w[0] = ld4_if(row + piece, ok);
        }
    }
    // acc += f * values
    __device__ __forceinline__ void add(float2 (&acc)[(N + 1) / 2], float f) const {
        const float2 ff = dup2(f);
        if constexpr (!WIDE) {
            const float x = sizeof(V) == 2 ? __uint_as_float(w[0] << 16) : __uint_as_float(w[0]);
            acc[0].x = __fmaf_rn(f, x, acc[0].x);
        } else if constexpr (sizeof(V) == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                acc[e] = fma2(ff, make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u)), acc[e]);
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
                acc[e] = fma2(ff, make_float2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1])), acc[e]);
        }
    }
};

__device__ __forceinline__ float weight_rt(int wk, float d2, float m, float inv_g2) {
    if (wk == kWSoftmax) return weight_of<kWSoftmax>(d2, m, inv_g2);
    if (wk == kWInvEuclid) return weight_of<kWInvEuclid>(d2, m, inv_g2);
    return weight_of<kWCauchy>(d2, m, inv_g2);
}

__device__ __forceinline__ float warp_min(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fminf(x, __shfl_xor_sync(kFull, x, o));
    return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

// Barrier of the first `n` threads, the warps that take the own chunk.  It is one for
// whole warps: lanes that recorded a missing page meet the others first.
__device__ __forceinline__ void bar_own(int n) {
    __syncwarp();
    asm volatile("bar.sync 1, %0;\n" ::"r"(n) : "memory");
}

// Entries of the prefix with a code <= z: a warp probes 32 per step.  (64, 128 or 256
// probes take a step less and no less time, and their sectors come out of the other
// blocks' HBM time: 64 tokens under 64 K entries 18.1 us with 32, then 18.4, 19.2, 20.7.)
template <typename K, typename Page>
__device__ __forceinline__ int rank_of(const Args &g, Page page, int h, const K *codes, K z, int M,
                                       int lane) {
    int lo = 0, hi = M;
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step - 1;
        const int row = row_in(page(min(at, M - 1)), at, h, g.H, g.c.psh, g.c.pmask, g.c.opages);
        const K c = __ldg(codes + max(row, 0));
        const bool open = at < hi;
        if (open && row < 0) set_status(g.status, ZETA_ERR_BOUNDS);
        const int le = __popc(__ballot_sync(kFull, open && row >= 0 && c <= z));
        lo = min(lo + le * step, hi);
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

struct Total {
    float acc[kMaxDV];
    float s, m;
};

// V: value type; LPR lanes per value row, NP pieces per lane; LOW: d_K <= 4.
template <typename K, typename V, bool WIDE, int LPR, int NP, bool LOW>
__global__ void __launch_bounds__(128, kPerSM)
cache_rows_kernel(const __grid_constant__ Args g, const K *__restrict__ order_codes,
                  const V *__restrict__ v_pages, V *__restrict__ out, int cs, int ppr) {
    using P = Piece<V, WIDE>;
    constexpr int NT = 128, NW = NT / 32, NA = (P::N + 1) / 2, DM = LOW ? 4 : kMaxDK;
    constexpr int RPI = 32 / LPR, U = NP >= 4 ? 1 : 4 / NP, BR = RPI * U;   // rows per load, batch
    constexpr int UK = 2;                                        // keys a thread weighs at a time
    __shared__ float w_sh[kSeg];                                 // weights (softmax: distances) of a segment
    __shared__ int row_sh[kSeg];                                 // rows of long windows
    __shared__ float ww_sh[kWin];                                // the window's, prepared by the searching warp
    __shared__ int wr_sh[kWin];
    __shared__ float part[NW][LPR * NP * P::N];
    __shared__ float red_s[NW], red_m[NW];
    __shared__ int st_sh;
    __shared__ Total tot;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cr = cs == 1 ? 0 : (int)(blockIdx.x % (unsigned)cs);   // block in the cluster
    const int t = cs == 1 ? (int)blockIdx.x : (int)(blockIdx.x / (unsigned)cs);
    const int h = blockIdx.y, b = blockIdx.z;
    const int64_t rid = ((int64_t)b * g.H + h) * g.c.n + t;
    const int32_t *ptab = g.c.ptab + (int64_t)b * g.c.tlen, *otab = g.c.otab + (int64_t)b * g.c.tlen;
    auto ppage = [&](int j) { return page_id(ptab, j, g.c.psh); };
    auto opage = [&](int e) { return page_id(otab, e, g.c.psh); };
    const Seq seq = seq_of(g.c, b, g.N, g.status);
    float q[DM];
#pragma unroll
    for (int d = 0; d < DM; ++d) q[d] = d < g.dK ? __ldg(g.q + rid * g.dK + d) : 0.f;
    const float gm = __ldg(g.gamma + h);
    if (t >= seq.count) return;                                  // the whole cluster returns
    const int i = seq.start + t, chunk = i / g.C, cC = chunk * g.C;
    const float inv_g2 = __frcp_rn(gm * gm);
    const int64_t plane = ((int64_t)g.c.opages * g.H << g.c.psh) * (chunk & 1);
    const bool window = chunk > 0, soft = g.wk == kWSoftmax;
    const bool win_here = window && cr == cs - 1;                // this block takes the window
    const bool searcher = win_here && warp == NW - 1;
    // Own-chunk keys of this block: an equal share for each of the row's warps but the
    // one that searches.
    const int own = win_here ? NT - 32 : NT;                     // threads on the own chunk
    const int takers = cs * NW - (window ? 1 : 0);
    const int per = cs == 1 ? i - cC + 1 : ((i - cC + takers) / takers * NW + 31) & ~31;
    const int k0 = min(cC + cr * per, i + 1), k1 = cr == cs - 1 ? i + 1 : min(k0 + per, i + 1);

    float2 acc[NP][NA];
#pragma unroll
    for (int p = 0; p < NP; ++p)
#pragma unroll
        for (int e = 0; e < NA; ++e) acc[p][e] = make_float2(0.f, 0.f);
    float sum = 0.f, m_own = INFINITY;
    auto rescale = [&](float f) {
        sum *= f;
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int e = 0; e < NA; ++e) acc[p][e] = mul2(acc[p][e], dup2(f));
    };
    const int sub = lane % LPR, grp = lane / LPR;
    auto row_of = [&](int id, int j) { return row_in(id, j, h, g.H, g.c.psh, g.c.pmask, g.c.pages); };
    // Squared distances of UK rows (row 0 in the place of none), all asked for together.
    auto dists = [&](const int (&row)[UK], float (&d2)[UK]) {
        float x[UK][DM];
#pragma unroll
        for (int u = 0; u < UK; ++u) {
            const float *kp = g.k_pages + (int64_t)max(row[u], 0) * g.dK;
#pragma unroll
            for (int d = 0; d < DM; ++d) x[u][d] = d < g.dK ? __ldg(kp + d) : 0.f;
        }
#pragma unroll
        for (int u = 0; u < UK; ++u) {
            d2[u] = 0.f;
#pragma unroll
            for (int d = 0; d < DM; ++d) {
                const float e = q[d] - x[u][d];                  // both 0 beyond d_K
                d2[u] = __fmaf_rn(e, e, d2[u]);
            }
        }
    };
    // Pool rows of UK window entries (looked up through the order's and the keys' pages).
    auto window_rows = [&](int st, const int (&slot)[UK], int (&row)[UK]) {
        int j[UK];
#pragma unroll
        for (int u = 0; u < UK; ++u) j[u] = opage(min(st + slot[u], cC - 1));
#pragma unroll
        for (int u = 0; u < UK; ++u) {
            const int r = row_in(j[u], st + slot[u], h, g.H, g.c.psh, g.c.pmask, g.c.opages);
            j[u] = ldi_if(g.order_idx + plane + r, slot[u] < g.k && r >= 0);
        }
#pragma unroll
        for (int u = 0; u < UK; ++u) row[u] = ppage((unsigned)j[u] < (unsigned)cC ? j[u] : 0);
#pragma unroll
        for (int u = 0; u < UK; ++u) {
            const bool in = (unsigned)j[u] < (unsigned)cC;
            row[u] = in ? row_of(row[u], j[u]) : -1;
            if (slot[u] < g.k) {
                if (row[u] < 0) set_status(g.status, ZETA_ERR_BOUNDS);
                if (g.idx) g.idx[rid * g.k + slot[u]] = in ? j[u] : -1;
            }
        }
    };
    P buf[U][NP], buf2[U][NP];
    // Ask for the value rows of own keys j0 .. j0 + BR - 1 (below k1).
    auto ask = [&](P (&buf)[U][NP], int j0) {
        if (j0 + BR <= k1 && (j0 & g.c.pmask) + BR - 1 <= g.c.pmask) {   // one run in one page
            const int row = row_of(ppage(j0), j0);
            const V *src = v_pages + ((int64_t)max(row, 0) + grp) * g.dV;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    buf[u][p].load(src + u * RPI * g.dV, sub + p * LPR, row >= 0 && sub + p * LPR < ppr);
        } else {
            int row[U];
#pragma unroll
            for (int u = 0; u < U; ++u) row[u] = ppage(min(j0 + u * RPI + grp, i));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int j = j0 + u * RPI + grp;
                row[u] = j < k1 ? row_of(row[u], j) : -1;
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    buf[u][p].load(v_pages + (int64_t)max(row[u], 0) * g.dV, sub + p * LPR,
                                   row[u] >= 0 && sub + p * LPR < ppr);
            }
        }
    };
    // Value rows rows[0 .. n) (weights ws) by every warp of the block, the rows spread
    // over the warps.
    auto stream = [&](const int *rows, const float *ws, int n) {
        for (int r0 = warp * RPI + grp; r0 < n; r0 += NW * BR) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * NW * RPI, row = r < n ? rows[r] : -1;
#pragma unroll
                for (int p = 0; p < NP; ++p)
                    buf[u][p].load(v_pages + (int64_t)max(row, 0) * g.dV, sub + p * LPR,
                                   row >= 0 && sub + p * LPR < ppr);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * NW * RPI;
                const float w = r < n ? ws[r] : 0.f;
#pragma unroll
                for (int p = 0; p < NP; ++p) buf[u][p].add(acc[p], w);
            }
        }
    };
    // Weigh rows into ws (softmax: distances) and this thread's sum; the least distance.
    auto weigh = [&](const int (&row)[UK], const float (&d2)[UK], int r0, int stride, int n, float *ws) {
        float least = INFINITY;
#pragma unroll
        for (int u = 0; u < UK; ++u) {
            const int r = r0 + u * stride;
            if (r < n) {
                const float x2 = row[u] >= 0 ? d2[u] : INFINITY;
                const float w = row[u] >= 0 && !soft ? weight_rt(g.wk, x2, 0.f, inv_g2) : 0.f;
                ws[r] = soft ? x2 : w;
                sum += w;
                least = fminf(least, x2);
            }
        }
        return least;
    };
    // Softmax: distances ws[0 .. n) become weights on the shift m_own.
    auto soften = [&](float *ws, int n, int threads) {
        for (int r = tid; r < n; r += threads) {
            const float w = ws[r] == INFINITY ? 0.f : weight_of<kWSoftmax>(ws[r], m_own, inv_g2);
            ws[r] = w;
            sum += w;
        }
    };
    auto shift_down = [&](float least) {                         // the same value in all threads
        if (least < m_own) {
            rescale(m_own == INFINITY ? 0.f : expf((least - m_own) * inv_g2));
            m_own = least;
        }
    };

    if (searcher) {
        float x[kMaxDK];
#pragma unroll
        for (int d = 0; d < kMaxDK; ++d) x[d] = d < DM ? q[d < DM ? d : 0] : 0.f;
        const K z = (K)code_of(x, g.dK, g.bits);
        const int rk = rank_of<K>(g, opage, h, order_codes + plane, z, cC, lane);
        const int st = min(max(rk - (g.k + 1) / 2, 0), cC - g.k);
        int slot[UK];                                            // two a lane
#pragma unroll
        for (int u = 0; u < UK; ++u) slot[u] = u < 2 ? u * 32 + lane : g.k;
        int row[UK];
        float d2[UK];
        window_rows(st, slot, row);
        dists(row, d2);
        wr_sh[lane] = row[0];
        wr_sh[32 + lane] = row[1];
        const float least = warp_min(weigh(row, d2, lane, 32, kWin, ww_sh));
        if (lane == 0) {
            st_sh = st;
            red_m[NW - 1] = least;
        }
    } else {
        for (int j0 = k0; j0 < k1; j0 += kSeg) {
            const int n = min(kSeg, k1 - j0);
            const int step = own / 32 * BR, r1 = warp * BR;      // the warp's batches: r1, r1 + step, ...
            if (r1 < n) ask(buf, j0 + r1);
            if (r1 + step < n) ask(buf2, j0 + r1 + step);
            float least = INFINITY;
            for (int r0 = tid; r0 < n; r0 += UK * own) {
                int row[UK];
                float d2[UK];
#pragma unroll
                for (int u = 0; u < UK; ++u) row[u] = ppage(min(j0 + r0 + u * own, i));
#pragma unroll
                for (int u = 0; u < UK; ++u) row[u] = row_of(row[u], j0 + r0 + u * own);
                dists(row, d2);
#pragma unroll
                for (int u = 0; u < UK; ++u)
                    if (r0 + u * own < n && row[u] < 0) set_status(g.status, ZETA_ERR_BOUNDS);
                least = fminf(least, weigh(row, d2, r0, own, n, w_sh));
            }
            if (soft) {                                          // onto the least distance so far
                least = warp_min(least);
                if (lane == 0) red_s[warp] = least;
                bar_own(own);
                for (int w = 0; w < own / 32; ++w) least = fminf(least, red_s[w]);
                shift_down(least);
                soften(w_sh, n, own);
            }
            bar_own(own);
            auto use = [&](P (&buf)[U][NP], int r0) {            // add a batch, ask for the one after the next
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + u * RPI + grp;
                    const float w = r < n ? w_sh[r] : 0.f;
#pragma unroll
                    for (int p = 0; p < NP; ++p) buf[u][p].add(acc[p], w);
                }
                if (r0 + 2 * step < n) ask(buf, j0 + r0 + 2 * step);
            };
            for (int r0 = r1; r0 < n; r0 += 2 * step) {
                use(buf, r0);
                if (r0 + step < n) use(buf2, r0 + step);
            }
            if (j0 + kSeg < k1) bar_own(own);                    // the array is free again
        }
    }
    if (!window && g.idx && cr == 0)
        for (int slot = tid; slot < g.k; slot += NT) g.idx[rid * g.k + slot] = -1;

    // The window, by all warps; for the softmax everything onto one shift.
    if (win_here) {
        if (soft && lane == 0 && !searcher) red_m[warp] = m_own;
        __syncthreads();
        const int st = st_sh;
        if (soft) {
            float least = INFINITY;
            for (int w = 0; w < NW; ++w) least = fminf(least, red_m[w]);
            shift_down(least);
            soften(ww_sh, min(kWin, g.k), NT);
            __syncthreads();
        }
        stream(wr_sh, ww_sh, min(kWin, g.k));
        for (int t0 = kWin; t0 < g.k; t0 += kSeg) {              // windows of more entries
            const int n = min(kSeg, g.k - t0);
            float least = INFINITY;
            __syncthreads();
            for (int r0 = tid; r0 < n; r0 += UK * NT) {
                int slot[UK], row[UK];
                float d2[UK];
#pragma unroll
                for (int u = 0; u < UK; ++u) slot[u] = r0 + u * NT < n ? t0 + r0 + u * NT : g.k;
                window_rows(st, slot, row);
                dists(row, d2);
#pragma unroll
                for (int u = 0; u < UK; ++u)
                    if (r0 + u * NT < n) row_sh[r0 + u * NT] = row[u];
                least = fminf(least, weigh(row, d2, r0, NT, n, w_sh));
            }
            if (soft) {
                least = warp_min(least);
                if (lane == 0) red_m[warp] = least;
                __syncthreads();
                for (int w = 0; w < NW; ++w) least = fminf(least, red_m[w]);
                shift_down(least);
                soften(w_sh, n, NT);
            }
            __syncthreads();
            stream(row_sh, w_sh, n);
        }
    }

    // Join the lanes of a column, the warps, the blocks.
    sum = warp_sum(sum);
#pragma unroll
    for (int o = 16; o >= LPR; o >>= 1)
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int e = 0; e < NA; ++e) {
                acc[p][e].x += __shfl_xor_sync(kFull, acc[p][e].x, o);
                if (P::N > 1) acc[p][e].y += __shfl_xor_sync(kFull, acc[p][e].y, o);
            }
    if (lane < LPR) {
#pragma unroll
        for (int p = 0; p < NP; ++p)
#pragma unroll
            for (int e = 0; e < P::N; ++e)
                part[warp][(lane + p * LPR) * P::N + e] = e & 1 ? acc[p][e / 2].y : acc[p][e / 2].x;
    }
    __syncthreads();                                             // red_s may still be read above
    if (lane == 0) red_s[warp] = sum;
    __syncthreads();
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) total += red_s[w];
    auto column = [&](int d) {
        float o = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) o += part[w][d];
        return o;
    };
    if (cs == 1) {
        for (int d = tid; d < g.dV; d += NT) VT<V>::st(out + rid * g.dV + d, __fdiv_rn(column(d), total));
        if (tid == 0) g.rowsum[rid] = total;
        return;
    }
    for (int d = tid; d < g.dV; d += NT) tot.acc[d] = column(d);
    if (tid == 0) {
        tot.s = total;
        tot.m = m_own;
    }
    cg::cluster_group cl = cg::this_cluster();
    cl.sync();
    if (cr == 0) {
        float m = INFINITY, f[8], ssum = 0.f;
#pragma unroll
        for (int p = 0; p < 8; ++p)
            if (p < cs && soft) m = fminf(m, cl.map_shared_rank(&tot, p)->m);
#pragma unroll
        for (int p = 0; p < 8; ++p) {
            f[p] = 0.f;
            if (p < cs) {
                const Total *o = cl.map_shared_rank(&tot, p);
                f[p] = !soft ? 1.f : o->m == INFINITY ? 0.f : expf((m - o->m) * inv_g2);
                ssum = __fmaf_rn(f[p], o->s, ssum);
            }
        }
        for (int d = tid; d < g.dV; d += NT) {
            float o = 0.f;
#pragma unroll
            for (int p = 0; p < 8; ++p)
                if (p < cs) o = __fmaf_rn(f[p], cl.map_shared_rank(&tot, p)->acc[d], o);
            VT<V>::st(out + rid * g.dV + d, __fdiv_rn(o, ssum));
        }
        if (tid == 0) g.rowsum[rid] = ssum;
    }
    cl.sync();                                                   // read before any block ends
}

template <typename K, typename V, bool WIDE, int LPR, int NP>
cudaError_t run_rows(const Args &g, const Prob &p, const void *order_codes, const void *v_pages,
                     void *out, int ppr, cudaStream_t st) {
    const int64_t rows = p.S * g.c.n;
    // Blocks per token: split as far as all blocks run at once and the own chunk has
    // work for more than four warps (a cluster's joins cost 1.3 us).  64 tokens of 8
    // heads, C 1024: one block each 21 us, two 16, four 26.
    const int most = p.C <= 256 ? 1 : p.C <= 512 ? 2 : p.C <= 1024 ? 4 : 8;
    int cs = 1;
    while (cs < most && rows * cs * 2 <= 152 * kPerSM) cs *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(g.c.n * cs), (unsigned)p.H, (unsigned)p.B);
    cfg.blockDim = dim3(128);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    const K *oc = static_cast<const K *>(order_codes);
    const V *vp = static_cast<const V *>(v_pages);
    V *o = static_cast<V *>(out);
    const cudaError_t e =
        p.dK <= 4 ? cudaLaunchKernelEx(&cfg, cache_rows_kernel<K, V, WIDE, LPR, NP, true>, g, oc, vp, o, cs, ppr)
                  : cudaLaunchKernelEx(&cfg, cache_rows_kernel<K, V, WIDE, LPR, NP, false>, g, oc, vp, o, cs, ppr);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename K, typename V>
cudaError_t dispatch_rows(const Args &g, const Prob &p, const void *order_codes,
                          const void *v_pages, void *out, cudaStream_t st) {
    const int bytes = p.dV * (int)sizeof(V);
    const bool wide = bytes % 16 == 0;
    const int ppr = wide ? bytes / 16 : p.dV;
#define ZETA_ROWS(WIDE, LPR, NP) run_rows<K, V, WIDE, LPR, NP>(g, p, order_codes, v_pages, out, ppr, st)
    if (!wide) return ppr <= 64 ? ZETA_ROWS(false, 32, 2) : ZETA_ROWS(false, 32, 8);
    if (ppr <= 4) return ZETA_ROWS(true, 4, 1);
    if (ppr <= 8) return ZETA_ROWS(true, 8, 1);
    if (ppr <= 16) return ZETA_ROWS(true, 16, 1);
    if (ppr <= 32) return ZETA_ROWS(true, 32, 1);
    if constexpr (sizeof(V) == 4) return ZETA_ROWS(true, 32, 2);
    return cudaErrorInvalidValue;      // bf16 rows have at most 32 pieces
#undef ZETA_ROWS
}

// How many groups of 16 rows a block of the tile kernel takes for up to n rows of each
// of the S slices (0: the row kernel).  The row kernel reads the own chunk once per row;
// the tile kernel reads it once per block, but a block takes long and there are fewer.
// Measured, row kernel : blocks of 16 rows in us, with 8 heads, d_V 64 and windows of 64:
//  * The tile kernel takes rows enough to share (n sqrt(C) >= 220): 256 sequences of 8
//    rows 85 : 106 for C 256, of 4 rows 87 : 126 for C 1024, of 2 rows 185 : 241 for
//    C 4096; but of 16 rows 156 : 119, of 8 rows 151 : 130, of 4 rows 293 : 243.
//  * And enough in all to fill the SMs (S n sqrt(C) >= 55000): 4 sequences of 64 rows
//    14.5 : 15.9 for C 256, of 32 rows 14.2 : 17.0 for C 1024, of 16 rows 33 : 39 for
//    C 4096; of twice as many 27 : 17, 23.7 : 19.0, 60 : 40.
//  * Values wider than 64, whose tiles are half as long, want more of both: 16 sequences
//    of 16 rows 38 : 48 for C 1024, of 32 rows 30 : 51 for C 256; 64 of 16 104 : 81 for
//    C 1024, 64 of 4 166 : 129 for C 4096.
// Larger blocks share tiles and set-up among more rows.  They are taken where the smaller
// ones would not all run at once (two blocks an SM, three for values wider than 64; half
// as many again before 64 rows, more under long chunks, which are most of a block): C
// 1024, 4 sequences of 128 rows 20 us in blocks of 16, 27 in blocks of 32, of 256 rows 43
// and 33; 64 sequences of 128 rows 160 in blocks of 32, 146 of 64; C 4096, 16 of 128 rows
// 81 and 108.  For wider values blocks of 32 gain up to 1.1 in large calls, 64 never did.
// Over 552 cases (half of them drawn: C 128 to 8192, 1 to 256 sequences of 1 to 32 heads,
// 2 to 1024 rows, d_V 32 to 128, d_K 1 to 4, all weights) this takes the fastest form or
// one within 10 % in 523, and 1.3 times its time at worst.
int tile_groups(const Prob &p, int n) {
    const double root = std::sqrt((double)p.C), rows = (double)p.S * n;
    const bool wide = p.dV > 64;
    if (n * root < 220 || rows * root < 55000) return 0;
    if (wide && n * rows * p.C * root < 1.5e9) return 0;
    auto blocks = [&](int r) { return p.S * ((n + r - 1) / r); };
    if (wide) return n >= 48 && blocks(16) > 152 * 3 ? 2 : 1;
    if (n >= 48 && (double)blocks(32) > 152 * 3 * (p.C > 1024 ? p.C / 1024. : 1.)) return 4;
    return n > 16 && blocks(16) > 152 * 2 ? 2 : 1;
}

}  // namespace

cudaError_t launch_cache_attend(const Prob &p, const Cache &c, const float *q, const float *gamma,
                                const float *k_pages, const void *v_pages,
                                const void *order_codes, const int32_t *order_idx, void *out,
                                float *rowsum, int32_t *idx, int32_t *status, cudaStream_t st) {
    const Args g{c, q, gamma, k_pages, order_idx, rowsum, idx, status,
                 p.N, p.H, p.dK, p.dV, p.k, p.C, p.bits, p.wk};
    const int wm = p.vdt == ZETA_BF16 && p.dV % 8 == 0 && p.dV <= 128 && p.dK <= 4
                       ? tile_groups(p, c.n) : 0;
    if (wm > 0) {
        const TileArgs t{c, q, gamma, k_pages, static_cast<const __nv_bfloat16 *>(v_pages),
                         order_codes, order_idx, static_cast<__nv_bfloat16 *>(out), rowsum, idx,
                         status, p.N, p.H, p.dK, p.dV, p.k, p.C, p.bits, p.wk, p.code64};
        return p.dV <= 64 ? launch_cache_tile64(p, t, wm, st) : launch_cache_tile128(p, t, wm, st);
    }
    if (p.vdt == ZETA_BF16) {
        if (p.code64)
            return dispatch_rows<uint64_t, __nv_bfloat16>(g, p, order_codes, v_pages, out, st);
        return dispatch_rows<uint32_t, __nv_bfloat16>(g, p, order_codes, v_pages, out, st);
    }
    if (p.code64) return dispatch_rows<uint64_t, float>(g, p, order_codes, v_pages, out, st);
    return dispatch_rows<uint32_t, float>(g, p, order_codes, v_pages, out, st);
}

}  // namespace zeta
