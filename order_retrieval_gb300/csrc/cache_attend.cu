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
//  * Own chunk, in two phases per 1024 keys: a thread per key looks up its row and
//    computes its weight into shared memory; then LPR threads per value row stream
//    the rows, a 16-byte piece each, four pieces in flight per thread.  The first
//    pieces are asked for before the weights are computed.
//  * Meanwhile one warp searches the rank (32 P probes a step instead of one), looks
//    up the window's rows and weighs them; when it is done, all threads stream them.
//    In a cluster the last block takes the window and the others the own chunk.
//  * About 50 registers a thread leave five blocks on an SM, so that one block's
//    search and joins hide behind the others' loads.  (A warp per row with its rows
//    in flight through shared memory, summed on the tensor cores, needs a third of
//    the instructions but waits for each of its steps alone: 90 to 100 us where this
//    takes see below.)
//  * Sums of weights and of weighted values are held in float32 per thread and
//    joined in a fixed order, in shared memory and across the cluster through
//    distributed shared memory: no workspace, one launch, the same bits each run.
#include <cooperative_groups.h>

#include "cache_tile.cuh"

namespace zeta {
namespace {

namespace cg = cooperative_groups;

constexpr int kTileRows = 4;           // rows of a call from which the tile kernel runs
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

// Barrier of the first `n` threads' warps of the group that takes the own chunk.
__device__ __forceinline__ void bar_own(int n) { asm volatile("bar.sync 1, %0;\n" ::"r"(n) : "memory"); }

// Entries of the prefix with a code <= z: a warp probes 32 P of them per step.
template <typename K, int P>
__device__ __forceinline__ int rank_of(const Args &g, const int32_t *otab, int h, const K *codes, K z,
                                       int M, int lane) {
    int lo = 0, hi = M;
    while (lo < hi) {
        const int step = (hi - lo + 32 * P - 1) / (32 * P);
        auto at = [&](int p) { return lo + (p * 32 + lane + 1) * step - 1; };
        int row[P];
        K c[P];
#pragma unroll
        for (int p = 0; p < P; ++p) row[p] = page_id(otab, min(at(p), M - 1), g.c.psh);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            row[p] = row_in(row[p], at(p), h, g.H, g.c.psh, g.c.pmask, g.c.opages);
            c[p] = __ldg(codes + max(row[p], 0));
        }
        int le = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const bool open = at(p) < hi;
            if (open && row[p] < 0) set_status(g.status, ZETA_ERR_BOUNDS);
            le += __popc(__ballot_sync(kFull, open && row[p] >= 0 && c[p] <= z));
        }
        lo = min(lo + le * step, hi);
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

struct Total {
    float acc[kMaxDV];
    float s, m;
};

// V: value type; LPR: threads per value row; NT: threads.
template <typename K, typename V, bool WIDE, int LPR, int NT>
__global__ void __launch_bounds__(NT, LPR <= 32 ? 1280 / NT : 1024 / NT)
cache_rows_kernel(const __grid_constant__ Args g, const K *__restrict__ order_codes,
                  const V *__restrict__ v_pages, V *__restrict__ out, int cs, int ppr) {
    using P = Piece<V, WIDE>;
    constexpr int U = 4, NA = (P::N + 1) / 2, NW = NT / 32;
    __shared__ float w_sh[kSeg];                                 // weights (softmax: distances) of a segment
    __shared__ int row_sh[kSeg];
    __shared__ float ww_sh[kWin];                                // the window's, prepared by the searching warp
    __shared__ int wr_sh[kWin];
    __shared__ float part[NW][(LPR < 32 ? LPR : 32) * P::N];
    __shared__ float red_s[NW], red_m[NW];
    __shared__ int st_sh;
    __shared__ Total tot;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned rid = blockIdx.x / (unsigned)cs;
    const int cr = (int)(blockIdx.x - rid * (unsigned)cs);       // block in the cluster
    const unsigned s = rid / (unsigned)g.c.n;
    const int t = (int)(rid - s * (unsigned)g.c.n);
    const int b = (int)(s / (unsigned)g.H), h = (int)(s - (unsigned)b * (unsigned)g.H);
    float q[kMaxDK];
    load_point(q, g.q + (int64_t)rid * g.dK, g.dK);
    const float gm = g.gamma[h];
    const Seq seq = seq_of(g.c, b, g.N, g.status);
    if (t >= seq.count) return;                                  // the whole cluster returns
    const int32_t *ptab = g.c.ptab + (int64_t)b * g.c.tlen, *otab = g.c.otab + (int64_t)b * g.c.tlen;
    const int i = seq.start + t, chunk = i / g.C, cC = chunk * g.C;
    const float inv_g2 = __frcp_rn(gm * gm);
    const int64_t plane = ((int64_t)g.c.opages * g.H << g.c.psh) * (chunk & 1);
    const bool window = chunk > 0, soft = g.wk == kWSoftmax;
    const bool win_here = window && cr == cs - 1;                // this block takes the window
    const bool searcher = win_here && warp == NW - 1;
    // Own-chunk keys of this block: all of them, or an equal share of the cluster's
    // blocks but the one with the window.
    const int sharers = cs == 1 ? 1 : window ? cs - 1 : cs;
    const int per = ((i - cC + sharers) / sharers + 31) & ~31;
    const int k0 = cC + cr * per, k1 = cr < sharers ? min(k0 + per, i + 1) : k0;
    const int own = win_here ? NT - 32 : NT;                     // threads on the own chunk

    float2 acc[NA];
#pragma unroll
    for (int e = 0; e < NA; ++e) acc[e] = make_float2(0.f, 0.f);
    float sum = 0.f, m_own = INFINITY;
    const int sub = tid % LPR, grp = tid / LPR;
    auto row_of = [&](int id, int j) { return row_in(id, j, h, g.H, g.c.psh, g.c.pmask, g.c.pages); };
    auto dist = [&](int row) {
        float x[kMaxDK], d2 = 0.f;
        load_point(x, g.k_pages + (int64_t)row * g.dK, g.dK);
#pragma unroll
        for (int d = 0; d < kMaxDK; ++d) {
            if (d < g.dK) {
                const float e = q[d] - x[d];
                d2 = __fmaf_rn(e, e, d2);
            }
        }
        return d2;
    };
    // Pool row of window entry `slot` (looked up through the order's and the keys' pages).
    auto window_row = [&](int st, int slot, bool there) {
        const int e = st + slot;
        const int orow = row_in(page_id(otab, min(e, cC - 1), g.c.psh), e, h, g.H, g.c.psh, g.c.pmask, g.c.opages);
        const int j = ldi_if(g.order_idx + plane + orow, there && orow >= 0);
        const bool in = (unsigned)j < (unsigned)cC;
        const int row = in ? row_of(page_id(ptab, j, g.c.psh), j) : -1;
        if (there) {
            if (row < 0) set_status(g.status, ZETA_ERR_BOUNDS);
            if (g.idx) g.idx[(int64_t)rid * g.k + slot] = in ? j : -1;
        }
        return row;
    };
    // Stream n value rows (rows, weights in shared memory) with `groups` row groups; the
    // first U of the thread's rows may already be on their way in buf.
    auto stream = [&](const int *rows, const float *ws, int n, int groups, P (&buf)[U], bool have) {
        if (grp >= groups) return;
        for (int r0 = grp; r0 < n; r0 += U * groups) {
            if (!have || r0 != grp) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = r0 + u * groups, row = r < n ? rows[r] : -1;
                    buf[u].load(v_pages + (int64_t)max(row, 0) * g.dV, sub, row >= 0 && sub < ppr);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = r0 + u * groups;
                if (r < n) buf[u].add(acc, ws[r]);
            }
        }
    };
    P buf[U];

    if (searcher) {
        float x[kMaxDK];
#pragma unroll
        for (int d = 0; d < kMaxDK; ++d) x[d] = q[d];
        const K z = (K)code_of(x, g.dK, g.bits);
        const int rk = rank_of<K, 4>(g, otab, h, order_codes + plane, z, cC, lane);
        const int st = min(max(rk - (g.k + 1) / 2, 0), cC - g.k);
        float wmin = INFINITY;
        int row[2];
        float d2[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) row[u] = window_row(st, u * 32 + lane, u * 32 + lane < g.k);
#pragma unroll
        for (int u = 0; u < 2; ++u) d2[u] = dist(max(row[u], 0));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            wr_sh[u * 32 + lane] = row[u];
            const float x2 = row[u] >= 0 ? d2[u] : INFINITY;
            wmin = fminf(wmin, x2);
            const float w = row[u] >= 0 && !soft ? weight_rt(g.wk, x2, 0.f, inv_g2) : 0.f;
            sum += w;
            ww_sh[u * 32 + lane] = soft ? x2 : w;
        }
        wmin = warp_min(wmin);
        if (lane == 0) {
            st_sh = st;
            red_m[NW - 1] = wmin;                                // the searcher's own slot
        }
    } else if (cr < sharers) {
        const int groups = own / LPR;
        for (int j0 = k0; j0 < k1; j0 += kSeg) {
            const int n = min(kSeg, k1 - j0);
            // The first rows of this thread's pieces, then the weights.
            if (grp < groups) {
                int id[U];
#pragma unroll
                for (int u = 0; u < U; ++u) id[u] = page_id(ptab, min(j0 + grp + u * groups, i), g.c.psh);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int r = grp + u * groups, row = r < n ? row_of(id[u], j0 + r) : -1;
                    buf[u].load(v_pages + (int64_t)max(row, 0) * g.dV, sub, row >= 0 && sub < ppr);
                }
            }
            float dmin = INFINITY;
            for (int r = tid; r < n; r += own) {
                const int row = row_of(page_id(ptab, j0 + r, g.c.psh), j0 + r);
                if (row < 0) set_status(g.status, ZETA_ERR_BOUNDS);
                const float d2 = dist(max(row, 0));
                const float x2 = row >= 0 ? d2 : INFINITY;
                row_sh[r] = row;
                if (soft) {
                    w_sh[r] = x2;
                    dmin = fminf(dmin, x2);
                } else {
                    const float w = row >= 0 ? weight_rt(g.wk, x2, 0.f, inv_g2) : 0.f;
                    w_sh[r] = w;
                    sum += w;
                }
            }
            if (soft) {                                          // onto the least distance so far
                dmin = warp_min(dmin);
                if (lane == 0) red_s[warp] = dmin;
                bar_own(own);
                for (int w = 0; w < own / 32; ++w) dmin = fminf(dmin, red_s[w]);
                if (dmin < m_own) {
                    const float f = m_own == INFINITY ? 0.f : expf((dmin - m_own) * inv_g2);
#pragma unroll
                    for (int e = 0; e < NA; ++e) acc[e] = mul2(acc[e], dup2(f));
                    sum *= f;
                    m_own = dmin;
                }
                for (int r = tid; r < n; r += own) {
                    const float w = row_sh[r] >= 0 ? weight_of<kWSoftmax>(w_sh[r], m_own, inv_g2) : 0.f;
                    w_sh[r] = w;
                    sum += w;
                }
            }
            bar_own(own);
            stream(row_sh, w_sh, n, groups, buf, true);
            if (j0 + kSeg < k1) bar_own(own);                    // the arrays are free again
        }
    }
    if (!window && g.idx && cr == 0)
        for (int slot = tid; slot < g.k; slot += NT) g.idx[(int64_t)rid * g.k + slot] = -1;

    // The window, by all threads; for the softmax everything onto one shift.
    if (win_here) {
        if (soft && lane == 0 && !searcher) red_m[warp] = m_own;
        __syncthreads();
        const int st = st_sh;
        float m = m_own;
        if (soft) {
            for (int w = 0; w < NW; ++w) m = fminf(m, red_m[w]);
            if (tid < kWin) {
                const float w = wr_sh[tid] >= 0 ? weight_of<kWSoftmax>(ww_sh[tid], m, inv_g2) : 0.f;
                const float f = m_own == INFINITY ? 0.f : expf((m - m_own) * inv_g2);
                sum = sum * f + w;
                ww_sh[tid] = w;
            } else if (m_own != INFINITY) {
                sum *= expf((m - m_own) * inv_g2);
            }
            const float f = m_own == INFINITY ? 0.f : m_own == m ? 1.f : expf((m - m_own) * inv_g2);
#pragma unroll
            for (int e = 0; e < NA; ++e) acc[e] = mul2(acc[e], dup2(f));
            m_own = m;
            __syncthreads();
        }
        stream(wr_sh, ww_sh, min(kWin, g.k), NT / LPR, buf, false);
        for (int t0 = kWin; t0 < g.k; t0 += kSeg) {              // windows of more entries
            const int n = min(kSeg, g.k - t0);
            float dmin = INFINITY;
            __syncthreads();
            for (int r = tid; r < n; r += NT) {
                const int row = window_row(st, t0 + r, true);
                const float d2 = dist(max(row, 0)), x2 = row >= 0 ? d2 : INFINITY;
                row_sh[r] = row;
                dmin = fminf(dmin, x2);
                const float w = row >= 0 && !soft ? weight_rt(g.wk, x2, 0.f, inv_g2) : 0.f;
                w_sh[r] = soft ? x2 : w;
                sum += w;
            }
            if (soft) {
                dmin = warp_min(dmin);
                if (lane == 0) red_m[warp] = dmin;
                __syncthreads();
                for (int w = 0; w < NW; ++w) dmin = fminf(dmin, red_m[w]);
                if (dmin < m_own) {
                    const float f = m_own == INFINITY ? 0.f : expf((dmin - m_own) * inv_g2);
#pragma unroll
                    for (int e = 0; e < NA; ++e) acc[e] = mul2(acc[e], dup2(f));
                    sum *= f;
                    m_own = dmin;
                }
                for (int r = tid; r < n; r += NT) {
                    const float w = row_sh[r] >= 0 ? weight_of<kWSoftmax>(w_sh[r], m_own, inv_g2) : 0.f;
                    w_sh[r] = w;
                    sum += w;
                }
            }
            __syncthreads();
            stream(row_sh, w_sh, n, NT / LPR, buf, false);
        }
    }

    // Join the threads of a column, the warps, the blocks.
    sum = warp_sum(sum);
    if constexpr (LPR < 32) {
#pragma unroll
        for (int o = 16; o >= LPR; o >>= 1)
#pragma unroll
            for (int e = 0; e < NA; ++e) {
                acc[e].x += __shfl_xor_sync(kFull, acc[e].x, o);
                acc[e].y += __shfl_xor_sync(kFull, acc[e].y, o);
            }
    }
    if (LPR >= 32 || lane < LPR) {
#pragma unroll
        for (int e = 0; e < P::N; ++e) part[warp][(lane % (LPR < 32 ? LPR : 32)) * P::N + e] = e & 1 ? acc[e / 2].y : acc[e / 2].x;
    }
    __syncthreads();                                             // red_s may still be read above
    if (lane == 0) red_s[warp] = sum;
    __syncthreads();
    float total = 0.f;
    for (int w = 0; w < NW; ++w) total += red_s[w];
    constexpr int WPR = LPR <= 32 ? 1 : LPR / 32;                // warps that share a row
    auto column = [&](int d) {
        float o = 0.f;
        const int piece = d / P::N, at = (piece % 32) * P::N + d % P::N;
        for (int w = piece / 32; w < NW; w += WPR) o += part[w][LPR <= 32 ? d : at];
        return o;
    };
    if (cs == 1) {
        for (int d = tid; d < g.dV; d += NT) VT<V>::st(out + (int64_t)rid * g.dV + d, __fdiv_rn(column(d), total));
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
            VT<V>::st(out + (int64_t)rid * g.dV + d, __fdiv_rn(o, ssum));
        }
        if (tid == 0) g.rowsum[rid] = ssum;
    }
    cl.sync();                                                   // read before any block ends
}

template <typename K, typename V, bool WIDE, int LPR, int NT = 256>
cudaError_t run_rows(const Args &g, const Prob &p, const void *order_codes, const void *v_pages,
                     void *out, int ppr, cudaStream_t st) {
    const int64_t rows = p.S * g.c.n;
    // Blocks per token: split where the tokens alone leave SMs idle, as far as the own
    // chunk has a key per thread, beside the block of the window.
    const int most = p.C <= NT ? 2 : p.C <= 3 * NT ? 4 : 8;
    int cs = 1;
    while (cs < most && rows * cs * 2 <= 152 * 4) cs *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows * cs));
    cfg.blockDim = dim3(NT);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, cache_rows_kernel<K, V, WIDE, LPR, NT>, g,
                                             static_cast<const K *>(order_codes),
                                             static_cast<const V *>(v_pages),
                                             static_cast<V *>(out), cs, ppr);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename K, typename V>
cudaError_t dispatch_rows(const Args &g, const Prob &p, const void *order_codes,
                          const void *v_pages, void *out, cudaStream_t st) {
    const int bytes = p.dV * (int)sizeof(V);
    const bool wide = bytes % 16 == 0;
    const int ppr = wide ? bytes / 16 : p.dV;
#define ZETA_ROWS(WIDE, LPR) run_rows<K, V, WIDE, LPR>(g, p, order_codes, v_pages, out, ppr, st)
    if (!wide && ppr <= 32) return ZETA_ROWS(false, 32);
    if (!wide && ppr <= 64) return ZETA_ROWS(false, 64);
    if (!wide)                     // 512 threads: a row group beside the searching warp
        return run_rows<K, V, false, 256, 512>(g, p, order_codes, v_pages, out, ppr, st);
    if (ppr <= 4) return ZETA_ROWS(true, 4);
    if (ppr <= 8) return ZETA_ROWS(true, 8);
    if (ppr <= 16) return ZETA_ROWS(true, 16);
    if (ppr <= 32) return ZETA_ROWS(true, 32);
    return ZETA_ROWS(true, 64);
#undef ZETA_ROWS
}

}  // namespace

cudaError_t launch_cache_attend(const Prob &p, const Cache &c, const float *q, const float *gamma,
                                const float *k_pages, const void *v_pages,
                                const void *order_codes, const int32_t *order_idx, void *out,
                                float *rowsum, int32_t *idx, int32_t *status, cudaStream_t st) {
    const Args g{c, q, gamma, k_pages, order_idx, rowsum, idx, status,
                 p.N, p.H, p.dK, p.dV, p.k, p.C, p.bits, p.wk};
    if (p.vdt == ZETA_BF16 && p.dV % 8 == 0 && p.dV <= 128 && p.dK <= 4 && c.n >= kTileRows) {
        const TileArgs t{c, q, gamma, k_pages, static_cast<const __nv_bfloat16 *>(v_pages),
                         order_codes, order_idx, static_cast<__nv_bfloat16 *>(out), rowsum, idx,
                         status, p.N, p.H, p.dK, p.dV, p.k, p.C, p.bits, p.wk, p.code64};
        // Sixteen rows a block until the rows fill the SMs 128 at a time.
        const bool wide = p.S * c.n >= 152 * 128;
        return p.dV <= 64 ? launch_cache_tile64(p, t, wide, st) : launch_cache_tile128(p, t, wide, st);
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
