// cache_attend.cu -- attention of new tokens over the paged cache.
//
// Passages: as for the select and attend steps (OpenReview discussion of "ZETA:
// Leveraging Z-order Curves for Efficient Top-k Attention", reply A3 "Chunking
// ...": binary search of the insertion position and the window around it; reply
// A2 "Discussion on its robustness": the Cauchy softmax).
//
// Row kernel: one new token of one head per block, or per cluster of blocks when
// there are few of them.  The work is a read of the token's own chunk (up to C
// keys and values, contiguous within pages) and of k scattered rows, bound by
// HBM when many tokens come at once and by the chain of dependent loads (rank
// search, window entry, page, row) when few do:
//  * A warp takes 32 keys at a time: lane j computes the weight of key j while
//    the 16-byte pieces of the 32 value rows, LPR lanes per row, are in flight.
//  * The rank search probes 32 P entries of the sorted prefix per step instead
//    of one.
//  * One warp searches while the others read the own chunk; in a cluster the
//    last block takes the window and the others share the own chunk.
//  * Sums of weights and of weighted values are held in float32 per warp and
//    joined in a fixed order, in shared memory and across the cluster through
//    distributed shared memory: no workspace, one launch, the same bits each run.
#include <cooperative_groups.h>

#include "cache_tile.cuh"

namespace zeta {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kTileRows = 4;           // rows of a call from which the tile kernel runs
constexpr int kThreads = kWarps * 32;

// One (b, h, t): where its keys are and what they are weighed with.
struct Row {
    const int32_t *ptab, *otab;
    float q[kMaxDK];
    float inv_g2;
    int h, i, cC;              // head, position, first key of the own chunk
};

struct Args {
    Cache c;
    const float *q, *gamma, *k_pages;
    const int32_t *order_idx;
    float *rowsum;
    int32_t *idx, *status;
    int N, H, dK, dV, k, C, bits, wk;
};

// How a value row is cut among lanes: pieces of 16 bytes (WIDE) or single
// values, LPR lanes per row, NP pieces per lane.
template <typename V, int LPR_, int NP_, bool WIDE>
struct Cut {
    using Val = V;
    static constexpr int LPR = LPR_, NP = NP_;
    static constexpr int EPP = WIDE ? 16 / (int)sizeof(V) : 1;     // values per piece
    static constexpr int RPS = 32 / LPR;                           // rows per step
    static constexpr int U = !WIDE ? 4 : LPR < 8 / NP ? LPR : 8 / NP;  // steps in flight
    struct Piece {
        uint32_t w[WIDE ? 4 : 1];
    };
    static __device__ __forceinline__ Piece load(const V *row, int piece, bool ok) {
        Piece p;
        if constexpr (WIDE) {
            const uint4 x = ld16_if(reinterpret_cast<const uint4 *>(row) + piece, ok);
            p.w[0] = x.x; p.w[1] = x.y; p.w[2] = x.z; p.w[3] = x.w;
        } else if constexpr (sizeof(V) == 2) {
            p.w[0] = ld2_if(row + piece, ok);
        } else {
            p.w[0] = ld4_if(row + piece, ok);
        }
        return p;
    }
    static __device__ __forceinline__ float value(const Piece &p, int e) {
        if constexpr (sizeof(V) == 2)
            return __uint_as_float(e & 1 ? p.w[e >> 1] & 0xffff0000u : p.w[e >> 1] << 16);
        else return __uint_as_float(p.w[e]);
    }
};

// A warp's running sums: acc over the values of its lane's pieces for the rows
// its lane loads, s over the lane's own keys, m the softmax shift (smallest
// squared distance so far, the same in all lanes).
template <typename X>
struct Sums {
    float acc[X::NP * X::EPP];
    float s, m;
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < X::NP * X::EPP; ++e) acc[e] = 0.f;
        s = 0.f;
        m = INFINITY;
    }
};

__device__ __forceinline__ float weight_rt(int wk, float d2, float m, float inv_g2) {
    if (wk == kWSoftmax) return weight_of<kWSoftmax>(d2, m, inv_g2);
    if (wk == kWInvEuclid) return weight_of<kWInvEuclid>(d2, m, inv_g2);
    return weight_of<kWCauchy>(d2, m, inv_g2);
}

// Up to 32 keys: lane j < cnt holds the row of key j (-1: none).
template <typename X>
__device__ __forceinline__ void take(Sums<X> &a, const Args &g, const Row &r,
                                     const typename X::Val *v_pages, int row, int cnt, int lane,
                                     int ppr) {
    using V = typename X::Val;
    using Piece = typename X::Piece;
    const int sub = lane % X::LPR, grp = lane / X::LPR;
    const int steps = (cnt + X::RPS - 1) / X::RPS;
    float x[kMaxDK];
    load_point(x, g.k_pages + (int64_t)max(row, 0) * g.dK, g.dK);
    float w = 0.f;
    for (int u0 = 0; u0 < steps; u0 += X::U) {
        Piece buf[X::U][X::NP];
#pragma unroll
        for (int u = 0; u < X::U; ++u) {
            const int rr = __shfl_sync(kFull, row, ((u0 + u) * X::RPS + grp) & 31);
            const bool ok = u0 + u < steps && rr >= 0;
            const V *vr = v_pages + (int64_t)max(rr, 0) * g.dV;
#pragma unroll
            for (int p = 0; p < X::NP; ++p) {
                const int pc = sub + p * X::LPR;
                buf[u][p] = X::load(vr, pc, ok && pc < ppr);
            }
        }
        if (u0 == 0) {                                  // the weights, once the rows are asked for
            float d2 = 0.f;
#pragma unroll
            for (int d = 0; d < kMaxDK; ++d) {
                if (d < g.dK) {
                    const float e = r.q[d] - x[d];
                    d2 = __fmaf_rn(e, e, d2);
                }
            }
            if (row < 0) d2 = INFINITY;
            if (g.wk == kWSoftmax) {
                float pm = d2;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) pm = fminf(pm, __shfl_xor_sync(kFull, pm, o));
                if (pm < a.m) {
                    const float sc = a.m == INFINITY ? 0.f : expf((pm - a.m) * r.inv_g2);
#pragma unroll
                    for (int e = 0; e < X::NP * X::EPP; ++e) a.acc[e] *= sc;
                    a.s *= sc;
                    a.m = pm;
                }
            }
            w = row >= 0 ? weight_rt(g.wk, d2, a.m, r.inv_g2) : 0.f;
            a.s += w;
        }
#pragma unroll
        for (int u = 0; u < X::U; ++u) {
            const float wu = __shfl_sync(kFull, w, ((u0 + u) * X::RPS + grp) & 31);
            if (u0 + u < steps) {
#pragma unroll
                for (int p = 0; p < X::NP; ++p)
#pragma unroll
                    for (int e = 0; e < X::EPP; ++e)
                        a.acc[p * X::EPP + e] =
                            __fmaf_rn(wu, X::value(buf[u][p], e), a.acc[p * X::EPP + e]);
            }
        }
    }
}

// Entries of the prefix with a code <= z: a warp probes 32 P of them per step.
template <typename K, int P>
__device__ __forceinline__ int rank_of(const Args &g, const Row &r, const K *codes, K z, int M,
                                       int lane) {
    int lo = 0, hi = M;
    while (lo < hi) {
        const int step = (hi - lo + 32 * P - 1) / (32 * P);
        int le = 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const int e = lo + (p * 32 + lane + 1) * step - 1;
            bool in = false;
            if (e < hi) {
                const int row = page_row(r.otab, e, r.h, g.H, g.c.psh, g.c.pmask, g.c.opages);
                if (row < 0) set_status(g.status, ZETA_ERR_BOUNDS);
                in = row >= 0 && __ldg(codes + row) <= z;
            }
            le += __popc(__ballot_sync(kFull, in));
        }
        lo = min(lo + le * step, hi);
        hi = min(hi, lo + step - 1);
    }
    return lo;
}

struct Part {
    float acc[kMaxDV];
    float s, m;
};

// Sums of `cnt` parts (the p-th given by at(p)) at column d, in order.
template <typename At>
__device__ __forceinline__ float join(int wk, float inv_g2, int cnt, int d, At at, float &s,
                                      float &m) {
    m = INFINITY;
    if (wk == kWSoftmax)
        for (int p = 0; p < cnt; ++p) m = fminf(m, at(p)->m);
    float o = 0.f;
    s = 0.f;
    for (int p = 0; p < cnt; ++p) {
        const Part *x = at(p);
        const float f = wk != kWSoftmax ? 1.f
                        : x->m == INFINITY ? 0.f : expf((m - x->m) * inv_g2);
        o = __fmaf_rn(f, x->acc[d], o);
        s = __fmaf_rn(f, x->s, s);
    }
    return o;
}

template <typename K, typename X>
__global__ void __launch_bounds__(kThreads, 4)
cache_rows_kernel(Args g, const K *__restrict__ order_codes,
                  const typename X::Val *__restrict__ v_pages, typename X::Val *__restrict__ out,
                  int cs, int ppr) {
    using V = typename X::Val;
    __shared__ Part part[kWarps];
    __shared__ Part mine;
    __shared__ int rank_sh;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned rid = blockIdx.x / (unsigned)cs;
    const int cr = (int)(blockIdx.x - rid * (unsigned)cs);       // block in the cluster
    const unsigned s = rid / (unsigned)g.c.n;
    const int t = (int)(rid - s * (unsigned)g.c.n);
    const int b = (int)(s / (unsigned)g.H);
    Row r;
    r.h = (int)(s - (unsigned)b * (unsigned)g.H);
    const Seq seq = seq_of(g.c, b, g.N, g.status);
    if (t >= seq.count) return;                                  // the whole cluster returns
    r.ptab = g.c.ptab + (int64_t)b * g.c.tlen;
    r.otab = g.c.otab + (int64_t)b * g.c.tlen;
    r.i = seq.start + t;
    const int chunk = r.i / g.C;
    r.cC = chunk * g.C;
    load_point(r.q, g.q + (int64_t)rid * g.dK, g.dK);
    const float gm = g.gamma[r.h];
    r.inv_g2 = __frcp_rn(gm * gm);
    const int64_t plane = ((int64_t)g.c.opages * g.H << g.c.psh) * (chunk & 1);

    Sums<X> a;
    a.zero();
    const bool window = chunk > 0;
    const bool win_here = window && cr == cs - 1;
    // Own chunk: blocks 0 .. cs-2 of a cluster (all of them without a window);
    // in a lone block the warps that do not search.
    const bool own_here = cs == 1 || !window || cr < cs - 1;
    if (win_here && warp == 0) {
        const K z = (K)code_of(r.q, g.dK, g.bits);
        const int rk = cs > 1 ? rank_of<K, 8>(g, r, order_codes + plane, z, r.cC, lane)
                              : rank_of<K, 2>(g, r, order_codes + plane, z, r.cC, lane);
        if (lane == 0) rank_sh = rk;
    } else if (own_here) {
        const int skip = win_here ? 1 : 0;
        const int workers = cs == 1 ? kWarps - skip : (window ? cs - 1 : cs) * kWarps;
        const int me = cs == 1 ? warp - skip : cr * kWarps + warp;
        for (int j0 = r.cC + 32 * me; j0 <= r.i; j0 += 32 * workers) {
            const int j = j0 + lane;
            int row = -1;
            if (j <= r.i) {
                row = page_row(r.ptab, j, r.h, g.H, g.c.psh, g.c.pmask, g.c.pages);
                if (row < 0) set_status(g.status, ZETA_ERR_BOUNDS);
            }
            take<X>(a, g, r, v_pages, row, min(32, r.i - j0 + 1), lane, ppr);
        }
    }
    if (win_here) {
        __syncthreads();
        const int st = min(max(rank_sh - (g.k + 1) / 2, 0), r.cC - g.k);
        const int per = min(32, (g.k + kWarps - 1) / kWarps);
        for (int t0 = warp * per; t0 < g.k; t0 += kWarps * per) {
            int row = -1;
            const int slot = t0 + lane;
            if (lane < per && slot < g.k) {
                const int orow = page_row(r.otab, st + slot, r.h, g.H, g.c.psh, g.c.pmask,
                                          g.c.opages);
                int j = orow >= 0 ? __ldg(g.order_idx + plane + orow) : -1;
                if ((unsigned)j < (unsigned)r.cC)
                    row = page_row(r.ptab, j, r.h, g.H, g.c.psh, g.c.pmask, g.c.pages);
                else j = -1;
                if (row < 0) set_status(g.status, ZETA_ERR_BOUNDS);
                if (g.idx) g.idx[(int64_t)rid * g.k + slot] = j;
            }
            take<X>(a, g, r, v_pages, row, min(per, g.k - t0), lane, ppr);
        }
    } else if (!window && g.idx && cr == 0) {
        for (int slot = threadIdx.x; slot < g.k; slot += kThreads)
            g.idx[(int64_t)rid * g.k + slot] = -1;
    }

    // Join lanes, warps, blocks.
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a.s += __shfl_xor_sync(kFull, a.s, o);
        if (o >= X::LPR) {
#pragma unroll
            for (int e = 0; e < X::NP * X::EPP; ++e)
                a.acc[e] += __shfl_xor_sync(kFull, a.acc[e], o);
        }
    }
    if (lane < X::LPR) {
#pragma unroll
        for (int p = 0; p < X::NP; ++p)
            if (lane + p * X::LPR < ppr) {
#pragma unroll
                for (int e = 0; e < X::EPP; ++e)
                    part[warp].acc[(lane + p * X::LPR) * X::EPP + e] = a.acc[p * X::EPP + e];
            }
    }
    if (lane == 0) {
        part[warp].s = a.s;
        part[warp].m = a.m;
    }
    __syncthreads();
    float sum = 0.f, m = 0.f, o = 0.f;
    const int d = threadIdx.x;                                   // dV <= kThreads columns
    if (d < g.dV) o = join(g.wk, r.inv_g2, kWarps, d, [&](int p) { return &part[p]; }, sum, m);
    if (cs > 1) {
        if (d < g.dV) mine.acc[d] = o;
        if (d == 0) {
            mine.s = sum;
            mine.m = m;
        }
        cg::cluster_group cl = cg::this_cluster();
        cl.sync();
        if (cr == 0 && d < g.dV)
            o = join(g.wk, r.inv_g2, cs, d, [&](int p) { return cl.map_shared_rank(&mine, p); },
                     sum, m);
        cl.sync();                                               // read before any block ends
        if (cr != 0) return;
    }
    if (d < g.dV) VT<V>::st(out + (int64_t)rid * g.dV + d, __fdiv_rn(o, sum));
    if (d == 0) g.rowsum[rid] = sum;
}

template <typename K, typename X>
cudaError_t run_rows(const Args &g, const Prob &p, const void *order_codes, const void *v_pages,
                     void *out, cudaStream_t st) {
    using V = typename X::Val;
    const int64_t rows = p.S * g.c.n;
    // Blocks per token: split where the tokens alone leave SMs idle, as far as the
    // own chunk has work for (32 keys per warp) beside the block of the window.
    const int most = p.C <= 32 * kWarps ? 2 : p.C <= 96 * kWarps ? 4 : 8;
    int cs = 1;
    while (cs < most && rows * cs * 2 <= 152 * 4) cs *= 2;
    const int ppr = p.dV / X::EPP;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows * cs));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, cache_rows_kernel<K, X>, g,
                                       static_cast<const K *>(order_codes),
                                       static_cast<const V *>(v_pages), static_cast<V *>(out), cs,
                                       ppr);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <typename K, typename V>
cudaError_t dispatch_rows(const Args &g, const Prob &p, const void *order_codes,
                          const void *v_pages, void *out, cudaStream_t st) {
    const int bytes = p.dV * (int)sizeof(V);
    if (bytes % 16 != 0)
        return run_rows<K, Cut<V, 32, 8, false>>(g, p, order_codes, v_pages, out, st);
    if (bytes <= 64) return run_rows<K, Cut<V, 4, 1, true>>(g, p, order_codes, v_pages, out, st);
    if (bytes <= 128) return run_rows<K, Cut<V, 8, 1, true>>(g, p, order_codes, v_pages, out, st);
    if (bytes <= 256) return run_rows<K, Cut<V, 16, 1, true>>(g, p, order_codes, v_pages, out, st);
    if (bytes <= 512) return run_rows<K, Cut<V, 32, 1, true>>(g, p, order_codes, v_pages, out, st);
    return run_rows<K, Cut<V, 32, 2, true>>(g, p, order_codes, v_pages, out, st);
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
