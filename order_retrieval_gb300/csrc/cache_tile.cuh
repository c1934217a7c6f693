// cache_tile.cuh -- attention of many new tokens per sequence over the paged
// cache: bf16 values, d_V a multiple of 8 up to 128, d_K <= 4.
//
// Same definition as the row kernel (cache_attend.cu).  A block of NW warps takes
// 16 WM query rows of one head and one chunk.
//  * Rank: the first code of every block of 2^fsh prefix entries is staged in
//    shared memory; a warp finds a row's block there and its rank among the
//    block's entries with one coalesced read of up to 64.
//  * Own chunk: key tiles staged by cp.async through the page table into
//    swizzled shared memory; weights are built straight in mma A fragments and
//    rounded to bf16 once, products accumulate in float32, row sums come from the
//    unrounded weights.  NW / WM warps split each tile's keys and join at the end.
//  * Window, rows that have little in common (GATHER): a warp takes one row at a
//    time; 64 gathered value rows are in flight, four lanes per row, and the
//    weighted sum V^T w runs on the tensor cores (8x8 blocks transposed in
//    registers, w in column 0 of B).
//  * Window, many rows per prefix entry (BAND): the up to 1024 rows of a piece are
//    dealt to the warps in the order of their codes (a counting sort on the codes'
//    top ten bits), so that the 16 windows of a warp overlap.  The warp walks the
//    prefix positions that any of them covers, 16 at a time through a ring of
//    cp.async stages, as an mma tile whose weights are masked to each row's
//    window: a value row is read once for all rows that take it, and no row pays
//    for its own gather.  The own chunk then takes the block's rows in the order
//    of their positions, so that a warp stops at its last row's causal limit.
//    Dealing changes no row's arithmetic.
//  * A masked weight of zero times a value that is not finite would be NaN: a row
//    whose result is not finite is taken again, key by key, without the others.
#pragma once

#include "cache_gather.cuh"

namespace zeta {

struct TileArgs {
    Cache c;
    const float *q, *gamma, *k_pages;
    const __nv_bfloat16 *v_pages;
    const void *order_codes;
    const int32_t *order_idx;
    __nv_bfloat16 *out;
    float *rowsum;
    int32_t *idx, *status;
    int N, H, dK, dV, k, C, bits, wk, code64;
};

cudaError_t launch_cache_tile64(const Prob &p, const TileArgs &g, bool wide, cudaStream_t st);
cudaError_t launch_cache_tile128(const Prob &p, const TileArgs &g, bool wide, cudaStream_t st);

namespace {

constexpr int kSortRows = 1024, kBuckets = 1024;
constexpr int kFences = 1024;
constexpr int kRing = 4;               // stages of 16 prefix entries per warp
constexpr int kBandRatio = 40;         // prefix entries per row below which rows are dealt

template <int DVP, int WM, int NW>
struct TileSmem {
    static constexpr int TQ = 16 * WM;
    static constexpr int TK = DVP == 64 && NW / WM >= 4 ? 128 : 64;
    static constexpr bool BAND = WM == NW;
    struct Own {
        __nv_bfloat16 v[3][TK * DVP];  // 16-byte chunk c of row r at c ^ (r & 7)
        float4 kt[3][TK];
    };
    struct Band {
        __nv_bfloat16 v[NW][kRing][16 * DVP];
        float4 kt[NW][kRing][16];
    };
    struct Deal {
        int cnt[kBuckets];
        int cuts[2][kSortRows / 32];
        int scan[NW];
    };
    union {
        Own own;
        Band band[BAND ? 1 : 0];
        Deal deal;
        uint64_t fence[kFences];
        float join[WM * (NW / WM - 1) * 16 * (DVP + 4) + 1];
    };
    float win[TQ][DVP + 4];            // window sums
    int rows[4][TK];                   // pool rows of the tile's keys, -1: none
    float swin[TQ], mwin[TQ];
    float lsum[NW][16], lmin[NW][16];  // the key splits' row sums and shifts
    int qrow[TQ];                      // the call's row of query l
    int perm[TQ];                      // query of own-chunk row r (by position)
    int wst[TQ];                       // window start of query l
    int bad;                           // a key of the own chunk has no page
};

__device__ __forceinline__ uint64_t order_code(const TileArgs &g, int64_t at) {
    return g.code64 ? __ldg(static_cast<const unsigned long long *>(g.order_codes) + at)
                    : (uint64_t)__ldg(static_cast<const uint32_t *>(g.order_codes) + at);
}

// One row key by key (a warp, lanes over the value columns): its keys and no
// others enter.  For results that are not finite.
template <int DVP, int DK, int WK>
__device__ __noinline__ void slow_row(const TileArgs &g, int64_t row0, int t, int h, int start,
                                      int cC, int wst, const int32_t *ptab, const int32_t *otab,
                                      int64_t plane, float inv_g2) {
    const int lane = threadIdx.x & 31;
    const float4 q4 = ld_key(g.q + (row0 + t) * g.dK, g.dK);
    const float q[4] = {q4.x, q4.y, q4.z, q4.w};
    const int nw = cC > 0 ? g.k : 0, keys = nw + start + t - cC + 1;
    float acc[DVP / 32], s = 0.f, m = INFINITY;
#pragma unroll
    for (int e = 0; e < DVP / 32; ++e) acc[e] = 0.f;
    for (int pass = WK == kWSoftmax ? 0 : 1; pass < 2; ++pass) {
        for (int i = 0; i < keys; ++i) {
            int j = cC + i - nw;
            if (i < nw) {
                const int row = page_row(otab, wst + i, h, g.H, g.c.psh, g.c.pmask, g.c.opages);
                j = row >= 0 ? g.order_idx[plane + row] : -1;
                if ((unsigned)j >= (unsigned)cC) continue;
            }
            const int row = page_row(ptab, j, h, g.H, g.c.psh, g.c.pmask, g.c.pages);
            if (row < 0) continue;
            const float4 k4 = ld_key(g.k_pages + (int64_t)row * g.dK, g.dK);
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
                if (lane + 32 * e < g.dV)
                    acc[e] = __fmaf_rn(w, __bfloat162float(g.v_pages[(int64_t)row * g.dV + lane + 32 * e]), acc[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < DVP / 32; ++e)
        if (lane + 32 * e < g.dV)
            g.out[(row0 + t) * g.dV + lane + 32 * e] = __float2bfloat16_rn(__fdiv_rn(acc[e], s));
}

template <int DVP, int DK, int WK, int WM, int NW>
__global__ void __launch_bounds__(NW * 32, (DVP == 64 ? 16 : 12) / NW)
cache_tile_kernel(const __grid_constant__ TileArgs g) {
    using Sm = TileSmem<DVP, WM, NW>;
    constexpr bool BAND = Sm::BAND;
    constexpr int TQ = Sm::TQ, TK = Sm::TK, KS = NW / WM;    // KS warps share a row group's keys
    constexpr int kTileThreads = NW * 32;
    constexpr int QW = TQ / NW;                              // window rows per warp
    constexpr int CB = DVP / 64;                             // 64-column blocks
    constexpr int NT = DVP / 8;
    extern __shared__ __align__(16) unsigned char raw[];
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int s = blockIdx.y, b = s / g.H, h = s - b * g.H;
    const Seq seq = seq_of(g.c, b, g.N, g.status);
    if (seq.count == 0) return;
    // The call's rows of this sequence lie in chunk c0 (nA of them) and the next.
    const int c0 = seq.start / g.C;
    const int nA = min(seq.count, (c0 + 1) * g.C - seq.start);
    int x = blockIdx.x;
    const int tA = (nA + TQ - 1) / TQ;
    const bool second = x >= tA;
    if (second) x -= tA;
    const int p0 = second ? nA : 0, np = second ? seq.count - nA : nA;
    if (x * TQ >= np) return;
    const int chunk = c0 + (second ? 1 : 0), cC = chunk * g.C;
    const int blk = x * TQ / kSortRows * kSortRows;          // rows dealt together
    const int bn = min(kSortRows, np - blk), lo = x * TQ - blk, nq = min(TQ, bn - lo);
    const int32_t *ptab = g.c.ptab + (int64_t)b * g.c.tlen, *otab = g.c.otab + (int64_t)b * g.c.tlen;
    const int64_t row0 = (int64_t)s * g.c.n;                 // the call's row 0 of this slice
    const float *qs = g.q + row0 * g.dK;
    const float gm = g.gamma[h];
    const float inv_g2 = __frcp_rn(gm * gm);
    const int64_t plane = ((int64_t)g.c.opages * g.H << g.c.psh) * (chunk & 1);

    auto code_at = [&](int t) {
        float p[kMaxDK];
#pragma unroll
        for (int d = 0; d < kMaxDK; ++d) p[d] = d < DK && d < g.dK ? qs[(int64_t)t * g.dK + d] : 0.f;
        return code_of(p, g.dK, g.bits);
    };

    auto order_row = [&](int id, int e) { return row_in(id, e, h, g.H, g.c.psh, g.c.pmask, g.c.opages); };
    auto pool_row = [&](int id, int t) { return row_in(id, t, h, g.H, g.c.psh, g.c.pmask, g.c.pages); };

    // ---------------------------------------------------- which rows -------
    // Where the prefix has less than kBandRatio entries per row, the windows are
    // walked together, and the rows dealt by code if there is more than one block.
    const bool band = BAND && chunk > 0 && (int64_t)bn * kBandRatio >= cC;
    const bool deal = band && bn > nq;
    if (deal) {
        int *cnt = sm.deal.cnt;
        for (int i = tid; i < kBuckets; i += kTileThreads) cnt[i] = 0;
        __syncthreads();
        const int sh = max(0, g.dK * g.bits - 10);
        int at[kSortRows / kTileThreads];                    // bucket << 16 | place in it
#pragma unroll
        for (int u = 0; u < kSortRows / kTileThreads; ++u) {
            const int l = u * kTileThreads + tid;
            at[u] = 0;
            if (l < bn) {
                const int bk = (int)(code_at(p0 + blk + l) >> sh);
                at[u] = bk << 16 | atomicAdd(&cnt[bk], 1);
            }
        }
        __syncthreads();
        constexpr int PER = kBuckets / kTileThreads;
        int loc[PER], sum = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            loc[i] = sum;
            sum += cnt[tid * PER + i];
        }
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += y;
        }
        if (lane == 31) sm.deal.scan[warp] = inc;
        __syncthreads();
        int before = inc - sum;
        for (int w = 0; w < warp; ++w) before += sm.deal.scan[w];
#pragma unroll
        for (int i = 0; i < PER; ++i) cnt[tid * PER + i] = before + loc[i];
        __syncthreads();
        // Every block of the piece has to deal alike: the places that the atomics
        // gave out differ from block to block, which matters only in the bucket that
        // this block shares with the one before and in the one it shares with the
        // next.  Rows of those two are placed in row order.
        constexpr int NU = kSortRows / kTileThreads;
        unsigned cut[2][NU];                                 // the warp's rows of the two buckets
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int l = u * kTileThreads + tid, bk = at[u] >> 16;
            const int first = cnt[bk], last = bk + 1 < kBuckets ? cnt[bk + 1] : bn;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int edge = lo + e * nq;
                cut[e][u] = __ballot_sync(kFull, l < bn && first < edge && last > edge);
                if (lane == 0) sm.deal.cuts[e][u * NW + warp] = __popc(cut[e][u]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < NU; ++u) {
            const int l = u * kTileThreads + tid, bk = at[u] >> 16;
            if (l < bn) {
                int place = at[u] & 0xffff;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (cut[e][u] >> lane & 1) {
                        place = __popc(cut[e][u] & lanemask_lt());
                        for (int i = 0; i < u * NW + warp; ++i) place += sm.deal.cuts[e][i];
                    }
                }
                const int p = cnt[bk] + place - lo;
                if (p >= 0 && p < nq) sm.qrow[p] = p0 + blk + l;
            }
        }
    } else if (tid < nq) {
        sm.qrow[tid] = p0 + blk + lo + tid;
    }
    if (tid == 0) sm.bad = 0;
    __syncthreads();
    if (tid < TQ) {                                          // order by position
        if (tid < nq) {
            int r = tid;
            if (deal) {
                const int t = sm.qrow[tid];
                r = 0;
                for (int j = 0; j < nq; ++j) r += sm.qrow[j] < t;
            }
            sm.perm[r] = tid;
        } else {
            sm.perm[tid] = -1;
        }
    }

    // ------------------------------------------------------ window part ---
    const int g4 = lane >> 2, s4 = lane & 3;
    const int wl0 = warp * QW, nqw = chunk > 0 ? max(0, min(QW, nq - wl0)) : 0;
    int wst = 0;                                             // lane r < nqw: start of row wl0 + r
    if (chunk > 0) {
        uint64_t *fence = sm.fence;
        int fsh = 5;
        while ((cC >> fsh) >= kFences) ++fsh;
        const int nf = (cC + (1 << fsh) - 1) >> fsh;
        __syncthreads();                                     // the counters have been read
        {
            constexpr int NF = kFences / kTileThreads;
            int fr[NF];
            uint64_t fz[NF];
            bool lost = false;
#pragma unroll
            for (int u = 0; u < NF; ++u)
                fr[u] = page_id(otab, min(u * kTileThreads + tid, nf - 1) << fsh, g.c.psh);
#pragma unroll
            for (int u = 0; u < NF; ++u) {
                fr[u] = order_row(fr[u], min(u * kTileThreads + tid, nf - 1) << fsh);
                fz[u] = order_code(g, plane + max(fr[u], 0));
            }
#pragma unroll
            for (int u = 0; u < NF; ++u) {
                const int f = u * kTileThreads + tid;
                if (f < nf) fence[f] = fr[u] < 0 ? ~0ull : fz[u];
                lost |= fr[u] < 0;
            }
            if (lost) set_status(g.status, ZETA_ERR_BOUNDS);
        }
        __syncthreads();
        uint64_t z = 0;
        int lo_f = 0;
        if (lane < nqw) {
            z = code_at(sm.qrow[wl0 + lane]);
            int hi = nf;
            while (lo_f < hi) {                              // fences with code <= z
                const int mid = (lo_f + hi) >> 1;
                if (fence[mid] <= z) lo_f = mid + 1; else hi = mid;
            }
        }
        // A row's rank among its block's entries: four rows at a time, two entries a
        // lane (blocks of more than 64 entries take further steps).
        constexpr int RB = QW < 4 ? QW : 4;
#pragma unroll 1
        for (int r0 = 0; r0 < nqw; r0 += RB) {
            uint64_t zr[RB];
            int a[RB], e[RB];
#pragma unroll
            for (int i = 0; i < RB; ++i) {
                zr[i] = __shfl_sync(kFull, z, r0 + i);
                const int fr = r0 + i < nqw ? __shfl_sync(kFull, lo_f, r0 + i) : 0;
                a[i] = fr > 0 ? ((fr - 1) << fsh) + 1 : 0;   // entries before a are <= z
                e[i] = fr > 0 ? min(cC, fr << fsh) : 0;      // entries from e on are > z
            }
            for (int len = 1 << fsh; len > 0; ) {            // most entries still open
                const int step = (len + 63) / 64;
                int row[RB][2];
                uint64_t zz[RB][2];
                auto at = [&](int i, int u) { return min(a[i] + (u * 32 + lane + 1) * step - 1, cC - 1); };
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u) row[i][u] = page_id(otab, at(i, u), g.c.psh);
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        row[i][u] = order_row(row[i][u], at(i, u));
                        zz[i][u] = order_code(g, plane + max(row[i][u], 0));
                    }
#pragma unroll
                for (int i = 0; i < RB; ++i) {
                    int le = 0;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const bool open = a[i] + (u * 32 + lane + 1) * step - 1 < e[i];
                        if (open && row[i][u] < 0) set_status(g.status, ZETA_ERR_BOUNDS);
                        le += __popc(__ballot_sync(kFull, open && row[i][u] >= 0 && zz[i][u] <= zr[i]));
                    }
                    a[i] = min(a[i] + le * step, e[i]);
                    e[i] = min(e[i], a[i] + step - 1);
                }
                len = step - 1;
            }
#pragma unroll
            for (int i = 0; i < RB; ++i)
                if (lane == r0 + i) wst = min(max(a[i] - (g.k + 1) / 2, 0), cC - g.k);
        }
        if (lane < nqw) sm.wst[wl0 + lane] = wst;
        __syncthreads();                                     // fences read before the tiles arrive
    }
    // Weights in A fragments and products of KN steps of 16 keys: lane (g4, s4) has
    // rows g4 (qab .x) and g4 + 8 (.y) of its group and keys 2 s4, +1, +8, +9 of a
    // step; mask(key, x, none) puts `none` where a row does not take the key.
    const int tig = s4;
    const float2 ig2 = dup2(inv_g2);
    const int nc = (g.dV + 15) >> 4;                         // 16-column pairs in use
    float2 qab[DK], sab, mab;
    float acc[NT][4];
    auto clear = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
        sab = make_float2(0.f, 0.f);
        mab = make_float2(INFINITY, INFINITY);
    };
    auto take_rows = [&](int ta, int tb) {                   // the call's rows, -1: none
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 a = ta >= 0 ? ld_key(qs + (int64_t)ta * g.dK, g.dK) : z;
        const float4 c = tb >= 0 ? ld_key(qs + (int64_t)tb * g.dK, g.dK) : z;
        const float av[4] = {a.x, a.y, a.z, a.w}, cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int d = 0; d < DK; ++d) qab[d] = make_float2(av[d], cv[d]);
    };
    auto d2ab = [&](const float4 *Ks, int kl) {
        const float4 kv = Ks[kl];
        const float kc[4] = {kv.x, kv.y, kv.z, kv.w};
        float2 d2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int d = 0; d < DK; ++d) {
            const float2 e = sub2(qab[d], dup2(kc[d]));
            d2 = fma2(e, e, d2);
        }
        return d2;
    };
    auto steps = [&](auto kn, const float4 *Ks, const __nv_bfloat16 *Vs, int kb0, auto mask) {
        constexpr int KN = decltype(kn)::value;
        if constexpr (WK == kWSoftmax) {                     // move the shift to the least d2
            float2 tm = make_float2(INFINITY, INFINITY);
#pragma unroll
            for (int ks = 0; ks < KN; ++ks)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int kl = kb0 + ks * 16 + 2 * tig + (e & 1) + (e >> 1) * 8;
                    const float2 d2 = mask(kl, d2ab(Ks, kl), INFINITY);
                    tm = make_float2(fminf(tm.x, d2.x), fminf(tm.y, d2.y));
                }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                tm.x = fminf(tm.x, __shfl_xor_sync(kFull, tm.x, o));
                tm.y = fminf(tm.y, __shfl_xor_sync(kFull, tm.y, o));
            }
            const float2 mn = make_float2(fminf(mab.x, tm.x), fminf(mab.y, tm.y));
            const float fa = mn.x == mab.x ? 1.f : mab.x == INFINITY ? 0.f : __expf((mn.x - mab.x) * inv_g2);
            const float fb = mn.y == mab.y ? 1.f : mab.y == INFINITY ? 0.f : __expf((mn.y - mab.y) * inv_g2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                acc[nt][0] *= fa;
                acc[nt][1] *= fa;
                acc[nt][2] *= fb;
                acc[nt][3] *= fb;
            }
            sab = mul2(sab, make_float2(fa, fb));
            mab = mn;
        }
        float2 sh = mab;                                     // finite even where no key is taken yet
        if constexpr (WK == kWSoftmax)
            sh = make_float2(mab.x == INFINITY ? 0.f : mab.x, mab.y == INFINITY ? 0.f : mab.y);
        const uint32_t vbase = smem_u32(Vs);
#pragma unroll
        for (int ks = 0; ks < KN; ++ks) {
            const int kb = kb0 + ks * 16;
            float wv[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int kl = kb + 2 * tig + (e & 1) + (e >> 1) * 8;
                const float2 w = mask(kl, weight_fast2<WK>(d2ab(Ks, kl), sh, ig2), 0.f);
                wv[e] = w.x;
                wv[4 + e] = w.y;
                sab = add2(sab, w);
            }
            const uint32_t a[4] = {pack_bf16(wv[0], wv[1]), pack_bf16(wv[4], wv[5]),
                                   pack_bf16(wv[2], wv[3]), pack_bf16(wv[6], wv[7])};
            const int m = lane >> 3, key = kb + (m & 1) * 8 + (lane & 7);
#pragma unroll
            for (int n2 = 0; n2 < NT / 2; ++n2) {
                if (n2 < nc) {
                    uint32_t b[4];
                    ldsm_x4_trans(b, vbase + (uint32_t)(key * DVP + (((n2 * 2 + (m >> 1)) ^ (key & 7)) * 8)) * 2u);
                    mma16816(acc[2 * n2], a, b[0], b[1]);
                    mma16816(acc[2 * n2 + 1], a, b[2], b[3]);
                }
            }
        }
    };
    const int ppr = g.dV >> 3;                               // 16-byte pieces per value row

    if constexpr (BAND) if (band) {
        // ------------------------------------ windows walked together ------
        clear();
        const int none = INT_MAX;
        take_rows(g4 < nqw ? sm.qrow[wl0 + g4] : -1, g4 + 8 < nqw ? sm.qrow[wl0 + g4 + 8] : -1);
        const int far = -(1 << 30);                          // no position is within k of it
        const int wa = __shfl_sync(kFull, wst, g4), wb = __shfl_sync(kFull, wst, g4 + 8);
        const int sta = g4 < nqw ? wa : far, stb = g4 + 8 < nqw ? wb : far;
        auto next = [&](int p) {                             // first position >= p that a row takes
            const int c = p < cC && lane < nqw && wst + g.k > p ? max(wst, p) : none;
            return __reduce_min_sync(kFull, c);
        };
        const int l16 = lane & 15;
        auto entry = [&](int bp) { return min(bp == none ? 0 : bp + l16, cC - 1); };   // lane's entry of a block
        auto &ring = sm.band[0];
        auto copy = [&](int stage, int row) {                // an entry without a row: infinitely far
            const float *kp = g.k_pages + (int64_t)max(row, 0) * g.dK;
            if (lane < 16) {
                float *kd = reinterpret_cast<float *>(&ring.kt[warp][stage][lane]);
#pragma unroll
                for (int d = 0; d < DK; ++d) {
                    if (row < 0) kd[d] = INFINITY;
                    else if (d < g.dK) cp_async4(smem_u32(kd + d), kp + d, 4);
                    else kd[d] = 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < DVP / 16; ++i) {
                const int id = i * 32 + lane, r = id / (DVP / 8), ch = id % (DVP / 8);
                const int pr = __shfl_sync(kFull, row, r);
                if (ch < ppr)
                    cp_async16(smem_u32(&ring.v[warp][stage][r * DVP + ((ch ^ (r & 7)) * 8)]),
                               g.v_pages + (int64_t)max(pr, 0) * g.dV + ch * 8, pr >= 0 ? 16 : 0);
            }
            cp_async_commit();
        };
        // Block i is walked while blocks i+1, i+2 arrive and i+3 is asked for; the
        // pages of the tokens of i+4, the tokens of i+5 and the pages of the entries of
        // i+6 are on their way, each looked at one turn later.
        int bp[7];
        bp[0] = next(0);
#pragma unroll
        for (int i = 1; i < 7; ++i) bp[i] = bp[i - 1] == none ? none : next(bp[i - 1] + 16);
        int oid[7], tok[6], tid_[5];
#pragma unroll
        for (int i = 0; i < 7; ++i) oid[i] = page_id(otab, entry(bp[i]), g.c.psh);
        bool lost = false;
        auto ask_tok = [&](int id, int block) {              // the token of the lane's entry
            const int row = order_row(id, entry(block));
            lost |= block != none && row < 0;
            return ldi_if(g.order_idx + plane + row, row >= 0);
        };
        auto ask_page = [&](int j) { return page_id(ptab, (unsigned)j < (unsigned)cC ? j : 0, g.c.psh); };
        auto got_row = [&](int id, int j, int block) {       // -1: no entry, or dropped
            if (block == none || block + l16 >= cC) return -1;
            const int row = (unsigned)j < (unsigned)cC ? pool_row(id, j) : -1;
            lost |= row < 0;
            return row;
        };
#pragma unroll
        for (int i = 0; i < 6; ++i) tok[i] = ask_tok(oid[i], bp[i]);
#pragma unroll
        for (int i = 0; i < 5; ++i) tid_[i] = ask_page(tok[i]);
#pragma unroll
        for (int i = 0; i < 3; ++i) copy(i, got_row(tid_[i], tok[i], bp[i]));
        int id3 = tid_[3], j3 = tok[3], id4 = tid_[4], j4 = tok[4], j5 = tok[5], o6 = oid[6];
        for (int i = 0; bp[0] != none; ++i) {
            const int row = got_row(id3, j3, bp[3]);
            cp_async_wait<2>();
            __syncwarp();                                    // block i is here, i - 1 used up
            copy((i + 3) & 3, row);
            const int nb = bp[6] == none ? none : next(bp[6] + 16);
            id3 = id4;
            j3 = j4;
            id4 = ask_page(j5);
            j4 = j5;
            j5 = ask_tok(o6, bp[6]);
            o6 = page_id(otab, entry(nb), g.c.psh);
            const int base = bp[0];
            steps(std::integral_constant<int, 1>{}, ring.kt[warp][i & 3], ring.v[warp][i & 3], 0,
                  [&](int kl, float2 x, float no) {
                      return make_float2((unsigned)(base + kl - sta) < (unsigned)g.k ? x.x : no,
                                         (unsigned)(base + kl - stb) < (unsigned)g.k ? x.y : no);
                  });
#pragma unroll
            for (int e = 0; e < 6; ++e) bp[e] = bp[e + 1];
            bp[6] = nb;
        }
        if (lost) set_status(g.status, ZETA_ERR_BOUNDS);
        cp_async_wait<0>();
        if (g.idx) {
            for (int r = 0; r < nqw; ++r) {
                const int st = __shfl_sync(kFull, wst, r);
                for (int u = lane; u < g.k; u += 32) {
                    const int row = page_row(otab, st + u, h, g.H, g.c.psh, g.c.pmask, g.c.opages);
                    const int j = row >= 0 ? __ldg(g.order_idx + plane + row) : -1;
                    g.idx[(row0 + sm.qrow[wl0 + r]) * g.k + u] = (unsigned)j < (unsigned)cC ? j : -1;
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            if (nt < 2 * nc) {
                *reinterpret_cast<float2 *>(&sm.win[wl0 + g4][nt * 8 + 2 * tig]) = make_float2(acc[nt][0], acc[nt][1]);
                *reinterpret_cast<float2 *>(&sm.win[wl0 + g4 + 8][nt * 8 + 2 * tig]) = make_float2(acc[nt][2], acc[nt][3]);
            }
        float sa = sab.x, sb = sab.y;
#pragma unroll
        for (int o = 1; o <= 2; o <<= 1) {
            sa += __shfl_xor_sync(kFull, sa, o);
            sb += __shfl_xor_sync(kFull, sb, o);
        }
        if (tig == 0) {
            sm.swin[wl0 + g4] = sa;
            sm.swin[wl0 + g4 + 8] = sb;
            sm.mwin[wl0 + g4] = mab.x;
            sm.mwin[wl0 + g4 + 8] = mab.y;
        }
        __syncthreads();                                     // the ring's space goes to the tiles
    }

    // Own-chunk tiles: keys cC .. last row's position (they all exist).
    int tmax = 0;
    for (int l = 0; l < nq; ++l) tmax = max(tmax, sm.qrow[l]);
    const int kend = seq.start + tmax + 1 - cC;              // keys of the chunk that matter
    const int nkt = (kend + TK - 1) / TK;
    auto ask_rows = [&](int kt) {                            // page of the thread's key of tile kt
        return tid < TK && kt * TK + tid < kend ? page_id(ptab, cC + kt * TK + tid, g.c.psh) : -1;
    };
    auto put_rows = [&](int kt, int id) {                    // its pool row, for every thread to see
        if (tid < TK && kt < nkt) {
            const int row = pool_row(id, cC + kt * TK + tid);
            if (row < 0 && kt * TK + tid < kend) {
                set_status(g.status, ZETA_ERR_BOUNDS);
                sm.bad = 1;
            }
            sm.rows[kt & 3][tid] = row;
        }
    };
    auto load_tile = [&](int kt) {                           // into stage kt % 3, asynchronously
        if (kt < nkt) {
            const int bf = kt % 3;
            const int *rows = sm.rows[kt & 3];
#pragma unroll
            for (int i = 0; i < TK * (DVP / 8) / kTileThreads; ++i) {
                const int id = i * kTileThreads + tid;
                const int row = id / (DVP / 8), ch = id % (DVP / 8);
                if (ch < ppr) {
                    const int pr = rows[row];
                    cp_async16(smem_u32(&sm.own.v[bf][row * DVP + ((ch ^ (row & 7)) * 8)]),
                               g.v_pages + (int64_t)max(pr, 0) * g.dV + ch * 8, pr >= 0 ? 16 : 0);
                }
            }
            for (int id = tid; id < TK * DK; id += kTileThreads) {
                const int row = id / DK, d = id - row * DK;
                const int pr = rows[row];
                const bool ok = pr >= 0 && d < g.dK;
                cp_async4(smem_u32(reinterpret_cast<float *>(&sm.own.kt[bf][row]) + d),
                          g.k_pages + (ok ? (int64_t)pr * g.dK + d : 0), ok ? 4 : 0);
            }
        }
        cp_async_commit();
    };
    int kid = ask_rows(3);
    {
        const int i0 = ask_rows(0), i1_ = ask_rows(1), i2 = ask_rows(2);
        put_rows(0, i0);
        put_rows(1, i1_);
        put_rows(2, i2);
    }
    __syncthreads();
    load_tile(0);
    load_tile(1);

    // Window entries come in passes of up to 64 (item it: pass it % np64 of row
    // it / np64).  While pass i is weighted, the pages of the tokens of i+1, the
    // tokens of i+2 and the pages of the entries of i+3 are on their way, each looked
    // at one turn later.
    const int np64 = (g.k + 63) >> 6, items = band ? 0 : nqw * np64;
    bool lost = false;
    struct Two { int u[2]; };
    auto entries = [&](int it, Two &e) {                     // the lane's two entries, -1: none
        const int r = it / np64, t0 = (it - r * np64) << 6;
        const int st = __shfl_sync(kFull, wst, r);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int t = t0 + u * 32 + lane;
            e.u[u] = it < items && t < g.k ? st + t : -1;
        }
    };
    auto ask_oid = [&](const Two &e, Two &id) {
#pragma unroll
        for (int u = 0; u < 2; ++u) id.u[u] = page_id(otab, max(e.u[u], 0), g.c.psh);
    };
    auto ask_tok = [&](const Two &e, const Two &id, Two &j) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int row = order_row(id.u[u], max(e.u[u], 0));
            j.u[u] = ldi_if(g.order_idx + plane + row, row >= 0);
        }
    };
    auto ask_page = [&](const Two &j, Two &id) {
#pragma unroll
        for (int u = 0; u < 2; ++u)
            id.u[u] = page_id(ptab, (unsigned)j.u[u] < (unsigned)cC ? j.u[u] : 0, g.c.psh);
    };
    Two e0, e1, e2, e3, o1, j0, j1, i1;
    if (items > 0) {
        Two o0, o2;
        entries(0, e0);
        entries(1, e1);
        entries(2, e2);
        ask_oid(e0, o0);
        ask_oid(e1, o1);
        ask_oid(e2, o2);
        ask_tok(e0, o0, j0);
        ask_tok(e1, o1, j1);
        ask_page(j0, i1);
        o1 = o2;
    }
    int it = 0;
    for (int r = 0; r < (band ? 0 : QW); ++r) {
        const int l = wl0 + r;
        GatherSum<CB> sum;
        sum.zero();
        float sw = 0.f, mrun = INFINITY;
        if (r < nqw) {
            const int t = sm.qrow[l];
            const float4 qi = ld_key(qs + (int64_t)t * g.dK, g.dK);
            const float qa[4] = {qi.x, qi.y, qi.z, qi.w};
            for (int t0 = 0; t0 < g.k; t0 += 64) {
                // e0: this pass's entries, j0 its tokens, i1 their pages; e1, j1 the next
                // pass's; e2 and o1 entries and pages of the one after.
                float d2v[2];
                int pcur[2];
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if ((unsigned)j0.u[u] >= (unsigned)cC) j0.u[u] = -1;
                    pcur[u] = e0.u[u] >= 0 && j0.u[u] >= 0 ? pool_row(i1.u[u], j0.u[u]) : -1;
                    lost |= e0.u[u] >= 0 && pcur[u] < 0;
                    if (g.idx && e0.u[u] >= 0) g.idx[(row0 + t) * g.k + t0 + u * 32 + lane] = j0.u[u];
                }
                float4 kk[2];
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    kk[u] = ld_key(g.k_pages + (int64_t)max(pcur[u], 0) * g.dK, g.dK);
                gather64<CB>(sum, g.v_pages, g.dV, ppr, pcur, min(4, (g.k - t0 + 15) >> 4), lane, [&] {
                    ask_page(j1, i1);
                    j0 = j1;
                    ask_tok(e2, o1, j1);                     // into j1: a copy would wait for it
                    entries(it + 3, e3);
                    ask_oid(e3, o1);
                    e0 = e1;
                    e1 = e2;
                    e2 = e3;
                    ++it;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const float kc[4] = {kk[u].x, kk[u].y, kk[u].z, kk[u].w};
                        float d2 = 0.f;
#pragma unroll
                        for (int d = 0; d < DK; ++d) {
                            const float e = qa[d] - kc[d];
                            d2 = __fmaf_rn(e, e, d2);
                        }
                        d2v[u] = pcur[u] >= 0 ? d2 : INFINITY;
                    }
                    if constexpr (WK == kWSoftmax) {
                        float pm = fminf(d2v[0], d2v[1]);
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1) pm = fminf(pm, __shfl_xor_sync(kFull, pm, o));
                        if (pm < mrun) {
                            const float sc = mrun == INFINITY ? 0.f : __expf((pm - mrun) * inv_g2);
                            sum.scale(sc);
                            sw *= sc;
                            mrun = pm;
                        }
                    }
                    float w[2];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        w[u] = pcur[u] >= 0 ? weight_fast<WK>(d2v[u], mrun, inv_g2) : 0.f;
                        sw += w[u];
                    }
                    return make_float2(w[0], w[1]);
                });
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sw += __shfl_xor_sync(kFull, sw, o);
        } else if (l < nq && g.idx) {                        // chunk 0 selects nothing
            const int t = sm.qrow[l];
            for (int u = lane; u < g.k; u += 32) g.idx[(row0 + t) * g.k + u] = -1;
        }
        sum.each(lane, [&](int d, float x) { sm.win[l][d] = x; });
        if (lane == 0) {
            sm.swin[l] = sw;
            sm.mwin[l] = mrun;
        }
    }
    if (lost) set_status(g.status, ZETA_ERR_BOUNDS);
    __syncthreads();

    // --------------------------------------------------- own-chunk part ---
    const int rg = warp / KS, kg = warp % KS;                // row group, key split
    const int la = sm.perm[rg * 16 + g4], lb = sm.perm[rg * 16 + 8 + g4];
    const int ta = la >= 0 ? sm.qrow[la] : -1, tb = lb >= 0 ? sm.qrow[lb] : -1;
    const int lim_a = ta >= 0 ? seq.start + ta - cC : -1;    // last key of the chunk row a sees
    const int lim_b = tb >= 0 ? seq.start + tb - cC : -1;
    take_rows(ta, tb);
    const int wmin = __reduce_min_sync(kFull, min(lim_a, lim_b));
    const int wmax = __reduce_max_sync(kFull, max(lim_a, lim_b));
    clear();
    if (WK == kWSoftmax && kg == 0)                          // from the window's shift
        mab = make_float2(la >= 0 ? sm.mwin[la] : INFINITY, lb >= 0 ? sm.mwin[lb] : INFINITY);
    using KSteps = std::integral_constant<int, TK / 16 / KS>;   // this warp's steps per tile
    for (int kt = 0; kt < nkt; ++kt) {
        cp_async_wait<1>();
        __syncthreads();                                     // tile kt is here, kt - 1 used up
        load_tile(kt + 2);
        put_rows(kt + 3, kid);
        kid = ask_rows(kt + 4);
        const int key0 = kt * TK, bf = kt % 3, kb = kg * KSteps::value * 16;
        if (key0 + kb <= wmax) {                             // else every weight of this warp is 0
            if (!sm.bad && key0 + TK - 1 <= wmin) {
                steps(KSteps{}, sm.own.kt[bf], sm.own.v[bf], kb,
                      [](int, float2 x, float) { return x; });
            } else {
                const int *rows = sm.rows[kt & 3];
                steps(KSteps{}, sm.own.kt[bf], sm.own.v[bf], kb, [&](int kl, float2 x, float no) {
                    const bool there = rows[kl] >= 0;
                    return make_float2(there && key0 + kl <= lim_a ? x.x : no,
                                       there && key0 + kl <= lim_b ? x.y : no);
                });
            }
        }
    }
    __syncthreads();

    // --------------------------------------------------------- epilogue ---
    float sa = sab.x, sb = sab.y;
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        sa += __shfl_xor_sync(kFull, sa, o);
        sb += __shfl_xor_sync(kFull, sb, o);
    }
    if constexpr (KS > 1) {                                  // join the key splits in order
        constexpr int PW = DVP + 4;
        float *part = sm.join;                                      // [WM][KS - 1][16][PW]
        const int slot = rg * (KS - 1) - 1;                         // + split, from 1
        if (kg > 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (nt < 2 * nc) {
                    float *pa = part + ((slot + kg) * 16 + g4) * PW + nt * 8 + 2 * tig;
                    pa[0] = acc[nt][0];
                    pa[1] = acc[nt][1];
                    pa[8 * PW] = acc[nt][2];
                    pa[8 * PW + 1] = acc[nt][3];
                }
            if (tig == 0) {
                sm.lsum[warp][g4] = sa;
                sm.lsum[warp][g4 + 8] = sb;
                sm.lmin[warp][g4] = mab.x;
                sm.lmin[warp][g4 + 8] = mab.y;
            }
        }
        __syncthreads();
        if (kg > 0) return;
        float2 mall = mab;
        if constexpr (WK == kWSoftmax) {
#pragma unroll
            for (int w = 1; w < KS; ++w)
                mall = make_float2(fminf(mall.x, sm.lmin[warp + w][g4]), fminf(mall.y, sm.lmin[warp + w][g4 + 8]));
        }
        auto factor = [&](float mo, float mn) {
            if (WK != kWSoftmax || mo == mn) return 1.f;
            return mo == INFINITY ? 0.f : __expf((mn - mo) * inv_g2);
        };
        const float f0a = factor(mab.x, mall.x), f0b = factor(mab.y, mall.y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            acc[nt][0] *= f0a;
            acc[nt][1] *= f0a;
            acc[nt][2] *= f0b;
            acc[nt][3] *= f0b;
        }
        sa *= f0a;
        sb *= f0b;
#pragma unroll
        for (int w = 1; w < KS; ++w) {
            const float fa = factor(sm.lmin[warp + w][g4], mall.x);
            const float fb = factor(sm.lmin[warp + w][g4 + 8], mall.y);
            sa = __fmaf_rn(fa, sm.lsum[warp + w][g4], sa);
            sb = __fmaf_rn(fb, sm.lsum[warp + w][g4 + 8], sb);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (nt < 2 * nc) {
                    const float *pa = part + ((slot + w) * 16 + g4) * PW + nt * 8 + 2 * tig;
                    acc[nt][0] = __fmaf_rn(fa, pa[0], acc[nt][0]);
                    acc[nt][1] = __fmaf_rn(fa, pa[1], acc[nt][1]);
                    acc[nt][2] = __fmaf_rn(fb, pa[8 * PW], acc[nt][2]);
                    acc[nt][3] = __fmaf_rn(fb, pa[8 * PW + 1], acc[nt][3]);
                }
        }
        mab = mall;
    }
    float fa = 1.f, fb = 1.f;                                // window sums onto the final shift
    if constexpr (WK == kWSoftmax) {
        const float ma = la >= 0 ? sm.mwin[la] : INFINITY, mb = lb >= 0 ? sm.mwin[lb] : INFINITY;
        fa = ma == INFINITY ? 0.f : shift_scale(mab.x, ma, inv_g2);
        fb = mb == INFINITY ? 0.f : shift_scale(mab.y, mb, inv_g2);
    }
    const float tta = la >= 0 ? __fmaf_rn(sm.swin[la], fa, sa) : 1.f;
    const float ttb = lb >= 0 ? __fmaf_rn(sm.swin[lb], fb, sb) : 1.f;
    const float ia = __frcp_rn(tta), ib = __frcp_rn(ttb);
    float za = 0.f, zb = 0.f;                                // NaN once a result is not finite
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int col = nt * 8 + 2 * tig;
        if (nt * 8 < g.dV) {
            if (la >= 0) {
                const float2 w = *reinterpret_cast<const float2 *>(&sm.win[la][col]);
                const float x = __fmaf_rn(w.x, fa, acc[nt][0]) * ia, y = __fmaf_rn(w.y, fa, acc[nt][1]) * ia;
                za = __fmaf_rn(x, 0.f, __fmaf_rn(y, 0.f, za));
                *reinterpret_cast<__nv_bfloat162 *>(g.out + (row0 + ta) * g.dV + col) = __floats2bfloat162_rn(x, y);
            }
            if (lb >= 0) {
                const float2 w = *reinterpret_cast<const float2 *>(&sm.win[lb][col]);
                const float x = __fmaf_rn(w.x, fb, acc[nt][2]) * ib, y = __fmaf_rn(w.y, fb, acc[nt][3]) * ib;
                zb = __fmaf_rn(x, 0.f, __fmaf_rn(y, 0.f, zb));
                *reinterpret_cast<__nv_bfloat162 *>(g.out + (row0 + tb) * g.dV + col) = __floats2bfloat162_rn(x, y);
            }
        }
    }
    if (tig == 0) {
        if (la >= 0) g.rowsum[row0 + ta] = tta;
        if (lb >= 0) g.rowsum[row0 + tb] = ttb;
    }
    unsigned again[2] = {__ballot_sync(kFull, za != za), __ballot_sync(kFull, zb != zb)};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        while (again[e]) {
            const int r = (__ffs(again[e]) - 1) >> 2;
            again[e] &= ~(15u << (4 * r));
            const int l = sm.perm[rg * 16 + 8 * e + r];
            __syncwarp();                                    // the fast result is written first
            slow_row<DVP, DK, WK>(g, row0, sm.qrow[l], h, seq.start, cC, cC > 0 ? sm.wst[l] : 0, ptab,
                                  otab, plane, inv_g2);
        }
    }
}

template <int DVP, int DK, int WK, int WM, int NW>
cudaError_t run_tile(const Prob &p, TileArgs g, cudaStream_t st) {
    static PerDeviceOnce once;
    constexpr size_t smem = sizeof(TileSmem<DVP, WM, NW>);
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(cache_tile_kernel<DVP, DK, WK, WM, NW>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    // Row tiles of a sequence: its rows are cut once, at a chunk's end.
    const unsigned tiles = (unsigned)((g.c.n + 16 * WM - 1) / (16 * WM) + (g.c.n > 1 ? 1 : 0));
    cache_tile_kernel<DVP, DK, WK, WM, NW><<<dim3(tiles, (unsigned)p.S), NW * 32, smem, st>>>(g);
    return cudaGetLastError();
}

template <int DVP, int WM, int NW>
cudaError_t dispatch_tile(const Prob &p, const TileArgs &g, cudaStream_t st) {
#define ZETA_TILE(D)                                                                \
    (p.wk == kWSoftmax     ? run_tile<DVP, D, kWSoftmax, WM, NW>(p, g, st)              \
     : p.wk == kWInvEuclid ? run_tile<DVP, D, kWInvEuclid, WM, NW>(p, g, st)            \
                           : run_tile<DVP, D, kWCauchy, WM, NW>(p, g, st))
    return p.dK == 3 ? ZETA_TILE(3) : ZETA_TILE(4);
#undef ZETA_TILE
}

}  // namespace
}  // namespace zeta
