// cache_tile.cuh -- attention of many new tokens per sequence over the paged
// cache: bf16 values, d_V a multiple of 8 up to 128, d_K <= 4.
//
// Same definition as the row kernel (cache_attend.cu).  A block of NW warps takes
// 16 WM query rows of one head and one chunk.
//  * Rank: the first code of every block of 2^fsh prefix entries is staged in
//    shared memory; a warp finds a row's block there and its rank among the
//    block's entries with one coalesced read of up to 64.
//  * Own chunk: key tiles staged by cp.async through the page table into
//    swizzled shared memory; weights are built straight in mma A fragments, two keys of
//    a row to an instruction (the coordinates are staged apart, so that a pair of keys
//    is one operand).  A weight enters as a bf16 half and the bf16 of what that leaves,
//    two products into one float32 accumulator: within 2^-16 of the weight, so that a
//    row's result does not tell which kernel the size of its batch chose.  Row sums come
//    from the float32 weights.  NW / WM warps split each tile's keys and join at the end.
//  * Window: a warp takes two rows at a time; their entries are looked up and weighed
//    a lane each, the four dependent lookups of the next two rows run between the
//    batches of value rows of these two, which are streamed and summed on the FMA
//    pipes.  (Dealing the rows of a piece to the warps by their codes, so that their
//    windows overlap, and walking them as masked mma tiles was built and taken out
//    again: 210 us against 204 here for 16 pieces of up to 1024 rows; it gained for
//    4 whole pieces alone, 64 against 82 us.)
//  * A masked weight of zero times a value that is not finite would be NaN: a row
//    whose result is not finite is taken again, key by key, without the others.
//
// 16 pieces of up to 1024 rows (9,704 together), 8 heads, 19 K tokens before each on
// average, C 1024, k 64, d_V 64: 213 us, where the bytes take 66 at the HBM rate and the
// products 5.  The windows are 64 scattered value rows a row: with their keys and the
// own chunks 1.04 GB come out of L2 (289 MB of it from DRAM), 4.9 TB/s; 46 % of the issue
// slots are used, with two blocks of 8 warps an SM (128 registers, 48 to 128 bytes of
// spills up to 64 wide; 168 and none above).  What bounds it is waiting: for the gathers,
// and then for the own chunk, which starts when every window of the block is done.  It is
// no ceiling of the machine: the training forward spends 1.6 to 1.8 ns a row on the same
// work, this 2.7.  One piece of 1024 rows: 40 us, a block's latency.  d_K of 1 and 2 run the
// form for four coordinates, the missing ones zero.
#pragma once

#include "cache.cuh"
#include "mma.cuh"

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

// wm: 1, 2 or (up to 64 wide) 4, for 16 wm rows a block.
cudaError_t launch_cache_tile64(const Prob &p, const TileArgs &g, int wm, cudaStream_t st);
cudaError_t launch_cache_tile128(const Prob &p, const TileArgs &g, int wm, cudaStream_t st);

namespace {

constexpr int kFences = 1024;

template <int DVP, int WM, int NW>
struct TileSmem {
    static constexpr int TQ = 16 * WM;
    static constexpr int TK = DVP == 64 && NW / WM >= 4 ? 128 : 64;
    struct Own {
        __nv_bfloat16 v[3][TK * DVP];  // 16-byte chunk c of row r at c ^ (r & 7)
        float k[3][4][TK];             // coordinates apart
    };
    struct Gather {                    // a warp's two rows
        float w[NW][2][64];
        int row[NW][2][64];
    };
    union {
        Own own;
        float join[WM * (NW / WM - 1) * 16 * (DVP + 4)];
    };
    uint64_t fence[kFences];
    Gather gather;
    float win[TQ][DVP + 4];            // window sums
    int rows[4][TK];                   // pool rows of the tile's keys, -1: none
    float swin[TQ], mwin[TQ];
    float lsum[NW][16], lmin[NW][16];  // the key splits' row sums and shifts
    int wst[TQ];                       // window start of a row
};

// The 4-byte form of cp_async16, for single coordinates.
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int src_bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src),
                 "r"(src_bytes));
}

// Weights of two keys (the reciprocals by the approximate instructions, 1 ulp).
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int WK>
__device__ __forceinline__ float2 weight_pair(float2 d2, float m, float2 ig2) {
    if constexpr (WK == kWCauchy) {
        const float2 t = fma2(d2, ig2, dup2(1.0f));
        return make_float2(rcp_approx(t.x), rcp_approx(t.y));
    } else {
        return weight_fast2<WK>(d2, dup2(m), ig2);
    }
}

// What two weights' bf16 halves (pack_bf16) leave of them, as bf16 again.
__device__ __forceinline__ uint32_t pack_rest(float2 w, uint32_t half) {
    const float2 r = sub2(w, make_float2(__uint_as_float(half << 16), __uint_as_float(half & 0xffff0000u)));
    return pack_bf16(r.x, r.y);
}

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
__global__ void __launch_bounds__(NW * 32, DVP == 64 ? 2 : 3)
cache_tile_kernel(const __grid_constant__ TileArgs g) {
    using Sm = TileSmem<DVP, WM, NW>;
    constexpr int TQ = Sm::TQ, TK = Sm::TK, KS = NW / WM;    // KS warps share a row group's keys
    constexpr int kTileThreads = NW * 32;
    constexpr int QW = TQ / NW;                              // window rows per warp
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
    const int f0 = p0 + x * TQ, nq = min(TQ, np - x * TQ);   // the call's rows f0 .. f0 + nq - 1
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

    // Own-chunk tiles: keys cC .. last row's position (they all exist).
    const int kend = seq.start + f0 + nq - cC;               // keys of the chunk that matter
    const int nkt = (kend + TK - 1) / TK;
    auto ask_rows = [&](int kt) {                            // page of the thread's key of tile kt
        return tid < TK && kt * TK + tid < kend ? page_id(ptab, cC + kt * TK + tid, g.c.psh) : -1;
    };
    bool lost_key = false;                                   // this thread met a key without a page
    auto put_rows = [&](int kt, int id) {                    // its pool row, for every thread to see
        if (tid < TK && kt < nkt) {
            const int row = pool_row(id, cC + kt * TK + tid);
            if (row < 0 && kt * TK + tid < kend) {
                set_status(g.status, ZETA_ERR_BOUNDS);
                lost_key = true;
            }
            sm.rows[kt & 3][tid] = row;
        }
        __syncwarp();                                        // one branch again before the products
    };
    const int ppr = g.dV >> 3;                               // 16-byte pieces per value row
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
                const int d = id / TK, row = id % TK;
                const int pr = rows[row];
                const bool ok = pr >= 0 && d < g.dK;
                cp_async4(smem_u32(&sm.own.k[bf][d][row]),
                          g.k_pages + (ok ? (int64_t)pr * g.dK + d : 0), ok ? 4 : 0);
            }
        }
        cp_async_commit();
    };
    int kid = ask_rows(3);
    {
        const int i0 = ask_rows(0), i1 = ask_rows(1), i2 = ask_rows(2);
        put_rows(0, i0);
        put_rows(1, i1);
        put_rows(2, i2);
    }
    __syncthreads();
    load_tile(0);
    load_tile(1);

    // ------------------------------------------------------ window part ---
    const int g4 = lane >> 2, s4 = lane & 3;
    const int wl0 = warp * QW, nqw = chunk > 0 ? max(0, min(QW, nq - wl0)) : 0;
    int wst = 0;                                             // lane r < nqw: start of row wl0 + r
    if (chunk > 0) {
        uint64_t *fence = sm.fence;
        int fsh = 5;
        while ((cC >> fsh) >= kFences) ++fsh;
        const int nf = (cC + (1 << fsh) - 1) >> fsh;
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
            z = code_at(f0 + wl0 + lane);
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
    }
    // Weights in A fragments and products of KN steps of 16 keys: lane (g4, s4) has
    // rows g4 (a) and g4 + 8 (b) of its group and the key pairs 2 s4, +1 and +8, +9 of
    // a step; mask(a or b, key, pair, none) puts `none` where the row does not take a
    // key.  Ks: [4][stride] coordinates.
    const int tig = s4;
    const float2 ig2 = dup2(inv_g2);
    const int nc = (g.dV + 15) >> 4;                         // 16-column pairs in use
    float2 qa[DK], qb[DK];                                   // each coordinate twice
    float2 sa2, sb2;                                         // row sums, over the first and second keys of the pairs
    float ma, mb;                                            // softmax shifts
    float acc[NT][4];
    auto clear = [&] {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
        sa2 = sb2 = make_float2(0.f, 0.f);
        ma = mb = INFINITY;
    };
    auto take_rows = [&](int ta, int tb) {                   // the call's rows, -1: none
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 a = ta >= 0 ? ld_key(qs + (int64_t)ta * g.dK, g.dK) : z;
        const float4 c = tb >= 0 ? ld_key(qs + (int64_t)tb * g.dK, g.dK) : z;
        const float av[4] = {a.x, a.y, a.z, a.w}, cv[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int d = 0; d < DK; ++d) {
            qa[d] = dup2(av[d]);
            qb[d] = dup2(cv[d]);
        }
    };
    auto dist_pair = [&](const float *Ks, int stride, int kl, float2 &da, float2 &db) {
        da = db = make_float2(0.f, 0.f);
#pragma unroll
        for (int d = 0; d < DK; ++d) {
            const float2 kc = *reinterpret_cast<const float2 *>(Ks + d * stride + kl);
            const float2 ea = sub2(qa[d], kc), eb = sub2(qb[d], kc);
            da = fma2(ea, ea, da);
            db = fma2(eb, eb, db);
        }
    };
    auto steps = [&](auto kn, const float *Ks, int stride, const __nv_bfloat16 *Vs, int kb0, auto mask) {
        constexpr int KN = decltype(kn)::value;
        if constexpr (WK == kWSoftmax) {                     // move the shifts to the least d2
            float la = INFINITY, lb = INFINITY;
#pragma unroll
            for (int e = 0; e < 2 * KN; ++e) {
                const int kl = kb0 + e * 8 + 2 * tig;
                float2 da, db;
                dist_pair(Ks, stride, kl, da, db);
                da = mask(std::false_type{}, kl, da, INFINITY);
                db = mask(std::true_type{}, kl, db, INFINITY);
                la = fminf(la, fminf(da.x, da.y));
                lb = fminf(lb, fminf(db.x, db.y));
            }
#pragma unroll
            for (int o = 1; o <= 2; o <<= 1) {
                la = fminf(la, __shfl_xor_sync(kFull, la, o));
                lb = fminf(lb, __shfl_xor_sync(kFull, lb, o));
            }
            const float na = fminf(ma, la), nb = fminf(mb, lb);
            const float fa = na == ma ? 1.f : ma == INFINITY ? 0.f : __expf((na - ma) * inv_g2);
            const float fb = nb == mb ? 1.f : mb == INFINITY ? 0.f : __expf((nb - mb) * inv_g2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                acc[nt][0] *= fa;
                acc[nt][1] *= fa;
                acc[nt][2] *= fb;
                acc[nt][3] *= fb;
            }
            sa2 = mul2(sa2, dup2(fa));
            sb2 = mul2(sb2, dup2(fb));
            ma = na;
            mb = nb;
        }
        // Finite even where no key is taken yet.
        const float xa = ma == INFINITY ? 0.f : ma, xb = mb == INFINITY ? 0.f : mb;
        const uint32_t vbase = smem_u32(Vs);
#pragma unroll
        for (int ks = 0; ks < KN; ++ks) {
            const int kb = kb0 + ks * 16;
            uint32_t a[4], rest[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int kl = kb + e * 8 + 2 * tig;
                float2 da, db;
                dist_pair(Ks, stride, kl, da, db);
                const float2 wa = mask(std::false_type{}, kl, weight_pair<WK>(da, xa, ig2), 0.f);
                const float2 wb = mask(std::true_type{}, kl, weight_pair<WK>(db, xb, ig2), 0.f);
                sa2 = add2(sa2, wa);
                sb2 = add2(sb2, wb);
                a[2 * e] = pack_bf16(wa.x, wa.y);
                a[2 * e + 1] = pack_bf16(wb.x, wb.y);
                rest[2 * e] = pack_rest(wa, a[2 * e]);
                rest[2 * e + 1] = pack_rest(wb, a[2 * e + 1]);
            }
            const int m = lane >> 3, key = kb + (m & 1) * 8 + (lane & 7);
#pragma unroll
            for (int n2 = 0; n2 < NT / 2; ++n2) {
                if (n2 < nc) {
                    uint32_t b[4];
                    ldsm_x4_trans(b, vbase + (uint32_t)(key * DVP + (((n2 * 2 + (m >> 1)) ^ (key & 7)) * 8)) * 2u);
                    mma16816(acc[2 * n2], a, b[0], b[1]);
                    mma16816(acc[2 * n2 + 1], a, b[2], b[3]);
                    mma16816(acc[2 * n2], rest, b[0], b[1]);
                    mma16816(acc[2 * n2 + 1], rest, b[2], b[3]);
                }
            }
        }
    };

    if (chunk > 0) {
        typename Sm::Gather &ga = sm.gather;
        constexpr int LPR = DVP / 8, RPI = 32 / LPR;         // lanes per value row, rows per load
        const int grp = lane / LPR, sub = lane % LPR;
        bool lost = false;
        // Items of two rows and up to 64 of their entries.  Entries are looked up in four
        // dependent steps (page of the entry, token, page of the token, key); those of the
        // next item run between the four batches of value rows of this one.
        const int np64 = (g.k + 63) >> 6, items = (nqw + 1) / 2 * np64;
        int it = -1, r0 = -2, t0 = 0;                        // the item being looked up
        int t[2] = {0, 0}, st[2], j[4], row[4];
        float q[2][DK], x[4][DK];
        auto slot = [&](int v) { return t0 + (v & 1) * 32 + lane; };
        auto there = [&](int v) { return it < items && r0 + (v >> 1) < nqw && slot(v) < g.k; };
        auto look = [&](int step) {
            if (step == 0) {
                ++it;
                t0 += 64;
                if (t0 >= g.k || r0 < 0) {
                    t0 = 0;
                    r0 += 2;
                }
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    t[u] = min(f0 + wl0 + r0 + u, f0 + nq - 1);
                    st[u] = __shfl_sync(kFull, wst, (r0 + u) & 31);
                    const float4 q4 = ld_key(qs + (int64_t)t[u] * g.dK, g.dK);
                    const float qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
                    for (int d = 0; d < DK; ++d) q[u][d] = qq[d];
                }
#pragma unroll
                for (int v = 0; v < 4; ++v) j[v] = page_id(otab, min(st[v >> 1] + slot(v), cC - 1), g.c.psh);
            } else if (step == 1) {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const int orow = order_row(j[v], st[v >> 1] + slot(v));
                    j[v] = ldi_if(g.order_idx + plane + orow, there(v) && orow >= 0);
                }
            } else if (step == 2) {
#pragma unroll
                for (int v = 0; v < 4; ++v) row[v] = page_id(ptab, (unsigned)j[v] < (unsigned)cC ? j[v] : 0, g.c.psh);
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    row[v] = (unsigned)j[v] < (unsigned)cC ? pool_row(row[v], j[v]) : -1;
                    const float *kp = g.k_pages + (int64_t)max(row[v], 0) * g.dK;
#pragma unroll
                    for (int d = 0; d < DK; ++d) x[v][d] = d < g.dK ? __ldg(kp + d) : 0.f;
                }
            }
        };
        float2 o[2][4];
        float sw[2], mr[2];
        if (items > 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) look(e);
        }
        for (int i = 0; i < items; ++i) {
            const int row0_ = r0, ent0 = t0;                 // this item's rows and entries
            if (ent0 == 0) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    sw[u] = 0.f;
                    mr[u] = INFINITY;
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[u][e] = make_float2(0.f, 0.f);
                }
            }
            float d2[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                d2[v] = 0.f;
#pragma unroll
                for (int d = 0; d < DK; ++d) {
                    const float e = q[v >> 1][d] - x[v][d];
                    d2[v] = __fmaf_rn(e, e, d2[v]);
                }
                if (row[v] < 0) d2[v] = INFINITY;
                lost |= there(v) && row[v] < 0;
                if (g.idx && there(v))
                    g.idx[(row0 + t[v >> 1]) * g.k + slot(v)] = (unsigned)j[v] < (unsigned)cC ? j[v] : -1;
            }
            if constexpr (WK == kWSoftmax) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float least = fminf(d2[2 * u], d2[2 * u + 1]);
#pragma unroll
                    for (int e = 16; e > 0; e >>= 1) least = fminf(least, __shfl_xor_sync(kFull, least, e));
                    if (least < mr[u]) {
                        const float f = mr[u] == INFINITY ? 0.f : __expf((least - mr[u]) * inv_g2);
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[u][e] = mul2(o[u][e], dup2(f));
                        sw[u] *= f;
                        mr[u] = least;
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float w = row[v] >= 0 ? weight_fast<WK>(d2[v], mr[v >> 1], inv_g2) : 0.f;
                sw[v >> 1] += w;
                ga.w[warp][v >> 1][(v & 1) * 32 + lane] = w;
                ga.row[warp][v >> 1][(v & 1) * 32 + lane] = row[v];
            }
            __syncwarp();
            // Value rows in batches of 4 RPI entries of both rows, two batches in flight.
            constexpr int EB = 4 * RPI, NB = 64 / EB;
            uint4 bufs[2][2][4];
            auto load = [&](uint4 (&buf)[2][4], int e0) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int pr = ga.row[warp][u][e0 + grp + v * RPI];
                        buf[u][v] = ld16_if(g.v_pages + (int64_t)max(pr, 0) * g.dV + sub * 8, pr >= 0 && sub < ppr);
                    }
            };
            auto add = [&](const uint4 (&buf)[2][4], int e0) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const float2 w = dup2(ga.w[warp][u][e0 + grp + v * RPI]);
                        const uint32_t b4[4] = {buf[u][v].x, buf[u][v].y, buf[u][v].z, buf[u][v].w};
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            o[u][c] = fma2(w, make_float2(__uint_as_float(b4[c] << 16),
                                                          __uint_as_float(b4[c] & 0xffff0000u)), o[u][c]);
                    }
            };
            load(bufs[0], 0);
            load(bufs[1], EB);
            const bool more = i + 1 < items;
#pragma unroll
            for (int e = 0; e < NB; ++e) {
                if (more && e * 4 % NB == 0) look(e * 4 / NB);
                add(bufs[e & 1], e * EB);
                if (e + 2 < NB) load(bufs[e & 1], (e + 2) * EB);
            }
            __syncwarp();                                    // the weights have been read
            if (ent0 + 64 < g.k) continue;                   // more entries of these rows
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float ssum = sw[u];
#pragma unroll
                for (int e = 16; e > 0; e >>= 1) ssum += __shfl_xor_sync(kFull, ssum, e);
#pragma unroll
                for (int e = 16; e >= LPR; e >>= 1)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        o[u][c].x += __shfl_xor_sync(kFull, o[u][c].x, e);
                        o[u][c].y += __shfl_xor_sync(kFull, o[u][c].y, e);
                    }
                const int l = wl0 + row0_ + u;
                if (lane < LPR) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) *reinterpret_cast<float2 *>(&sm.win[l][sub * 8 + 2 * c]) = o[u][c];
                }
                if (lane == 0) {
                    sm.swin[l] = ssum;
                    sm.mwin[l] = mr[u];
                }
            }
        }
        if (lost) set_status(g.status, ZETA_ERR_BOUNDS);
    } else {                                                 // nothing selected
        for (int l = wl0; l < wl0 + QW; ++l) {
            for (int e = lane; e < DVP; e += 32) sm.win[l][e] = 0.f;
            if (lane == 0) {
                sm.swin[l] = 0.f;
                sm.mwin[l] = INFINITY;
            }
            if (g.idx && l < nq)
                for (int e = lane; e < g.k; e += 32) g.idx[(row0 + f0 + l) * g.k + e] = -1;
        }
    }
    __syncthreads();

    // --------------------------------------------------- own-chunk part ---
    const int rg = warp / KS, kg = warp % KS;                // row group, key split
    const int la = rg * 16 + g4 < nq ? rg * 16 + g4 : -1;    // the thread's two rows, -1: none
    const int lb = rg * 16 + 8 + g4 < nq ? rg * 16 + 8 + g4 : -1;
    const int ta = la >= 0 ? f0 + la : -1, tb = lb >= 0 ? f0 + lb : -1;
    const int lim_a = ta >= 0 ? seq.start + ta - cC : -1;    // last key of the chunk row a sees
    const int lim_b = tb >= 0 ? seq.start + tb - cC : -1;
    take_rows(ta, tb);
    const int wmin = __reduce_min_sync(kFull, min(lim_a, lim_b));
    const int wmax = __reduce_max_sync(kFull, max(lim_a, lim_b));
    clear();
    if (WK == kWSoftmax && kg == 0) {                        // from the window's shift
        ma = la >= 0 ? sm.mwin[la] : INFINITY;
        mb = lb >= 0 ? sm.mwin[lb] : INFINITY;
    }
    using KSteps = std::integral_constant<int, TK / 16 / KS>;   // this warp's steps per tile
    for (int kt = 0; kt < nkt; ++kt) {
        cp_async_wait<1>();
        // Tile kt is here, kt - 1 used up.  The barrier tells every thread alike whether a
        // key up to tile kt + 2 has no page: the branch below holds warp-wide instructions.
        const bool lost = __syncthreads_or(lost_key);
        load_tile(kt + 2);
        put_rows(kt + 3, kid);
        kid = ask_rows(kt + 4);
        const int key0 = kt * TK, bf = kt % 3, kb = kg * KSteps::value * 16;
        if (key0 + kb <= wmax) {                             // else every weight of this warp is 0
            if (!lost && key0 + TK - 1 <= wmin) {
                steps(KSteps{}, &sm.own.k[bf][0][0], TK, sm.own.v[bf], kb,
                      [](auto, int, float2 x, float) { return x; });
            } else {
                const int *rows = sm.rows[kt & 3];
                steps(KSteps{}, &sm.own.k[bf][0][0], TK, sm.own.v[bf], kb,
                      [&](auto second_row, int kl, float2 x, float no) {
                          const int2 r = *reinterpret_cast<const int2 *>(rows + kl);
                          const int lim = decltype(second_row)::value ? lim_b : lim_a;
                          return make_float2(r.x >= 0 && key0 + kl <= lim ? x.x : no,
                                             r.y >= 0 && key0 + kl + 1 <= lim ? x.y : no);
                      });
            }
        }
    }
    __syncthreads();

    // --------------------------------------------------------- epilogue ---
    float2 mab = make_float2(ma, mb);
    float sa = sa2.x + sa2.y, sb = sb2.x + sb2.y;
#pragma unroll
    for (int o = 1; o <= 2; o <<= 1) {
        sa += __shfl_xor_sync(kFull, sa, o);
        sb += __shfl_xor_sync(kFull, sb, o);
    }
    static_assert(KS > 1);                                   // join the key splits in order
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
    float fa = 1.f, fb = 1.f;                                // window sums onto the final shift
    if constexpr (WK == kWSoftmax) {
        const float wa = la >= 0 ? sm.mwin[la] : INFINITY, wb = lb >= 0 ? sm.mwin[lb] : INFINITY;
        fa = wa == INFINITY ? 0.f : shift_scale(mab.x, wa, inv_g2);
        fb = wb == INFINITY ? 0.f : shift_scale(mab.y, wb, inv_g2);
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
            const int l = rg * 16 + 8 * e + r;
            __syncwarp();                                    // the fast result is written first
            slow_row<DVP, DK, WK>(g, row0, f0 + l, h, seq.start, cC, cC > 0 ? sm.wst[l] : 0, ptab,
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
