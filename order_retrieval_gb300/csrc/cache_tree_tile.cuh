// cache_tree_tile.cuh -- attention of trees of drafted tokens: bf16 values with d_V a
// multiple of 8, float32 with a multiple of 4, up to 128 wide, d_K <= 4.
//
// Same definition as the row kernel (cache_tree.cu).  A block takes 8 or 16 nodes of one
// sequence and head, or a cluster of up to 8 blocks does where there are few: every block of
// it has some of the nodes' windows and some of the keys that all of them share, and the sums
// are joined through distributed shared memory.  A warp takes its part of the shared keys,
// then its windows one by one; between set-up and join none waits for another but once, for
// the lines.
//  * Lines: a bit per node above, found by climbing in shared memory.  A run of nodes
//    that hang below one another by number (a chain) is one step of the climb.
//  * Window: the first code of every block of 2^fsh prefix entries lies in shared memory; a
//    warp counts there and among the block's entries, and asks with those for the entries
//    that the window may hold.  It looks up and weighs the entries a lane each, then their
//    value rows stream through registers.
//  * Shared keys: the sequence's tokens of the chunk, then the nodes, 16 (float32: 8) a step
//    and warp, straight from global memory.
//  * bf16 products run on mma.sync without shared memory: of 16 keys lane (g, t) loads 32
//    bytes (values 16t ..) of the rows of keys g and g + 8, a whole row to four lanes, so that
//    a load touches 8 lines of L1; movmatrix turns the 8 x 8 blocks into A operands (values
//    times keys).  B (keys times columns) has 8 nodes' weights, a window's in columns 0 to 2.
//    A weight enters as three bf16 parts, each the nearest to what those before it leave: 3 x 8
//    bits hold all 24 of it (below 2^-110, where the last ones are no longer bf16 numbers, all
//    but 2^-133), so that sums are those of float32 weights.  (Two parts, within 2^-16,
//    let one output in a thousand round to the other neighbour; the third costs 2.9 of the 55 us
//    below.)
//  * A weight of zero times a value that is not finite is NaN: a node whose result is not
//    finite is taken again, key by key, without the others.
//
// 59 sequences with trees of 25 nodes on average, 8 heads, 10 K tokens before each and 508 of
// them in its chunk of 1024, windows of 48, d_V 64: 55 us for 120 MB, 2.2 TB/s (32 % of the
// measured HBM rate; DRAM reads 156 MB: every search reads the fences' and its block's sectors).
// What bounds it is the warps' own way: 21.3 M instructions (half of them in windows: about 800
// for a search, its lookups, weights and sums; about 160 for 16 shared keys and 16 nodes) at 31 % of the
// issue slots, with 16 warps an SM that wait for DRAM in turn and for results of their own
// instructions; a fifth of the time SMs run empty at the end.  Other d_K than 3 and chunks that begin
// off a multiple of 16 (C = 1000: every other one) have no whole steps: the same trees take 63 to
// 66 us with d_K 1, 2 or 4, 58 with C 1000.  Softmax 64 us, d_V 128 81, float32 77.
// Tried on the way, with weights in two parts (52 us at the end of it, 57 on texts of over 2 K tokens
// where those that lie in L2 took 43): value rows by cp.async through rings in shared memory, half the
// warps on windows and half on shared keys 86; operands put together by byte permutes, a load
// touching 32 rows' lines instead of 8, 59; windows of two nodes at once 66; three blocks an SM with
// 80 registers 64 to 72 (spills); 8 nodes and 4 warps a block 60; two steps of shared keys at
// once 59; their values asked into L2 ahead, no difference; all slices' first nodes before their
// others 54 (what they share leaves L2).
#pragma once

#include <cooperative_groups.h>

#include "cache_tile.cuh"
#include "cache_tree.cuh"

namespace zeta {

// ng: groups of 8 nodes to a block (1, or 2 up to 64 wide); cs: blocks to them (1, 2, 4 or 8).
cudaError_t launch_tree_tile_bf16(const Prob &p, const TreeArgs &g, int ng, int cs, cudaStream_t st);
cudaError_t launch_tree_tile_f32(const Prob &p, const TreeArgs &g, int ng, int cs, cudaStream_t st);

namespace {

namespace cg = cooperative_groups;

constexpr int kTreeFences = 256;
constexpr int kTreeTable = 1024;                     // pages whose numbers lie in shared memory

template <typename V, int DVP, int NG>
struct TreeSmem {
    static constexpr bool MMA = sizeof(V) == 2;
    // NG groups of 8 nodes a block; warps, blocks an SM (128 registers a thread), a window's steps
    // under way (64 sequences, 16 nodes a block: 2, 3, 4 of them 54, 52, 56 us; lines of 200, 128
    // wide, 8 nodes: 2, 3 of them 48.6, 51.7; weights in two parts).
    static constexpr int ROWS = 8 * NG, NW = 4 * NG, PER_SM = 4 / NG, NB = NG + 1;
    static constexpr int KS = MMA ? 16 : 8, KL = KS / 4, KP = KL / 2;    // shared keys a step, a lane; pairs
    static constexpr int NV = DVP / 16;              // 16-byte pieces of them a lane holds (float32: of four keys)
    float part[NW][ROWS][DVP + 4];                   // sums over shared keys, warp by warp
    struct {                                         // of a warp's window
        int row[64];
        union {
            int cand[128];                           // entries that it may hold
            float w[64];                             // float32: weights
            uint16_t bits[3][64];                    // bf16: weights' parts
        };
        float x[64 * 4];                             // coordinates
    } gather[NW];
    uint64_t fence[kTreeFences], z[ROWS];            // codes of the fences, of the nodes
    int ptab[kTreeTable];
    float w[MMA ? 1 : NW][8][20];            // float32, shared keys: weights [key][node]
    union {
        int parent[kMaxDraft];
        float win[ROWS][DVP + 4];               // window sums
    };
    uint32_t run[kMaxDraft / 32];                    // bit u: parent[u] == u - 1
    uint32_t above[ROWS][kMaxDraft / 32];       // nodes of a line
    float q[ROWS][4];
    int depth[ROWS], wst[ROWS];
    float swin[ROWS], mwin[ROWS];
    float psum[NW][ROWS], pmin[NW][ROWS];
    float factor[(NW > 8 ? NW : 8) + 1][ROWS], least[ROWS];   // softmax: of the parts (warps, or up to 8
                                                     // blocks) and the window; the shift
    float total[ROWS];
    bool again[ROWS];                           // not finite
};

__device__ __forceinline__ uint4 ld16(const void *p) {
    uint4 a;
    asm volatile("ld.global.nc.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w)
                 : "l"(p));
    return a;
}
// 32 bytes: one load where P is 32-byte aligned (WIDE), else two of 16 at p and q.
template <bool WIDE>
__device__ __forceinline__ void ld32(uint32_t (&x)[8], const char *p, const char *q) {
    if constexpr (WIDE) {
        asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                     : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
                     : "l"(p));
    } else {
        const uint4 a = ld16(p), b = ld16(q);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
}

// The bf16 next to each of two numbers, packed; what that leaves of them stays (exact).
__device__ __forceinline__ uint32_t take_part(float2 &left) {
    const uint32_t part = pack_bf16(left.x, left.y);
    left = sub2(left, make_float2(__uint_as_float(part << 16), __uint_as_float(part & 0xffff0000u)));
    return part;
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

// A code of the order, 32 or 64 bits wide.
__device__ __forceinline__ uint64_t ld_code(const char *codes, uint32_t row, int code64) {
    const char *p = codes + ((uint64_t)row << (2 + code64));
    return (uint64_t)ld4_if(p + 4, code64) << 32 | __ldg(reinterpret_cast<const uint32_t *>(p));
}

template <typename V, int DVP, int NG, int DK, int WK, bool WIDE>
__global__ void __launch_bounds__(TreeSmem<V, DVP, NG>::NW * 32, TreeSmem<V, DVP, NG>::PER_SM)
tree_tile_kernel(const __grid_constant__ TreeArgs g, int cs) {
    using Sm = TreeSmem<V, DVP, NG>;
    constexpr int NW = Sm::NW, NT = 32 * NW, ROWS = Sm::ROWS;
    constexpr int PPR = DVP * (int)sizeof(V) / 16;           // 16-byte pieces of a padded row
    extern __shared__ __align__(16) unsigned char raw[];
    Sm &sm = *reinterpret_cast<Sm *>(raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cr = cs == 1 ? 0 : (int)(blockIdx.x % (unsigned)cs);   // block in the cluster
    const int f0 = (int)(blockIdx.x / (unsigned)cs) * ROWS;     // first node
    const int s = blockIdx.y, b = s / g.H, h = s - b * g.H;
    const int64_t node0 = (int64_t)s * g.c.n;                // the slice's node 0
    const int32_t *ptab = g.c.ptab + (int64_t)b * g.c.tlen, *otab = g.c.otab + (int64_t)b * g.c.tlen;
    // What does not depend on the lengths is asked for with them.
    const int ahead = min(f0 + ROWS, g.c.n), pages_near = min(g.c.tlen, kTreeTable);
    const int parent = tid < ahead ? __ldg(g.parent + (int64_t)b * g.c.n + tid) : 0;
    const float q_in = tid < ROWS * 4 && f0 + (tid >> 2) < ahead && (tid & 3) < g.dK
                           ? __ldg(g.q + (node0 + f0 + (tid >> 2)) * g.dK + (tid & 3)) : 0.f;
    for (int e = tid; e < pages_near; e += NT) sm.ptab[e] = __ldg(ptab + e);
    const Seq seq = drafts_of(g.c, b, g.N, g.status);
    if (f0 >= seq.count) return;                             // the whole cluster returns
    const int nn = min(f0 + ROWS, seq.count), nq = nn - f0;
    const int chunk = seq.start / g.C, cC = chunk * g.C, L = seq.start - cC;
    const float gm = __ldg(g.gamma + h);
    const float inv_g2 = __frcp_rn(gm * gm);
    const int psh = g.c.psh, pmask = g.c.pmask;
    const int ppr = g.dV * (int)sizeof(V) / 16, vrow = g.dV * (int)sizeof(V);
    const int krow = (DK == 3 ? 3 : g.dK) * 4;               // bytes of a row
    const int64_t plane = ((int64_t)g.c.opages * g.H << psh) * (chunk & 1);
    const char *codes = static_cast<const char *>(g.order_codes) + (plane << (2 + g.code64));
    const int32_t *entries = g.order_idx + plane;
    // Row of position t in the pools where its page's number is id, which must be in range.
    const int hp = g.H << psh, hb = h << psh;
    auto row_at = [&](int id, int t) { return id * hp + hb + (t & pmask); };
    // Page numbers: of the sequence's tokens from shared memory where they fit, of the
    // order's entries from there too where both go by one table.
    const bool near = ((seq.start + pmask) >> psh) <= pages_near;
    const int32_t *pt = near ? sm.ptab : ptab, *ot = near && otab == ptab ? sm.ptab : otab;

    bool lost = false;                                       // this thread met what is out of range

    // ------------------------------------------------------------ set-up ---
    if (tid < nn) sm.parent[tid] = parent;
    for (int u = NT + tid; u < nn; u += NT) sm.parent[u] = __ldg(g.parent + (int64_t)b * g.c.n + u);
    if (tid < ROWS * 4) sm.q[tid >> 2][tid & 3] = q_in;
    if (tid < ROWS) sm.again[tid] = false;
    for (int e = tid; e < ROWS * (kMaxDraft / 32); e += NT) (&sm.above[0][0])[e] = 0u;
    __syncthreads();
    const int fsh = max(5, 24 - __clz(cC | 1));              // one fence in 2^fsh entries: up to 256
    const int nf = (cC + (1 << fsh) - 1) >> fsh;
    constexpr int NF = kTreeFences / NT;                     // a thread's
    uint64_t fz[NF];
#pragma unroll
    for (int u = 0; u < NF; ++u) {
        const int f = u * NT + tid;
        fz[u] = ~0ull;
        if (f < nf) {
            const int e = f << fsh, id = ot[e >> psh];
            if ((unsigned)id < (unsigned)g.c.opages) fz[u] = ld_code(codes, row_at(id, e), g.code64);
            else lost = true;
        }
    }
    if (warp == NW - 1) {                                    // the lines and codes, by the warp with the fewest steps
        for (int w = 0; w * 32 < nn; ++w) {
            const uint32_t bits = run_bits(sm.parent, w, nn);
            if (lane == 0) sm.run[w] = bits;
        }
        __syncwarp();
        if (lane < ROWS) {
            int depth = -1;
            if (lane < nq) {
                depth = climb_bits(sm.parent, sm.run, f0 + lane, sm.above[lane]);
                lost |= depth < 0;
                if (seq.start + depth >= cC + g.C) depth = -1;   // behind the chunk's end
            }
            sm.depth[lane] = depth;                          // -1: no result
            float p[kMaxDK];
#pragma unroll
            for (int d = 0; d < kMaxDK; ++d) p[d] = d < DK ? sm.q[lane][d < DK ? d : 0] : 0.f;
            sm.z[lane] = code_of(p, DK == 3 ? 3 : g.dK, g.bits);
        }
        __syncwarp();
    }

    constexpr int H = Sm::MMA ? DVP / 64 : 1;                // 64-column halves (bf16)
    const int g4 = lane >> 2, s4 = lane & 3;
    // Of 16 keys' rows (x: g, g + 8), A operands m of the values 16 (g / 2) + g % 2 + 4c, + 2 for
    // c = 0..3: mul(c, m).
    auto operands = [](const uint32_t (*x)[8], auto mul) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t m[4] = {movmatrix_trans(x[0][2 * c]), movmatrix_trans(x[0][2 * c + 1]),
                                   movmatrix_trans(x[1][2 * c]), movmatrix_trans(x[1][2 * c + 1])};
            mul(c, m);
        }
    };
    const int column = 16 * (g4 >> 1) + (g4 & 1);            // the first of the lane's values
    // Where in a row the lane's 32 bytes of 64 columns are (bf16; within the row).
    auto spot = [&](int hh, int e) { return WIDE ? min(128 * hh + 32 * s4, vrow - 32) : min(8 * hh + 2 * s4 + e, ppr - 1) * 16; };

    // Shared keys: whole steps of the chunk's tokens where they lie within a page, the other
    // tokens, the nodes up to the block's last one.
    constexpr int KS = Sm::KS, KL = Sm::KL, KP = Sm::KP, NV = Sm::NV;
    const int CW = NW * cs, cw = warp * cs + cr;             // the cluster's warps, this one
    const bool pairs = (reinterpret_cast<uintptr_t>(g.k_pages) & 7) == 0;    // two coordinates a load
    const int n_main = DK == 3 && pairs && pmask >= KS - 1 && (cC & (KS - 1)) == 0 ? L / KS : 0;
    const int n_node = (nn + KS - 1) / KS, n_rest = (L + KS - 1) / KS - n_main + n_node;
    const char *vt = static_cast<const char *>(g.v_pages), *vf = static_cast<const char *>(g.v) + node0 * vrow;
    const char *kt = reinterpret_cast<const char *>(g.k_pages), *kf = reinterpret_cast<const char *>(g.k) + node0 * krow;
    const int first_key = Sm::MMA ? 2 * s4 : 2 * (lane >> 3);                // the lane's first key of a step
    const int piece = min(lane & 15, ppr - 1) * 16;          // float32: its bytes of a value row
    const int second = NV == 4 ? 0 : min((lane & 15) + 16, ppr - 1) * 16 - piece;

    // ------------------------------------------------------------ window ---
    // The cluster's warps take the nodes in turn.  While a window's keys and values are under
    // way the next one's search begins.
    const int kh = (g.kw + 1) / 2;
    const bool few = g.kw <= 64;
    auto next = [&](int r) {                                 // the warp's next node with a result, from r on
        while (r < nq && sm.depth[r] < 0) r += CW;
        return r;
    };
    // Rank: among the fences, then among a block's entries, 64 probes a step; the last step's are
    // asked for here and looked at in found.  Where a window has up to 64 entries, those that
    // it may hold are asked for with them.
    uint64_t z = 0, zz[2] = {0, 0};
    int ra = 0, re = 0, cand[4], lo = 0;                     // entries before ra are <= z, from re on > z
    bool open[2] = {false, false};
    auto probe = [&](int step) {
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            const int at = ra + (v * 32 + lane + 1) * step - 1, to = min(at, cC - 1);
            const int id = ot[to >> psh];
            const bool in = (unsigned)id < (unsigned)g.c.opages;
            open[v] = at < re && in;
            lost |= at < re && !in;
            zz[v] = ld_code(codes, in ? row_at(id, to) : 0, g.code64);
        }
    };
    auto found = [&](int step) {
        __syncwarp();
        const int le = __popc(__ballot_sync(kFull, open[0] && zz[0] <= z)) + __popc(__ballot_sync(kFull, open[1] && zz[1] <= z));
        ra = min(ra + le * step, re);
        re = min(re, ra + step - 1);
    };
    auto search = [&](int r) {
        if (chunk == 0) return;
        z = sm.z[r];
        const int f8 = 8 * __popc(__ballot_sync(kFull, lane * 8 + 7 < nf && sm.fence[lane * 8 + 7] <= z));
        const int f = f8 + (lane & 7);
        const int n = f8 + __popc(__ballot_sync(kFull, lane < 8 && f < nf && sm.fence[min(f, kTreeFences - 1)] <= z));
        ra = n > 0 ? ((n - 1) << fsh) + 1 : 0;
        re = n > 0 ? min(cC, n << fsh) : 0;
        for (int len = 1 << fsh; len > 64;) {                // most entries still open
            const int step = (len + 63) / 64;
            probe(step);
            found(step);
            len = step - 1;
        }
        probe(1);
        if (few) {
            lo = min(max(ra - kh, 0), cC - g.kw);
            const int hi = min(max(re - kh, 0), cC - g.kw) + g.kw;
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const int at = lo + v * 32 + lane, id = ot[min(at, cC - 1) >> psh];
                cand[v] = ldi_if(entries + row_at(id, at), at < hi && (unsigned)id < (unsigned)g.c.opages);
            }
        }
    };
    auto take_window = [&](int r) {
        constexpr int LPR = PPR, RPI = 32 / LPR;             // float32: lanes a value row, rows a load
        constexpr int WS = Sm::MMA ? 16 : 4 * RPI;           // entries a step
        auto &ga = sm.gather[warp];
        float *win = sm.win[r];
        const int64_t rid = node0 + f0 + r;
        found(1);
        const int st = min(max(ra - kh, 0), cC - g.kw), from = st - lo;
        if (lane == 0) sm.wst[r] = st;
        if (few) {
#pragma unroll
            for (int v = 0; v < 4; ++v) ga.cand[v * 32 + lane] = cand[v];
            __syncwarp();
        }
        float q[DK], sw = 0.f, mr = INFINITY;
#pragma unroll
        for (int d = 0; d < DK; ++d) q[d] = sm.q[r][d];
        int following = nq;
        for (int t0 = 0; t0 < g.kw; t0 += 64) {              // up to 64 entries at a time, two a lane
            int row[2];
            bool is[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const int slot = t0 + v * 32 + lane;
                const bool there = slot < g.kw;
                int j;
                if (few) {
                    j = there ? ga.cand[min(from + slot, 127)] : -1;
                } else {
                    const int at = st + slot, id = ot[min(at, cC - 1) >> psh];
                    j = ldi_if(entries + row_at(id, at), there && (unsigned)id < (unsigned)g.c.opages);
                }
                const bool in = (unsigned)j < (unsigned)cC;
                if (g.idx && there) g.idx[rid * g.kw + slot] = in ? j : -1;
                const int id = pt[(in ? j : 0) >> psh];
                is[v] = in && (unsigned)id < (unsigned)g.c.pages;
                row[v] = row_at(id, j);
                lost |= there && !is[v];
            }
            __syncwarp();                                    // the entries have been read
            // In the place of an entry that is none, another of the window: its values enter the
            // sum anyway, so that a zero weight adds no NaN of its own.
            const unsigned h0 = __ballot_sync(kFull, is[0]), h1 = __ballot_sync(kFull, is[1]);
            if ((h0 & h1) != kFull) {
                const int some = __shfl_sync(kFull, h0 ? row[0] : row[1], __ffs(h0 ? h0 : h1 | 1u << 31) - 1);
                if (!is[0]) row[0] = h0 | h1 ? some : 0;
                if (!is[1]) row[1] = h0 | h1 ? some : 0;
            }
            ga.row[lane] = row[0];
            ga.row[32 + lane] = row[1];
            __syncwarp();                                    // the rows are there
            // Coordinates one a lane, CR rows a load, so that a load touches a row's line once.
            constexpr int CR = 32 / DK, CL = (64 + CR - 1) / CR;
            const int steps = (min(64, g.kw - t0) + WS - 1) / WS;
            const int c_row = lane / DK, c_at = lane % DK, entries_here = min(64, g.kw - t0);
            float x[CL];
#pragma unroll
            for (int v = 0; v < CL; ++v) {
                x[v] = 0.f;
                if (v * CR < entries_here && c_row < CR && v * CR + c_row < 64 && (DK == 3 || c_at < g.dK))
                    x[v] = __ldg(reinterpret_cast<const float *>(kt + (uint64_t)(uint32_t)ga.row[v * CR + c_row] * (uint32_t)krow) + c_at);
            }
            auto load = [&](uint32_t (&y)[2][8], int i, int hh) {
                if (i >= steps) return;
                const int *rows = ga.row + i * WS;
                if constexpr (Sm::MMA) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const char *p = vt + (uint64_t)(uint32_t)rows[8 * v + g4] * (uint32_t)vrow;
                        ld32<WIDE>(y[v], p + spot(hh, 0), p + spot(hh, 1));
                    }
                } else {
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        *reinterpret_cast<uint4 *>(&y[v / 2][v % 2 * 4]) =
                            ld16(vt + (uint64_t)(uint32_t)rows[v * RPI + lane / LPR] * (uint32_t)vrow + min(lane % LPR, ppr - 1) * 16);
                }
            };
            constexpr int NB = Sm::NB;                       // steps under way
            uint32_t buf[NB][2][8];
#pragma unroll
            for (int o = 0; o < NB; ++o) load(buf[o], o, 0);
            if (t0 + 64 >= g.kw) {
                following = next(r + CW);
                if (following < nq) search(following);
            }
#pragma unroll
            for (int v = 0; v < CL; ++v)
                if (v * CR < entries_here && c_row < CR && v * CR + c_row < 64) ga.x[v * CR * DK + lane] = x[v];
            __syncwarp();
            float d2[2];
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                d2[v] = 0.f;
#pragma unroll
                for (int d = 0; d < DK; ++d) {
                    const float f = q[d] - ga.x[(v * 32 + lane) * DK + d];
                    d2[v] = __fmaf_rn(f, f, d2[v]);
                }
                if (!is[v]) d2[v] = INFINITY;
            }
            float scale = 1.f;                               // of the sums so far
            if constexpr (WK == kWSoftmax) {
                float least = fminf(d2[0], d2[1]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) least = fminf(least, __shfl_xor_sync(kFull, least, o));
                if (least < mr) {
                    scale = mr == INFINITY ? 0.f : __expf((least - mr) * inv_g2);
                    sw *= scale;
                    mr = least;
                }
            }
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float w = is[v] ? weight_fast<WK>(d2[v], mr, inv_g2) : 0.f;
                sw += w;
                if constexpr (Sm::MMA) {
                    float left = w;
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        const __nv_bfloat16 part = __float2bfloat16_rn(left);
                        ga.bits[p][v * 32 + lane] = __bfloat16_as_ushort(part);
                        left -= __bfloat162float(part);
                    }
                } else {
                    ga.w[v * 32 + lane] = w;
                }
            }
            __syncwarp();                                    // the weights are there
            for (int hh = 0;; ++hh) {                        // 64 columns at a time (bf16)
                float acc[16] = {0.f};                       // float32: a piece's sums
                auto use = [&](const uint32_t (&y)[2][8], int i) {
                    if constexpr (Sm::MMA) {
                        // The weights' parts in columns 0, 1 and 2 of B.
                        uint32_t b0 = 0u, b1 = 0u;
                        if (g4 < 3) {
                            b0 = *reinterpret_cast<const uint32_t *>(&ga.bits[g4][i * WS + 2 * s4]);
                            b1 = *reinterpret_cast<const uint32_t *>(&ga.bits[g4][i * WS + 2 * s4 + 8]);
                        }
                        __syncwarp();
                        operands(y, [&](int w, const uint32_t (&m)[4]) {
                            mma16816(*reinterpret_cast<float(*)[4]>(&acc[4 * w]), m, b0, b1);
                        });
                    } else {
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const uint32_t *u = &y[v / 2][v % 2 * 4];
                            const float2 w = dup2(ga.w[i * WS + v * RPI + lane / LPR]);
                            const float2 a = fma2(w, make_float2(__uint_as_float(u[0]), __uint_as_float(u[1])), make_float2(acc[0], acc[1]));
                            const float2 b = fma2(w, make_float2(__uint_as_float(u[2]), __uint_as_float(u[3])), make_float2(acc[2], acc[3]));
                            acc[0] = a.x;
                            acc[1] = a.y;
                            acc[2] = b.x;
                            acc[3] = b.y;
                        }
                    }
                };
                for (int i = 0; i < steps; i += NB) {
#pragma unroll
                    for (int o = 0; o < NB; ++o) {
                        if (i + o < steps) use(buf[o], i + o);
                        load(buf[o], i + o + NB, hh);
                    }
                }
                const bool more = hh + 1 < H && ppr > 8;
                if (more) {
#pragma unroll
                    for (int o = 0; o < NB; ++o) load(buf[o], o, 1);
                }
                auto put = [&](int c, float a) {             // onto the sums so far
                    float *to = win + hh * 64 + c;
                    *to = t0 > 0 ? __fmaf_rn(scale, *to, a) : a;
                };
                if constexpr (Sm::MMA) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {            // column 2 is the next lane's
                        const float a = __shfl_down_sync(kFull, acc[4 * c], 1), b = __shfl_down_sync(kFull, acc[4 * c + 2], 1);
                        if (s4 == 0) {
                            put(column + 4 * c, acc[4 * c] + (acc[4 * c + 1] + a));
                            put(column + 4 * c + 2, acc[4 * c + 2] + (acc[4 * c + 3] + b));
                        }
                    }
                } else {
#pragma unroll
                    for (int o = 16; o >= LPR; o >>= 1)
#pragma unroll
                        for (int c = 0; c < 4; ++c) acc[c] += __shfl_xor_sync(kFull, acc[c], o);
                    if (lane < LPR) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) put(lane * 4 + c, acc[c]);
                    }
                }
                if (!more) break;
            }
            __syncwarp();                                    // rows and weights have been read
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sw += __shfl_xor_sync(kFull, sw, o);
        if (lane == 0) {
            sm.swin[r] = sw;
            sm.mwin[r] = mr;
        }
        return following;
    };
    auto no_window = [&](int r) {
        for (int c = lane; c < DVP; c += 32) sm.win[r][c] = 0.f;
        if (g.idx)
            for (int c = lane; c < g.kw; c += 32) g.idx[(node0 + f0 + r) * g.kw + c] = -1;
        if (lane == 0) {
            sm.swin[r] = 0.f;
            sm.mwin[r] = INFINITY;
        }
        return next(r + CW);
    };
    int mine = nq;                                           // the node that is searched for

    // ------------------------------------------------------- shared keys ---
    // Dealt to the cluster's warps.  A lane has the weights of one node of a group and 4
    // (float32: 2) keys: node lane / 4 and keys 2 s4, + 1, + 8, + 9; or node lane % 8 and keys
    // 2 (lane / 8), + 1.
    {
        constexpr int ACC = DVP / 4;
        const bool two = nq > 8;                             // nodes in both groups
        const int node = Sm::MMA ? g4 : lane & 7;
        float acc[NG][ACC];                                  // MMA: [half][w][4]; else [4 nodes][DVP / 64][4]
        float2 sum[NG];                                      // weights of first and second keys
        float m[NG];                                         // softmax shifts
        float q[NG][DK];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
#pragma unroll
            for (int e = 0; e < ACC; ++e) acc[n][e] = 0.f;
            sum[n] = make_float2(0.f, 0.f);
            m[n] = INFINITY;
#pragma unroll
            for (int d = 0; d < DK; ++d) q[n][d] = sm.q[8 * n + node][d];
        }
        // Weights of group n for KP pairs of keys given as 2 DK floats, one key after the other;
        // takes: which keys the node takes, a bit each (looked at where masked).
        auto weigh = [&](int n, const float2 (*k)[DK], float2 *w, unsigned takes, bool masked) {
#pragma unroll
            for (int e = 0; e < KP; ++e) {
                float x[2 * DK];
#pragma unroll
                for (int d = 0; d < DK; ++d) {
                    const float2 f = sub2(make_float2(q[n][2 * d % DK], q[n][(2 * d + 1) % DK]), k[e][d]);
                    x[2 * d] = f.x;
                    x[2 * d + 1] = f.y;
                }
                w[e] = make_float2(0.f, 0.f);
#pragma unroll
                for (int d = 0; d < DK; ++d) {
                    w[e].x = __fmaf_rn(x[d], x[d], w[e].x);
                    w[e].y = __fmaf_rn(x[DK + d], x[DK + d], w[e].y);
                }
                if (masked) {                                // infinitely far: no key of the node
                    if (!(takes >> (2 * e) & 1u)) w[e].x = INFINITY;
                    if (!(takes >> (2 * e) & 2u)) w[e].y = INFINITY;
                }
            }
            if constexpr (WK == kWSoftmax) {                 // move the shift to the least d2
                float least = fminf(w[0].x, w[0].y);
                if (KP == 2) least = fminf(least, fminf(w[KP - 1].x, w[KP - 1].y));
#pragma unroll
                for (int o = Sm::MMA ? 1 : 8; o <= (Sm::MMA ? 2 : 16); o <<= 1) least = fminf(least, __shfl_xor_sync(kFull, least, o));
                const float to = fminf(m[n], least);
                if (__any_sync(kFull, to != m[n])) {
                    const float f = to == m[n] ? 1.f : m[n] == INFINITY ? 0.f : __expf((to - m[n]) * inv_g2);
                    if constexpr (Sm::MMA) {                 // the sums of nodes 2 s4 and + 1
                        const float fa = __shfl_sync(kFull, f, 8 * s4), fb = __shfl_sync(kFull, f, 8 * s4 + 4);
#pragma unroll
                        for (int c = 0; c < ACC; ++c) acc[n][c] *= c & 1 ? fb : fa;
                    } else {
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float fr = __shfl_sync(kFull, f, (lane >> 4) * 4 + r);
#pragma unroll
                            for (int c = 0; c < DVP / 16; ++c) acc[n][r * (DVP / 16) + c] *= fr;
                        }
                    }
                    sum[n] = mul2(sum[n], dup2(f));
                    m[n] = to;
                }
            }
            const float shift = m[n] == INFINITY ? 0.f : m[n];   // finite even where no key is taken yet
#pragma unroll
            for (int e = 0; e < KP; ++e) {
                w[e] = weight_pair<WK>(w[e], shift, dup2(inv_g2));
                if (masked) {
                    if (!(takes >> (2 * e) & 1u)) w[e].x = 0.f;
                    if (!(takes >> (2 * e) & 2u)) w[e].y = 0.f;
                }
                sum[n] = add2(sum[n], w[e]);
            }
        };
        // The step's values times the weights of both groups' nodes.
        auto multiply = [&](const float2 (*w)[Sm::KP], const uint32_t (*v)[8], auto &more) {
            if constexpr (Sm::MMA) {
                uint32_t b[NG][6];                           // three parts of two pairs
#pragma unroll
                for (int n = 0; n < NG; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float2 left = w[n][e];
#pragma unroll
                        for (int p = 0; p < 3; ++p) b[n][2 * p + e] = take_part(left);
                    }
                __syncwarp();
#pragma unroll
                for (int hh = 0; hh < H; ++hh)
                    operands(v + 2 * hh, [&](int c, const uint32_t (&x)[4]) {
#pragma unroll
                        for (int n = 0; n < NG; ++n) {
                            if (n > 0 && !two) break;
                            float(&o)[4] = *reinterpret_cast<float(*)[4]>(&acc[n][16 * hh + 4 * c]);
#pragma unroll
                            for (int p = 0; p < 3; ++p) mma16816(o, x, b[n][2 * p], b[n][2 * p + 1]);
                        }
                    });
            } else {
                float(&ws)[8][20] = sm.w[warp];
#pragma unroll
                for (int n = 0; n < NG; ++n) {
                    ws[first_key][8 * n + node] = w[n][0].x;
                    ws[first_key + 1][8 * n + node] = w[n][0].y;
                }
                __syncwarp();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (e == 4) more(4);                     // the values of the other four keys
#pragma unroll
                    for (int n = 0; n < NG; ++n) {
                        if (n > 0 && !two) break;
                        const float4 w4 = *reinterpret_cast<const float4 *>(&ws[e][8 * n + (lane >> 4) * 4]);
                        const float wr[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int c = 0; c < DVP / 64; ++c) {
                            const int at = (e & 3) * (DVP / 64) + c;
                            const uint32_t *y = &v[at / 2][at % 2 * 4];
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                float *o = &acc[n][r * (DVP / 16) + 4 * c];
                                const float2 lo = fma2(dup2(wr[r]), make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), make_float2(o[0], o[1]));
                                const float2 hi = fma2(dup2(wr[r]), make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])), make_float2(o[2], o[3]));
                                o[0] = lo.x;
                                o[1] = lo.y;
                                o[2] = hi.x;
                                o[3] = hi.y;
                            }
                        }
                    }
                }
                __syncwarp();                                // the weights have been read
            }
        };
        // Whole steps within a page.
        for (int i = cw; i < n_main; i += CW) {
            const int first = cC + i * KS, id = pt[first >> psh];
            if (__any_sync(kFull, (unsigned)id >= (unsigned)g.c.pages)) {
                lost = true;
                continue;
            }
            const uint32_t r0 = (uint32_t)row_at(id, first);
            const float2 *kp = reinterpret_cast<const float2 *>(kt + (uint64_t)r0 * 12u + 12 * first_key);
            float2 kc[KP][DK];
#pragma unroll
            for (int e = 0; e < KP; ++e)
#pragma unroll
                for (int d = 0; d < DK; ++d) kc[e][d] = __ldg(kp + 12 * e + d);
            const char *src = vt + (uint64_t)r0 * (uint32_t)vrow;
            uint32_t v[NV / 2][8];
            auto values = [&](int e0) {
                if constexpr (Sm::MMA) {
#pragma unroll
                    for (int e = 0; e < 2 * H; ++e) {
                        const char *p = src + (8 * (e & 1) + g4) * vrow;
                        ld32<WIDE>(v[e], p + spot(e / 2, 0), p + spot(e / 2, 1));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < NV; ++e)
                        *reinterpret_cast<uint4 *>(&v[e / 2][e % 2 * 4]) =
                            ld16(src + (e0 + e / (NV / 4)) * vrow + piece + e % (NV / 4) * second);
                }
            };
            values(0);
            float2 w[NG][KP];
#pragma unroll
            for (int n = 0; n < NG; ++n)
                if (n == 0 || two) weigh(n, kc, w[n], 0u, false);
                else w[n][0] = w[n][KP - 1] = make_float2(0.f, 0.f);
            multiply(w, v, values);
        }
        // The lines and fences are there for the rest; the first window's search begins.
#pragma unroll
        for (int u = 0; u < NF; ++u) sm.fence[u * NT + tid] = fz[u];
        __syncthreads();
        mine = next(cw);
        if (mine < nq) search(mine);
        // The others, key by key; the deal goes on where the whole steps' ended.
        for (int i = (cw + CW - n_main % CW) % CW; i < n_rest; i += CW) {
            const bool fresh = i >= n_rest - n_node;
            const int x0 = (fresh ? i - (n_rest - n_node) : n_main + i) * KS, end = fresh ? nn : L;
            const char *kb = fresh ? kf : kt, *vb = fresh ? vf : vt;
            // Row of key k of the step (any where there is none), and whether there is one.
            auto row_of = [&](int k, bool &in) {
                const int x = min(x0 + k, end - 1);
                in = x0 + k < end;
                if (fresh) return (uint32_t)x;
                const int id = pt[(cC + x) >> psh];
                const bool page = (unsigned)id < (unsigned)g.c.pages;
                lost |= !page;
                in = in && page;
                return (uint32_t)(page ? row_at(id, cC + x) : 0);
            };
            uint32_t row[KL], vrows[2];
            unsigned takes[NG] = {0};                        // which the node takes, a bit each
            unsigned above[NG];
#pragma unroll
            for (int n = 0; n < NG; ++n) above[n] = fresh ? sm.above[8 * n + node][x0 >> 5] >> (x0 & 31) : ~0u;
#pragma unroll
            for (int e = 0; e < KL; ++e) {
                const int key = first_key + (e & 1) + 4 * (e & 2);
                bool in;
                row[e] = row_of(key, in);
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    if (in && (above[n] >> key & 1u)) takes[n] |= 1u << e;
            }
            bool in;
            vrows[0] = Sm::MMA ? row_of(g4, in) : row[0];
            vrows[1] = Sm::MMA ? row_of(g4 + 8, in) : row[1];
            __syncwarp();
            uint32_t v[NV / 2][8];
            auto values = [&](int e0) {
                if constexpr (Sm::MMA) {
#pragma unroll
                    for (int e = 0; e < 2 * H; ++e) {
                        const char *p = vb + (uint64_t)vrows[e & 1] * (uint32_t)vrow;
                        ld32<WIDE>(v[e], p + spot(e / 2, 0), p + spot(e / 2, 1));
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < NV; ++e) {
                        const int k = e0 + e / (NV / 4);
                        const uint32_t r = __shfl_sync(kFull, vrows[e / (NV / 4) & 1], k / 2 * 8);
                        *reinterpret_cast<uint4 *>(&v[e / 2][e % 2 * 4]) =
                            ld16(vb + (uint64_t)r * (uint32_t)vrow + piece + e % (NV / 4) * second);
                    }
                }
            };
            values(0);
            float2 kc[KP][DK], w[NG][KP];
#pragma unroll
            for (int e = 0; e < KP; ++e) {
                float x[2 * DK];
#pragma unroll
                for (int d = 0; d < 2 * DK; ++d)
                    x[d] = DK == 3 || d % DK < g.dK ? __ldg(reinterpret_cast<const float *>(kb + (uint64_t)row[2 * e + d / DK] * (uint32_t)krow) + d % DK) : 0.f;
#pragma unroll
                for (int d = 0; d < DK; ++d) kc[e][d] = make_float2(x[2 * d], x[2 * d + 1]);
            }
#pragma unroll
            for (int n = 0; n < NG; ++n) weigh(n, kc, w[n], takes[n], true);
            multiply(w, v, values);
        }
        float(&part)[ROWS][DVP + 4] = sm.part[warp];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
            float total = sum[n].x + sum[n].y;
#pragma unroll
            for (int o = Sm::MMA ? 1 : 8; o <= (Sm::MMA ? 2 : 16); o <<= 1) total += __shfl_xor_sync(kFull, total, o);
            if (Sm::MMA ? s4 == 0 : lane < 8) {
                sm.psum[warp][8 * n + node] = total;
                sm.pmin[warp][8 * n + node] = m[n];
            }
            if (n > 0 && !two) break;
            if constexpr (Sm::MMA) {
#pragma unroll
                for (int c = 0; c < 4 * H; ++c) {
                    float *to = &part[8 * n + 2 * s4][c / 4 * 64 + column + c % 4 * 4];
                    to[0] = acc[n][4 * c];
                    to[2] = acc[n][4 * c + 2];
                    to[DVP + 4] = acc[n][4 * c + 1];
                    to[DVP + 6] = acc[n][4 * c + 3];
                }
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int c = 0; c < DVP / 64; ++c) {
                        const float *o = &acc[n][r * (DVP / 16) + 4 * c];
                        *reinterpret_cast<float4 *>(&part[8 * n + (lane >> 4) * 4 + r][(lane & 15) * 4 + 64 * c]) = make_float4(o[0], o[1], o[2], o[3]);
                    }
            }
        }
    }

    while (mine < nq) mine = chunk > 0 ? take_window(mine) : no_window(mine);
    if (lost) set_status(g.status, ZETA_ERR_BOUNDS);

    // ---------------------------------------------------------- epilogue ---
    // Node r is finished by block r % cs, which has its window: the warps' parts of its sums are
    // joined in each block, the blocks' by that one.
    cg::cluster_group cl = cg::this_cluster();
    __syncthreads();
    // P parts onto one shift: factors of the parts, of the window (where it takes part), and the
    // sum of weights.
    auto join = [&](int P, int r, bool window, auto psum, auto pmin) {
        float total = window ? sm.swin[r] : 0.f;
        if constexpr (WK == kWSoftmax) {
            float least = window ? sm.mwin[r] : INFINITY;
            for (int p = 0; p < P; ++p) least = fminf(least, pmin(p));
            auto factor = [&](float m) { return m == INFINITY ? 0.f : __expf((least - m) * inv_g2); };
            if (window) total *= sm.factor[P][r] = factor(sm.mwin[r]);
            for (int p = 0; p < P; ++p) total = __fmaf_rn(sm.factor[p][r] = factor(pmin(p)), psum(p), total);
            sm.least[r] = least;
        } else {
            for (int p = 0; p < P; ++p) total += psum(p);
        }
        sm.total[r] = total;
    };
    auto add = [&](float2 o, int p, int r, float2 x) { return WK == kWSoftmax ? fma2(dup2(sm.factor[p][r]), x, o) : add2(o, x); };
    if (cs > 1) {
        if (tid < nq)
            join(NW, tid, false, [&](int p) { return sm.psum[p][tid]; }, [&](int p) { return sm.pmin[p][tid]; });
        __syncthreads();
        for (int i = tid; i < ROWS * (DVP / 2); i += NT) {
            const int r = i / (DVP / 2), col = i % (DVP / 2) * 2;
            if (r >= nq) break;
            float2 o = make_float2(0.f, 0.f);
#pragma unroll
            for (int p = 0; p < NW; ++p) o = add(o, p, r, *reinterpret_cast<const float2 *>(&sm.part[p][r][col]));
            *reinterpret_cast<float2 *>(&sm.part[0][r][col]) = o;
        }
        if (tid < nq) {
            sm.psum[0][tid] = sm.total[tid];
            sm.pmin[0][tid] = WK == kWSoftmax ? sm.least[tid] : 0.f;
        }
        cl.sync();
    }
    const int parts = cs > 1 ? cs : NW;
    auto of = [&](int p) { return cs > 1 ? cl.map_shared_rank(&sm, p) : &sm; };
    const bool finish = tid < nq && tid % cs == cr && sm.depth[min(tid, ROWS - 1)] >= 0;
    if (finish) {
        join(parts, tid, true, [&](int p) { return of(p)->psum[cs > 1 ? 0 : p][tid]; }, [&](int p) { return of(p)->pmin[cs > 1 ? 0 : p][tid]; });
        g.rowsum[node0 + f0 + tid] = sm.total[tid];
    }
    __syncthreads();
    // Two columns a thread.
    bool bad = false;
    V *out = static_cast<V *>(g.out) + (node0 + f0) * g.dV;
    for (int i = tid; i < ROWS * (DVP / 2); i += NT) {
        const int r = i / (DVP / 2) * cs + cr, col = i % (DVP / 2) * 2;
        if (r >= nq) break;
        if (sm.depth[r] < 0 || col >= g.dV) continue;
        float2 o = *reinterpret_cast<const float2 *>(&sm.win[r][col]);
        if (WK == kWSoftmax) o = mul2(o, dup2(sm.factor[parts][r]));
        if (cs == 1) {
#pragma unroll
            for (int p = 0; p < NW; ++p) o = add(o, p, r, *reinterpret_cast<const float2 *>(&sm.part[p][r][col]));
        } else {
            for (int p = 0; p < cs; ++p) o = add(o, p, r, *reinterpret_cast<const float2 *>(&of(p)->part[0][r][col]));
        }
        o.x = __fdiv_rn(o.x, sm.total[r]);
        o.y = __fdiv_rn(o.y, sm.total[r]);
        if (!isfinite(o.x) || !isfinite(o.y)) sm.again[r] = bad = true;
        if constexpr (Sm::MMA) *reinterpret_cast<__nv_bfloat162 *>(out + r * g.dV + col) = __floats2bfloat162_rn(o.x, o.y);
        else *reinterpret_cast<float2 *>(out + r * g.dV + col) = o;
    }
    if (__syncthreads_or(bad)) {                             // the fast results are written first
        for (int r = cw; r < nq; r += CW)
            if (sm.depth[r] >= 0 && sm.again[r])
                slow_node<V, DVP, DK, WK>(g, node0 + f0 + r, b, h, seq.start, cC > 0 ? sm.wst[r] : 0, sm.above[r], inv_g2);
    }
    if (cs > 1) cl.sync();                                   // read before any block ends
}

template <typename V, int DVP, int NG, int DK, int WK, bool WIDE>
cudaError_t run_tree_tile(const Prob &p, const TreeArgs &g, int cs, cudaStream_t st) {
    static PerDeviceOnce once;
    constexpr size_t smem = sizeof(TreeSmem<V, DVP, NG>);
    constexpr int Rows = TreeSmem<V, DVP, NG>::ROWS;
    cudaError_t e = once.run([] {
        return cudaFuncSetAttribute(tree_tile_kernel<V, DVP, NG, DK, WK, WIDE>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((g.c.n + Rows - 1) / Rows * cs), (unsigned)p.S);
    cfg.blockDim = dim3(TreeSmem<V, DVP, NG>::NW * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = (unsigned)cs;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, tree_tile_kernel<V, DVP, NG, DK, WK, WIDE>, g, cs);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename V, int DVP, int NG, bool WIDE>
cudaError_t dispatch_tree_tile(const Prob &p, const TreeArgs &g, int cs, cudaStream_t st) {
#define ZETA_TREE(D)                                                                  \
    (p.wk == kWSoftmax     ? run_tree_tile<V, DVP, NG, D, kWSoftmax, WIDE>(p, g, cs, st)        \
     : p.wk == kWInvEuclid ? run_tree_tile<V, DVP, NG, D, kWInvEuclid, WIDE>(p, g, cs, st)      \
                           : run_tree_tile<V, DVP, NG, D, kWCauchy, WIDE>(p, g, cs, st))
    return p.dK == 3 ? ZETA_TREE(3) : ZETA_TREE(4);
#undef ZETA_TREE
}

}  // namespace
}  // namespace zeta
