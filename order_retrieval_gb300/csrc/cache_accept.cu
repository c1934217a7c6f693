// cache_accept.cu -- the accepted branch of a draft into the pages.
//
// The line of nodes that ends in leaf[b], up to the end of the chunk that start lies in and to
// granted[b] tokens where that is given, becomes the sequence's next tokens: a copy of rows, as cache_append.cu, through the
// line.  A block per sequence and head finds the line in the parents in shared memory as
// bits (one thread climbs, a run of nodes below one another in one step) and puts it in
// order by counting bits, then copies its rows, a thread per 16-byte piece of a value row (a
// value where the row is no multiple of 16 bytes), four rows a thread under way; the row's
// first threads also carry its coordinates.
//
// 64 sequences, lines of a few nodes, 8 heads: 3.3 us, a launch and four dependent loads.  48
// lines of 64 to 128 nodes, 4 heads, rows of 132 bytes a value a thread: 6.9 us for 4 MB (one
// row a thread at a time, the line climbed node by node: 14.7).
#include "cache_tree.cuh"

namespace zeta {
namespace {

constexpr int kThreads = 256;

template <typename Piece>
__global__ void __launch_bounds__(kThreads)
cache_accept_kernel(const float *__restrict__ k, const Piece *__restrict__ v,
                    float *__restrict__ k_pages, Piece *__restrict__ v_pages, Cache c,
                    const int32_t *__restrict__ parents, const int32_t *__restrict__ leaves,
                    const int32_t *__restrict__ granted, int32_t *__restrict__ accepted,
                    int32_t *__restrict__ path, int32_t *status,
                    int N, int H, int C, int dK, int ppr) {
    __shared__ int parent[kMaxDraft], line[kMaxDraft];
    __shared__ uint32_t run[kMaxDraft / 32], bits[kMaxDraft / 32];
    __shared__ int len_sh;
    const int tid = threadIdx.x, warp = tid >> 5, h = blockIdx.x, b = blockIdx.y;
    const int early = tid < c.n ? __ldg(parents + (int64_t)b * c.n + tid) : -1;
    int leaf = __ldg(leaves + b);
    const int most = granted ? max(__ldg(granted + b), 0) : INT32_MAX;
    const Seq seq = drafts_of(c, b, N, status);
    if (leaf < -1 || leaf >= seq.count) {
        if (tid == 0 && seq.count > 0) set_status(status, ZETA_ERR_BOUNDS);
        leaf = -1;
    }
    if (tid <= leaf) parent[tid] = early;
    for (int u = kThreads + tid; u <= leaf; u += kThreads) parent[u] = __ldg(parents + (int64_t)b * c.n + u);
    if (tid < kMaxDraft / 32) bits[tid] = 0u;
    __syncthreads();
    for (int w = warp; w * 32 <= leaf; w += kThreads / 32) {
        const uint32_t r = run_bits(parent, w, leaf + 1);
        if ((tid & 31) == 0) run[w] = r;
    }
    __syncthreads();
    if (tid == 0) {
        const int depth = climb_bits(parent, run, leaf, bits);
        if (leaf >= 0 && depth < 0) set_status(status, ZETA_ERR_BOUNDS);
        len_sh = depth + 1;
    }
    __syncthreads();
    const int len = min(min(len_sh, C - seq.start % C), most);       // no line: 0
    if (len > 0) {                                   // the line's nodes in order
        for (int u = tid; u <= leaf; u += kThreads) {
            const uint32_t own = bits[u >> 5];
            if (!(own >> (u & 31) & 1u)) continue;
            int at = __popc(own & ((1u << (u & 31)) - 1u));
            for (int w = 0; w < u >> 5; ++w) at += __popc(bits[w]);
            line[at] = u;
        }
        __syncthreads();
    }
    if (h == 0) {
        if (tid == 0) accepted[b] = len;
        if (path)
            for (int d = tid; d < c.n; d += kThreads) path[(int64_t)b * c.n + d] = d < len ? line[d] : -1;
    }
    const int32_t *ptab = c.ptab + (int64_t)b * c.tlen;
    const int64_t rows = ((int64_t)b * H + h) * c.n;
    const int in = tid / ppr, ch = tid - in * ppr, rpb = kThreads / ppr;
    if (in >= rpb) return;
    // Rows four at a time, so that their pages and values are under way together.
    constexpr int U = 4;
    for (int d0 = in; d0 < len; d0 += U * rpb) {
        int row[U];
        Piece x[U];
        float y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) row[u] = page_id(ptab, seq.start + min(d0 + u * rpb, len - 1), c.psh);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = rows + line[min(d0 + u * rpb, len - 1)];
            x[u] = v[r * ppr + ch];
            y[u] = k[r * dK + min(ch, dK - 1)];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int d = d0 + u * rpb;
            if (d >= len) break;
            const int to = row_in(row[u], seq.start + d, h, H, c.psh, c.pmask, c.pages);
            if (to < 0) {
                set_status(status, ZETA_ERR_BOUNDS);
                continue;
            }
            v_pages[(int64_t)to * ppr + ch] = x[u];
            if (ch < dK) k_pages[(int64_t)to * dK + ch] = y[u];
            for (int e = ch + ppr; e < dK; e += ppr) k_pages[(int64_t)to * dK + e] = k[(rows + line[d]) * dK + e];
        }
    }
}

}  // namespace

cudaError_t launch_cache_accept(const Prob &p, const Cache &c, const int32_t *parent,
                                const int32_t *leaf, const int32_t *granted, const float *k,
                                const void *v, float *k_pages, void *v_pages, int32_t *accepted,
                                int32_t *path, int32_t *status, cudaStream_t st) {
    const int esz = p.vdt == ZETA_BF16 ? 2 : 4;
    const int bytes = p.dV * esz;
#define ZETA_ACCEPT(Piece)                                                                     \
    cache_accept_kernel<Piece><<<dim3((unsigned)p.H, (unsigned)p.B), kThreads, 0, st>>>(       \
        k, static_cast<const Piece *>(v), k_pages, static_cast<Piece *>(v_pages), c, parent,   \
        leaf, granted, accepted, path, status, p.N, p.H, p.C, p.dK, bytes / (int)sizeof(Piece))
    if (bytes % 16 == 0) ZETA_ACCEPT(uint4);
    else if (esz == 4) ZETA_ACCEPT(uint32_t);
    else ZETA_ACCEPT(uint16_t);
#undef ZETA_ACCEPT
    return cudaGetLastError();
}

}  // namespace zeta
